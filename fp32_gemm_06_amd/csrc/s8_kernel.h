// C <- act(sA_i sB_j (A B^T)_ij + beta C_ij + bias_j) for 8-bit codes, on the
// integer matrix cores: A is M x K, B is N x K (a linear layer's weight), both
// with k contiguous.  The products of codes and their sums are exact in 32
// bits (K is at most 131071), so every split of K gives the same C.
//
// A workgroup owns a BM x BN tile of C and walks K in stages of KS slices of
// SB bytes, a slice for each of KS groups of waves, whose sums meet in LDS at
// the end.  NST stages of LDS: while one is multiplied, the next NST - 1 are
// on their way.
//
// LDS.  A slice is a row of SB / 16 16-byte chunks for each row of the operand,
// chunk c of row p at position c ^ swizzle(p), which spreads the chunks that
// a ds_read_b128 reads together over the banks.  The 128-bit path
// writes it with buffer loads straight into LDS; the other path loads through
// registers, at any alignment, into the same places.
//
// Matrix cores.  The weight's rows are the instruction's rows and A's rows its
// columns, so a lane ends up with several n of one m: C is row-major, and
// those are next to each other in it.  Which n they are is ours to choose, by
// which row of B is put where in LDS: a lane gets runs of 8 columns, a 16-byte
// store of 16-bit values or two of 32-bit ones, and neighbouring lanes
// neighbouring runs.
//
// K need not be a multiple of 16 on the 128-bit path: the last chunk of a row
// of A is cleared past K in LDS, and what B's holds there meets zeros.
#pragma once

#include "s8_common.h"

namespace fp32gemm {
namespace {

template <int BM_, int BN_, int WM_, int WN_, int KS_, int NST_, bool AHEAD_>
struct S8Tile {
  static constexpr bool AHEAD = AHEAD_;             // operands a step ahead, in two register sets
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KS = KS_, NST = NST_;
  static constexpr int SB = 128, CP = SB / 16;     // bytes and chunks of a row of a slice
  static constexpr int RL = 1024 / SB;             // rows of a 1 KB load
  static constexpr int WAVES_N = BN / WN;
  static constexpr int WT = (BM / WM) * WAVES_N;  // waves per K group
  static constexpr int WAVES = WT * KS;
  static constexpr int NT = WAVES * 64;
  static constexpr int TM = WM / 16, TN = WN / 16;  // 16 x 16 blocks of a wave
  static constexpr int STEPS = SB / 64;             // instructions a block takes per slice
  static constexpr int RUN = TN % 2 == 0 ? 8 : 4;   // columns next to each other in a lane
  static constexpr int SLICE = (BM + BN) * SB;    // bytes
  static constexpr int STAGE = SLICE * KS;
  static constexpr int NIA = KS * BM / RL / WAVES;  // 1 KB loads per wave per stage
  static constexpr int NIB = KS * BN / RL / WAVES;
  // Stages in registers on the path that loads through them (one more each
  // than 3 / 2 / 1 takes 2 to 5% off the small tiles and spills on the
  // largest).  Three leave 192x128 one workgroup a CU there (162 registers),
  // which has two on the 128-bit path.
  static constexpr int REG = NIA + NIB <= 4 ? 4 : NIA + NIB <= 6 ? 3 : 1;
  // One wave a K group: it loads what it reads, and nothing is shared before the end.
  static constexpr bool OWN = WT == 1;
  static_assert(BM % WM == 0 && BN % WN == 0 && WM % 16 == 0 && WN % 16 == 0, "wave tiling");
  static_assert(KS * BM / RL % WAVES == 0 && KS * BN / RL % WAVES == 0, "whole loads per wave");
  static_assert(NST >= 2 && NST * STAGE <= 160 * 1024, "LDS of a CU");
  static_assert((KS - 1) * BM * BN * 4 <= NST * STAGE, "the K groups' sums fit in the buffers");
  static_assert((NST - 1) * (NIA + NIB) <= 63, "vmcnt");
  static_assert(STEPS % 2 == 0, "operands in two register sets");
};

// Wait until at most N of this wave's memory operations are in flight.
template <int N> __device__ __forceinline__ void s8_wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0F70);
}

// What the chunk positions of row p are exclusive-ored with.  A ds_read_b128
// takes 16 lanes a cycle (0-3, 12-15, 20-23 and 24-27, and so on): rows 0-3
// and 12-15 at chunk c and rows 4-11 at chunk c + 1, c even.  Row and position
// together have to put their 16 chunks in different ones of the 64 banks.
// Counted on gfx950: no conflicts.
__device__ __forceinline__ int s8_swizzle(int p) { return p & 7; }

// The column, within a wave's WN, of row r of block j: runs of RUN columns in
// the registers of a lane, neighbouring runs in neighbouring lanes.
template <class T> __device__ __forceinline__ int s8_column(int j, int r) {
  if constexpr (T::RUN == 8) return 32 * (j >> 1) + 8 * (r >> 2) + 4 * (j & 1) + (r & 3);
  else return 16 * j + r;
}

__device__ __forceinline__ void s8_dma16(__amdgpu_buffer_rsrc_t rs, char *dst, uint32_t off, int soff) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) void lds_void_t;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)dst, 16, off, soff, 0, 0);
#else
  (void)rs; (void)dst; (void)off; (void)soff;
#endif
}

// 16 codes of a row of K from any address (the hardware takes wide accesses at
// any alignment), zero past the first `valid` of them, which end the row.  The
// row's last 16 are read then and moved down; only a row shorter than that is
// read byte by byte.
__device__ __forceinline__ intx4 s8_load16(const int8_t *p, int valid, int K) {
  typedef int anywhere __attribute__((ext_vector_type(4), aligned(1)));
  typedef unsigned long long longx2 __attribute__((ext_vector_type(2)));
  intx4 v = {0, 0, 0, 0};
  if (valid >= 16) {
    v = *reinterpret_cast<const anywhere *>(p);
  } else if (valid > 0) {
    if (K >= 16) {
      v = *reinterpret_cast<const anywhere *>(p + valid - 16);
      const longx2 w = __builtin_bit_cast(longx2, v);
      const unsigned long long lo = w[0], hi = w[1];
      const int bits = 8 * (16 - valid);  // 8 .. 120
      const longx2 moved = {bits < 64 ? lo >> bits | hi << (64 - bits) : hi >> (bits - 64),
                            bits < 64 ? hi >> bits : 0ull};
      v = __builtin_bit_cast(intx4, moved);
    } else {
#pragma unroll
      for (int e = 0; e < 15; ++e)
        if (e < valid) v[e / 4] |= (int)(uint8_t)p[e] << (8 * (e % 4));
    }
  }
  return v;
}

// One float at a byte offset of a buffer (kOob: zero).
__device__ __forceinline__ float s8_float(__amdgpu_buffer_rsrc_t rs, uint32_t off) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rs, off, 0, 0));
}

// N floats from p, zeros past the first n of them (which are all there is).
template <int N> struct Floats {
  typedef float type __attribute__((ext_vector_type(N)));
  typedef float anywhere __attribute__((ext_vector_type(N), aligned(4)));
};
template <int N> __device__ __forceinline__ void s8_floats(const float *p, int n, float (&v)[N]) {
  typename Floats<N>::type w = {};
  if (n >= N) {
    w = *reinterpret_cast<const typename Floats<N>::anywhere *>(p);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < n) w[e] = p[e];
  }
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = w[e];
}

// sum sa sb + bias.  The first product may pass fp32's range where the whole
// does not.  It cannot up to this sa, since a sum is at most 2^31.  Above it sa
// is taken times 2^-32, which is exact, and the 2^32 comes back with the bias.
// Nothing is lost at the lower end: sum sa is then zero or at least 2^64, and
// its product with the smallest sb still normal.  The branch costs nothing that
// shows (4096^3 fp32 out 64.0 us without it and 64.2, 256 x 4096 x 4096 11.4
// both).
constexpr float kWideScale = 0x1p96f;
__device__ __forceinline__ bool s8_wide(float sa) { return __builtin_fabsf(sa) > kWideScale; }
template <bool ANY_WIDE>
__device__ __forceinline__ float s8_scaled(int sum, float sa, float sb, float bias) {
  if constexpr (!ANY_WIDE) return __builtin_fmaf((float)sum * sa, sb, bias);
  const float x = (float)sum * (s8_wide(sa) ? sa * 0x1p-32f : sa);
  return s8_wide(sa) ? __builtin_fmaf(x * sb, 0x1p32f, bias) : __builtin_fmaf(x, sb, bias);
}

// A run of columns of C: scaled sums and bias in v, plus beta C, through the
// activation, in 32 bits, rounded once to C's type.  `cols`: the run's columns
// that are in C.  Wide accesses at any alignment of the element.
template <class F, int RUN>
__device__ __forceinline__ void s8_finish_run(const S8Args &a, F *c, int cols, float (&v)[RUN]) {
  typedef F fr __attribute__((ext_vector_type(RUN)));
  typedef F anywhere __attribute__((ext_vector_type(RUN), aligned(alignof(F))));
  fr w = {};
  if (a.beta != 0.0f) {
    if (cols >= RUN) {
      w = *reinterpret_cast<const anywhere *>(c);
    } else {
#pragma unroll
      for (int e = 0; e < RUN; ++e)
        if (e < cols) w[e] = c[e];
    }
#pragma unroll
    for (int e = 0; e < RUN; ++e) v[e] = __builtin_fmaf(a.beta, (float)w[e], v[e]);
  }
  if (a.act != kActNone) {
#pragma unroll
    for (int e = 0; e < RUN; ++e) v[e] = apply_act(v[e], kActRelu);
  }
#pragma unroll
  for (int e = 0; e < RUN; ++e) w[e] = (F)v[e];
  if (cols >= RUN) {
    *reinterpret_cast<anywhere *>(c) = w;
  } else {
#pragma unroll
    for (int e = 0; e < RUN; ++e)
      if (e < cols) c[e] = w[e];
  }
}

// One element of C, the same way.
template <class F> __device__ __forceinline__ void s8_finish_one(const S8Args &a, F *c, float v) {
  if (a.beta != 0.0f) v = __builtin_fmaf(a.beta, (float)*c, v);
  *c = (F)apply_act(v, a.act);
}

template <class T, bool DMA>
__global__ void __launch_bounds__(T::NT) s8_kernel(S8Args a, int tiles_m, int tiles_n, int group_m) {
  constexpr int BM = T::BM, BN = T::BN, KS = T::KS;
  // (the register path uses two of the NST stages)
  __shared__ __attribute__((aligned(16))) char lds[T::NST * T::STAGE];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kg = wave / T::WT, wt = wave % T::WT;
  const int wm = wt / T::WAVES_N, wn = wt % T::WAVES_N;

  // Workgroups go to the 8 XCDs in turn; logical ids give each XCD a run of
  // neighbouring tiles, in strips of group_m tile rows.
  const int G = gridDim.x;
  const int xcd = (int)blockIdx.x & 7;
  const int lid = xcd * (G >> 3) + min(xcd, G & 7) + ((int)blockIdx.x >> 3);
  const int strip = lid / (group_m * tiles_n);
  const int gsz = min(tiles_m - strip * group_m, group_m);
  const int within = lid - strip * group_m * tiles_n;
  const int m0 = (strip * group_m + within % gsz) * BM;
  const int n0 = (within / gsz) * BN;
  const int rows = a.M - m0, cols = a.N - n0;
  const int8_t *Ag = a.A + (size_t)m0 * a.lda;
  const int8_t *Bg = a.B + (size_t)n0 * a.ldb;

  constexpr int SB = T::SB;
  const int nst = (a.K + SB * KS - 1) / (SB * KS);
  const int klast = a.K - (nst - 1) * SB * KS;  // valid k of the last stage

  // Lane l of load `inst` moves the chunk at position l % CP of LDS row
  // RL inst + l / CP, counted over a slice's rows and then the stage's slices:
  // neighbouring lanes read a row's neighbouring chunks.
  const int pos = lane % T::CP;
  uint32_t offa[T::NIA], offb[T::NIB];
  int cola[T::NIA], colb[T::NIB];
  int rowa[T::NIA], rowb[T::NIB];
#pragma unroll
  for (int q = 0; q < T::NIA; ++q) {
    const int f = (wave * T::NIA + q) * T::RL + lane / T::CP;
    rowa[q] = f % BM;
    cola[q] = f / BM * SB + 16 * (pos ^ s8_swizzle(f % BM));
  }
#pragma unroll
  for (int q = 0; q < T::NIB; ++q) {
    const int f = (wave * T::NIB + q) * T::RL + lane / T::CP;
    const int p = f % BN;
    rowb[q] = p / T::WN * T::WN + s8_column<T>(p % T::WN / 16, p % 16);
    colb[q] = f / BN * SB + 16 * (pos ^ s8_swizzle(p));
  }
  auto set_offsets = [&](int kvalid) {
#pragma unroll
    for (int q = 0; q < T::NIA; ++q)
      offa[q] = rowa[q] < rows && cola[q] < kvalid ? (uint32_t)(rowa[q] * a.lda + cola[q]) : kOob;
#pragma unroll
    for (int q = 0; q < T::NIB; ++q)
      offb[q] = rowb[q] < cols && colb[q] < kvalid ? (uint32_t)(rowb[q] * a.ldb + colb[q]) : kOob;
  };
  // where a load goes: 1 KB a load, over the slices' operand areas
  auto dst_a = [&](int q) -> int {
    const int f = (wave * T::NIA + q) * T::RL;
    return f / BM * T::SLICE + f % BM * SB;
  };
  auto dst_b = [&](int q) -> int {
    const int f = (wave * T::NIB + q) * T::RL;
    return f / BN * T::SLICE + BM * SB + f % BN * SB;
  };

  const __amdgpu_buffer_rsrc_t rs_a = make_rsrc(Ag);
  const __amdgpu_buffer_rsrc_t rs_b = make_rsrc(Bg);
  // The register path: D stages' global loads in registers, and the writes to
  // LDS.  Rows past the matrix read its last row instead (they are multiplied,
  // and not stored), so only the last stage has anything to mask.
  constexpr int D = DMA ? 1 : T::REG;
  struct Regs {
    intx4 a[DMA ? 1 : T::NIA], b[DMA ? 1 : T::NIB];
  };
  Regs ring[D];
  (void)ring;
  auto fetch = [&](Regs &f, int st) {
    if constexpr (!DMA) {
      const int k0 = st * SB * KS;
      const bool inside = st + 1 < nst;
#pragma unroll
      for (int q = 0; q < T::NIA; ++q) {
        const int8_t *p = Ag + k0 + (uint32_t)(min(rowa[q], rows - 1) * a.lda + cola[q]);
        f.a[q] = s8_load16(p, inside ? 16 : a.K - k0 - cola[q], a.K);
      }
#pragma unroll
      for (int q = 0; q < T::NIB; ++q) {
        const int8_t *p = Bg + k0 + (uint32_t)(min(rowb[q], cols - 1) * a.ldb + colb[q]);
        f.b[q] = s8_load16(p, inside ? 16 : a.K - k0 - colb[q], a.K);
      }
    }
  };
  auto commit = [&](const Regs &f, char *buf) {
    if constexpr (!DMA) {
#pragma unroll
      for (int q = 0; q < T::NIA; ++q) *reinterpret_cast<intx4 *>(buf + dst_a(q) + 16 * lane) = f.a[q];
#pragma unroll
      for (int q = 0; q < T::NIB; ++q) *reinterpret_cast<intx4 *>(buf + dst_b(q) + 16 * lane) = f.b[q];
    } else {
      (void)f; (void)buf;
    }
  };
  // Publishes a stage to the waves that share it, or frees its buffer: this
  // wave's LDS accesses are done, and the others' too.  (Not __syncthreads,
  // whose fence may wait for the loads in flight as well.)
  auto meet = [&]() {
    if constexpr (T::OWN) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    else asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  // After the last stage has landed: the chunk of A's rows that K ends in.
  auto clear_tail = [&](char *buf) {
    if constexpr (DMA) {
      if ((a.K & 15) == 0 || (T::OWN && kg != klast / SB)) return;
      for (int p = T::OWN ? lane : tid; p < BM; p += T::OWN ? 64 : T::NT) {
        intx4 *c = reinterpret_cast<intx4 *>(buf + klast / SB * T::SLICE + p * SB +
                                             16 * ((klast % SB / 16) ^ s8_swizzle(p)));
        intx4 v = *c;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int keep = (klast & 15) - 4 * d;  // bytes of this word inside K
          v[d] = keep >= 4 ? v[d] : keep <= 0 ? 0 : v[d] & (int)((1u << (8 * keep)) - 1);
        }
        *c = v;
      }
      meet();
    } else {
      (void)buf;
    }
  };

  intx4 acc[T::TM][T::TN];
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j) acc[i][j] = intx4{0, 0, 0, 0};

  const int lr = lane & 15, lq = lane >> 4;
  const int pa = wm * T::WM + lr, pb = wn * T::WN + lr;  // LDS rows of block 0
  // The operands of one instruction step of every block.
  struct Frag {
    intx4 a[T::TM], b[T::TN];
  };
  auto read = [&](const char *buf, int step, Frag &f) {
    const char *As = buf + kg * T::SLICE, *Bs = As + BM * SB;
    const int c = 4 * step + lq;
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
      f.b[j] = *reinterpret_cast<const intx4 *>(Bs + (pb + j * 16) * SB +
                                                16 * (c ^ s8_swizzle(pb + j * 16)));
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
      f.a[i] = *reinterpret_cast<const intx4 *>(As + (pa + i * 16) * SB +
                                                16 * (c ^ s8_swizzle(pa + i * 16)));
  };
  auto mma_row = [&](const Frag &f, int i) {
#pragma unroll
    for (int j = 0; j < T::TN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[j], f.a[i], acc[i][j], 0, 0, 0);
  };
  Frag fr[2];

  if constexpr (DMA) {
    // NST stages in LDS.  A load instruction waits for its place in the
    // memory pipeline, and the wave with it, so a stage's loads follow the
    // barrier that freed their buffer a few at a time, between the first half
    // of the matrix instructions that follow it too.  Past the end of K the
    // loads are masked, so the count of them in flight stays.  The scheduling
    // barriers keep the order written here.  At 4096^3, 256 x 256 tiles of 8
    // waves: all loads first, then reads and instructions as the compiler
    // orders them, 1.75 us a stage; spread and read ahead 1.59; with the order
    // kept 1.49 (the instructions and LDS reads alone 1.24, the loads alone
    // 1.02).
    constexpr int NST = T::NST, NL = T::NIA + T::NIB, STEPS = T::STEPS;
    constexpr int PER_ROW = T::TM == 1 ? NL : (NL + T::TM / 2 - 1) / (T::TM / 2);
    auto load = [&](int q, char *buf, int st) {
      const int k0 = st * SB * KS;
      if (q < T::NIA) s8_dma16(rs_a, buf + dst_a(q), offa[q < T::NIA ? q : 0], k0);
      else s8_dma16(rs_b, buf + dst_b(q - T::NIA), offb[q >= T::NIA ? q - T::NIA : 0], k0);
    };
    auto mask_stage = [&](int st) {
      if (st == nst - 1) set_offsets(klast);
      else if (st == nst) set_offsets(0);
    };
    // one step's instructions, and stage st's loads into buf between them
    auto multiply_and_load = [&](const Frag &f, char *buf, int st) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < T::TM; ++i) {
        mma_row(f, i);
#pragma unroll
        for (int q = i * PER_ROW; q < (i + 1) * PER_ROW && q < NL; ++q) load(q, buf, st);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // stages in flight before the first is multiplied
    constexpr int FIRST = T::AHEAD ? NST : NST - 1;
    if (nst > 1) set_offsets(SB * KS);
#pragma unroll
    for (int st = 0; st < FIRST; ++st) {
      mask_stage(st);
#pragma unroll
      for (int q = 0; q < NL; ++q) load(q, lds + st * T::STAGE, st);
    }
    int at = 0;  // buffer of stage st
    if constexpr (T::AHEAD) {
      // The last step's instructions run after the barrier and cover the
      // first reads of the next stage.
      s8_wait_vm<(NST - 1) * NL>();
      meet();
      if (nst == 1) clear_tail(lds);
      read(lds, 0, fr[0]);
      for (int st = 0; st < nst; ++st) {
        char *cur = lds + at * T::STAGE;
#pragma unroll
        for (int s = 0; s + 1 < STEPS; ++s) {
          read(cur, s + 1, fr[(s + 1) & 1]);
#pragma unroll
          for (int i = 0; i < T::TM; ++i) mma_row(fr[s & 1], i);
        }
        s8_wait_vm<(NST - 2) * NL>();  // stage st + 1 has landed
        meet();                        // for every wave, and this stage's buffer is free
        at = at + 1 == NST ? 0 : at + 1;
        if (st + 1 < nst) {
          if (st + 2 == nst) clear_tail(lds + at * T::STAGE);
          read(lds + at * T::STAGE, 0, fr[0]);
        }
        mask_stage(st + NST);
        multiply_and_load(fr[(STEPS - 1) & 1], cur, st + NST);
      }
    } else {
      // One register set: four waves on a SIMD cover each other's reads.
      for (int st = 0; st < nst; ++st) {
        char *cur = lds + at * T::STAGE;
        char *old = lds + (at == 0 ? NST - 1 : at - 1) * T::STAGE;
        s8_wait_vm<(NST - 2) * NL>();  // this stage has landed
        meet();                        // for every wave, and the buffer of the one before is free
        if (st + 1 == nst) clear_tail(cur);
        mask_stage(st + NST - 1);
        read(cur, 0, fr[0]);
        multiply_and_load(fr[0], old, st + NST - 1);
#pragma unroll
        for (int s = 1; s < STEPS; ++s) {
          read(cur, s, fr[0]);
#pragma unroll
          for (int i = 0; i < T::TM; ++i) mma_row(fr[0], i);
        }
        at = at + 1 == NST ? 0 : at + 1;
      }
    }
    s8_wait_vm<0>();  // the masked loads have written their zeros
  } else {
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (u < nst) fetch(ring[u], u);
    for (int s0 = 0; s0 < nst; s0 += D) {
#pragma unroll
      for (int u = 0; u < D; ++u) {
        const int st = s0 + u;
        if (st >= nst) break;
        char *cur = lds + (st & 1) * T::STAGE;
        commit(ring[u], cur);
        meet();
        if (st + D < nst) fetch(ring[u], st + D);
#pragma unroll
        for (int s = 0; s < T::STEPS; ++s) {
          read(cur, s, fr[0]);
#pragma unroll
          for (int i = 0; i < T::TM; ++i) mma_row(fr[0], i);
        }
      }
    }
  }
  __syncthreads();

  // K groups 1.. leave their sums in LDS (free since the last barrier), group
  // 0 adds them.
  if constexpr (KS > 1) {
    constexpr int PER = T::TM * T::TN * 4 * 64;
    int *red = reinterpret_cast<int *>(lds);
    if (kg > 0) {
      int *mine = red + ((kg - 1) * T::WT + wt) * PER + lane;
#pragma unroll
      for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) mine[((i * T::TN + j) * 4 + v) * 64] = acc[i][j][v];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 1; g < KS; ++g) {
      const int *theirs = red + ((g - 1) * T::WT + wt) * PER + lane;
#pragma unroll
      for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][j][v] += theirs[((i * T::TN + j) * 4 + v) * 64];
    }
  }

  // Epilogue.  A lane has RUN columns at a time of one row.  What it costs is
  // instructions (64 elements a lane of a 256 x 256 tile): the conversion, a
  // multiplication, a fused one with the bias, the rounding, and the rest only
  // where it is asked for.
  constexpr int RUN = T::RUN, RUNS = T::TN * 4 / RUN;
  // the column of run t, and its sums of block row i
  auto run_col = [&](int t) -> int { return wn * T::WN + 4 * RUN * t + RUN * lq; };
  auto run_sum = [&](int i, int t, int e) -> int {
    if constexpr (RUN == 8) return acc[i][2 * t + (e >> 2)][e & 3];
    else return acc[i][t][e];
  };
  float sb[RUNS][RUN], bias[RUNS][RUN] = {};
#pragma unroll
  for (int t = 0; t < RUNS; ++t) s8_floats<RUN>(a.sB + n0 + run_col(t), cols - run_col(t), sb[t]);
  if (a.bias != nullptr) {
#pragma unroll
    for (int t = 0; t < RUNS; ++t) s8_floats<RUN>(a.bias + n0 + run_col(t), cols - run_col(t), bias[t]);
  }
  const __amdgpu_buffer_rsrc_t rs_sa = make_rsrc(a.sA + m0);
  float sa[T::TM];
#pragma unroll
  for (int i = 0; i < T::TM; ++i) {
    const int m = wm * T::WM + i * 16 + lr;
    sa[i] = s8_float(rs_sa, m < rows ? 4u * m : kOob);
  }
  auto finish = [&](auto zero) {
    typedef decltype(zero) F;
    F *Cg = static_cast<F *>(a.C) + (size_t)m0 * a.ldc + n0;
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
      const int m = wm * T::WM + i * 16 + lr;
      const bool any_wide = __any(s8_wide(sa[i]));  // rare, and one branch for the wave
#pragma unroll
      for (int t = 0; t < RUNS; ++t) {
        const int col = run_col(t);
        float v[RUN];
        if (any_wide) {
#pragma unroll
          for (int e = 0; e < RUN; ++e) v[e] = s8_scaled<true>(run_sum(i, t, e), sa[i], sb[t][e], bias[t][e]);
        } else {
#pragma unroll
          for (int e = 0; e < RUN; ++e) v[e] = s8_scaled<false>(run_sum(i, t, e), sa[i], sb[t][e], bias[t][e]);
        }
        if (m < rows && col < cols)
          s8_finish_run<F, RUN>(a, Cg + (uint32_t)(m * a.ldc + col), cols - col, v);
      }
    }
  };
  if (a.type == kTypeF32) finish(0.0f);
  else if (a.type == kTypeF16) finish((_Float16)0.0f);
  else finish((__bf16)0.0f);
}

// 16-byte loads of whole chunks: rows that start at multiples of 16 bytes.
// The chunk that K ends in is read whole.  It lies inside its row's lda or ldb
// bytes, multiples of 16 there; behind the last row, whose codes may end at K,
// it is the aligned 16 bytes that hold the last code, so no page without one
// is touched, and what it reads is multiplied by zeros.
inline bool s8_dma_ok(const S8Args &a) {
  return (uintptr_t)a.A % 16 == 0 && (uintptr_t)a.B % 16 == 0 && a.lda % 16 == 0 && a.ldb % 16 == 0;
}

// T on rows of 16-byte chunks, TR (the same tile) through registers.
template <class T, class TR> hipError_t s8_launch(const S8Args &a, hipStream_t s) {
  const int tm = (a.M + T::BM - 1) / T::BM, tn = (a.N + T::BN - 1) / T::BN;
  constexpr int group_m = 4;
  if (s8_dma_ok(a))
    s8_kernel<T, true><<<tm * tn, T::NT, 0, s>>>(a, tm, tn, group_m);
  else
    s8_kernel<TR, false><<<tm * tn, TR::NT, 0, s>>>(a, tm, tn, group_m);
  return hipGetLastError();
}

}  // namespace
}  // namespace fp32gemm
