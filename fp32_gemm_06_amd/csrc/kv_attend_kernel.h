// Attention of one new token for each of B sequences over the paged cache:
//
//   s_t = scale q . k_t,   o = sum_t exp(s_t) v_t / sum_t exp(s_t)
//
// over the tokens t that the sequence's length, the window and the page table
// leave.  One pass over K and V with a running maximum and sum.
//
// Work.  A unit is 4 TOK tokens of one key head (and up to 16 of its query
// heads) of one sequence.  Every workgroup adds up all sequences' units from
// their lengths, and takes an equal run of them, across heads and sequences:
// the lengths stay on the GPU, a captured graph follows them, and one long
// sequence among short ones is spread over all CUs.  The four waves take TOK
// tokens each and keep their own maximum, sum and output until the run leaves
// the head; then they are joined in LDS.  A head that several workgroups
// share is joined in the order of its tokens by the last of them to arrive, or
// in two or three steps, each by the last of its own parts' workgroups
// (partial results and arrival counters as in gemv_split.hip: agent-scope
// atomic stores and loads, a wait for the own stores before the counter, no
// fences, no spinning).  The result depends on the lengths and the launch
// alone.
//
// Products.  16 query heads (columns) by 16 tokens (rows) a matrix
// instruction, scores transposed: lane (n, g) = (lane % 16, lane / 16) holds
// head n's scores of tokens 16 blk + 4 g + i, and the second product takes
// its weights from where they are: its k slots are numbered to be those
// tokens, V's operand is loaded in the same numbering, and no value crosses
// lanes but for the maximum.  The operand of V wants a column of 16 (8, 4)
// tokens in a lane, memory has rows; a lane loads the tokens' pieces of 8
// columns, a whole line for 16 lanes, and turns them with byte permutations.
//
//  codes (s8): both products in integers.  The query's row, and each tile's
//    weights times V's scales, become fixed-point numbers relative to their
//    own largest, in three signed 8-bit digits (23 bits).  Two digits, 15 bits,
//    are too few for 16-bit outputs as well: a token whose scale is 512 times
//    the others' leaves those 6 bits, an error of .5% in the columns where its
//    own codes are small; with three it is 2^-15.  No code of the cache is
//    converted.
//  16-bit floats: products of the type, sums in fp32.  A weight goes in as two
//    numbers of the type (its rounding and what that left), 16 bits or more.
//  fp32: fp32 matrix instructions.
//
// Masked tokens get a score of minus infinity and weight 0 by selection; where
// V is floats their values are selected away too, so whatever unwritten pages
// hold does no harm.
//
// Long calls are bound by reading K and V once (counted: 1.01 times their bytes):
// 64 ragged sequences up to 8192 tokens, 32 heads on 8 of 128, codes 82.4 us (5.5
// TB/s; vector units half of the cycles busy, matrix cores an eighth), bf16 142 us
// (6.2 TB/s; a kernel that only reads such pages 6.3-6.7).  Few rows are bound by
// latency: one sequence of 4096 on codes 11.3 us; when it was 10.9, with a digit
// less, planning took .8, the first bytes 2.2, the tile 2.3, the waves' join and
// the stores 1.3, the counter .4, the join of 16 parts 1.9 and the launch the rest.
#pragma once

#include "kv_common.h"

namespace fp32gemm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_words __attribute__((aligned(4)));

constexpr float kNegInf = -__builtin_inff();
constexpr int kScoreBias16 = 15;  // fp16 weights are kept times 2^15: their second numbers stay normal

__device__ __forceinline__ float nan_max(float a, float b) {  // NaN if either is
  return __builtin_elementwise_maximum(a, b);
}
// Over the four lanes of a query head (lane ^ 16, ^ 32).
template <class F> __device__ __forceinline__ float over_groups(float v, F f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto p = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const float u = f(__builtin_bit_cast(float, (uint32_t)p[0]), __builtin_bit_cast(float, (uint32_t)p[1]));
  const uint32_t d = __builtin_bit_cast(uint32_t, u);
  const auto q = __builtin_amdgcn_permlane32_swap(d, d, false, false);
  return f(__builtin_bit_cast(float, (uint32_t)q[0]), __builtin_bit_cast(float, (uint32_t)q[1]));
}
__device__ __forceinline__ float fmax_groups(float v) {
  return over_groups(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ float nanmax_groups(float v) {
  return over_groups(v, [](float a, float b) { return nan_max(a, b); });
}
__device__ __forceinline__ float sum_groups(float v) {
  return over_groups(v, [](float a, float b) { return a + b; });
}

// Three signed 8-bit digits of v inv, to the nearest integer: that plus 0x80 in
// every digit, whose bytes, 0x80 taken off again, are the digits.  A row's or
// tile's largest becomes kTop.  The integer is rounded by itself: below 2^23, so
// for most negative numbers, the sum would have a half of its own to cut off.
constexpr int kDigits = 3;
constexpr float kTop = 8355000.0f;
__device__ __forceinline__ void digits4(const float (&v)[4], float inv, uint32_t (&w)[kDigits]) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = (uint32_t)(__builtin_rintf(v[e] * inv) + 8421504.0f);
  const uint32_t t = __builtin_amdgcn_perm(u[1], u[0], 0x05010400u);
  const uint32_t s = __builtin_amdgcn_perm(u[3], u[2], 0x05010400u);
  w[0] = __builtin_amdgcn_perm(s, t, 0x05040100u) ^ 0x80808080u;
  w[1] = __builtin_amdgcn_perm(s, t, 0x07060302u) ^ 0x80808080u;
  const uint32_t t2 = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0602u);
  const uint32_t s2 = __builtin_amdgcn_perm(u[3], u[2], 0x0c0c0602u);
  w[2] = __builtin_amdgcn_perm(s2, t2, 0x05040100u) ^ 0x80808080u;
}

// A product with fixed-point numbers: two digits' products one behind the other
// in the same accumulator, moved up a digit in between (they stay below
// 2^31: 256 products of 127 and 128, or 64), the third beside it.
template <int K> __device__ __forceinline__ floatx4 digit_product(const u32x4 (&x)[K], const u32x4 *w) {
  intx4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
  auto add = [&](intx4 &acc, int digit) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, x[j]),
                                                  __builtin_bit_cast(intx4, w[digit * K + j]), acc, 0, 0, 0);
  };
  add(hi, 2);
  hi <<= 8;
  add(hi, 1);
  add(lo, 0);
  floatx4 v;
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(256.0f, (float)hi[r], (float)lo[r]);
  return v;
}

template <bool V> struct Flag { static constexpr bool value = V; };
template <int V> struct Number { static constexpr int value = V; };

template <class T, bool S8> struct Kind;
template <class T> struct Kind<T, true> { static constexpr int ES = 1, TOK = 64, QDIG = kDigits; };
template <> struct Kind<float, false> { static constexpr int ES = 4, TOK = 16, QDIG = 1; };
template <class T> struct Kind<T, false> { static constexpr int ES = 2, TOK = 32, QDIG = 1; };

template <class T> __device__ __forceinline__ floatx4 mfma16(u32x4 a, u32x4 b, floatx4 c) {
  typedef T frag __attribute__((ext_vector_type(8)));
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
}

// What a partial result with maximum m and sum l counts for under the maximum
// of all; nothing where it saw no token.
__device__ __forceinline__ float weight_of(float m, float l, float all) {
  return m == kNegInf && l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - (all == kNegInf ? 0.0f : all));
}

// Stores through this XCD's L2 and loads past it, as relaxed atomics of agent
// scope are made (the sc1 bit), four words at a time.
constexpr int kThrough = 16, kNontemporal = 2;
__device__ __forceinline__ void store_through(floatx4 v, __amdgpu_buffer_rsrc_t r, uint32_t at) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at, 0, kThrough);
}
__device__ __forceinline__ void store_through(float v, __amdgpu_buffer_rsrc_t r, uint32_t at) {
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, v), r, at, 0, kThrough);
}
__device__ __forceinline__ floatx4 load_through4(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kThrough));
}
__device__ __forceinline__ float load_through(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, kThrough));
}

// Loads are issued on their side of this: a wait for all but the last N counts
// on the order in which they were asked for, and the compiler, which sees no
// dependence between loads into LDS and into registers, moves them past each
// other (heads below 64 on odd pages had 3 of K's 4 loads behind half of V's).
__device__ __forceinline__ void keep_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Waits until all but the last N of the wave's memory accesses are done.
template <int N> __device__ __forceinline__ void wait_loads() {
  static_assert(N <= 63, "six bits");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// 16 bytes a lane from memory into LDS, at dst + 16 lane, not kept in the
// caches.  (Behind the other form the compiler waits for all loads at once.)
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint32_t off, char *dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)dst, 16, off, 0, 0, kNontemporal);
#else
  (void)r; (void)off; (void)dst;
#endif
}
__device__ __forceinline__ void load_lds16(const char *src, char *dst) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef __attribute__((address_space(1))) const void global_void;
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_global_load_lds((global_void *)src, (lds_void *)dst, 16, 0, kNontemporal);
#else
  (void)src; (void)dst;
#endif
}

// Where in its row of CP pieces a piece of K lies (exclusive-ored with this).
// A cycle of ds_read_b128 takes rows 0-3 and 12-15 at an even piece and rows
// 4-11 at the one behind it (or the other way round), and 16 pieces fill the
// banks.
template <int CP> __device__ __forceinline__ int key_turn(int row) {
  return CP == 4 ? (row & 8 ? 3 : 0) : CP == 8 ? row & 7 : row & 15;
}

// One word at an address that is the same in all lanes, by the scalar unit.
__device__ __forceinline__ int load_uniform(const int *p) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef const __attribute__((address_space(4))) int constant_int;
  return *(constant_int *)p;
#else
  return *p;
#endif
}

// The sum of the lanes up to one's own.
template <int CTRL, int ROWS> __device__ __forceinline__ int lane_below(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int sum_to_lane(int v) {
  v += lane_below<0x111, 0xf>(v);  // from 1, 2, 4, 8 lanes below in a row of 16
  v += lane_below<0x112, 0xf>(v);
  v += lane_below<0x114, 0xf>(v);
  v += lane_below<0x118, 0xf>(v);
  v += lane_below<0x142, 0xa>(v);  // lane 15 of a row to the next row
  v += lane_below<0x143, 0xc>(v);  // lane 31 to the upper half
  return v;
}

// A sequence's units and where its tokens start: lo .. n are seen.
template <int UNIT> struct Span {
  int lo, n, base, units;
  __device__ __forceinline__ Span(const AttendArgs &a, int length) {
    n = length < 0 ? 0 : length > a.most ? a.most : length;
    lo = a.window > 0 && n > a.window ? n - a.window : 0;
    base = lo & ~63;
    units = (n - base + UNIT - 1) / UNIT;
    units = units < 1 ? 1 : units;  // an empty sequence's outputs are written too
  }
};

// B16: a page holds whole blocks of 16 tokens, so a block's address is the
// wave's; else every token has its own.  FULL: heads have DC values, not fewer.
// DC is DP, a power of two, but for heads of 192, whose rows have the places of
// 256 in LDS while queries, scores, V and outputs are done without the rest
// (64 ragged to 8192, 20 heads on 4: codes 97 -> 79 us, fp32 268 -> 240).
template <class T, bool S8, int DP, int DC, bool B16, bool FULL>
__global__ void __launch_bounds__(256, DP > 128 ? 1 : 2) attend_kernel(AttendArgs a) {
  typedef Kind<T, S8> KD;
  constexpr int ES = KD::ES, TOK = KD::TOK, QDIG = KD::QDIG, UNIT = 4 * TOK, BLK = TOK / 16;
  // columns of V of a lane, next to each other
  constexpr int CPL = DC != DP ? S8 ? 12 : 4 : DP >= 128 ? 8 : 4;
  constexpr int HALVES = DC / (16 * CPL);      // of which there are 16 lanes
  constexpr int KF = DC * ES / 64;             // 16-byte pieces of a token's K in a lane
  constexpr int VW = CPL * ES / 4;             // words of a token's V piece
  constexpr int CP = DP * ES / 16;             // 16-byte pieces of a row of K in LDS
  constexpr int PITCH = DC + 4;                // of a head's outputs in LDS: 16 heads hit 64 banks

  // each wave's tile of K; the waves' outputs when they are joined, beside it,
  // since the next head's first tile is on its way by then
  constexpr int KT = TOK * DP * ES;  // bytes of a tile
  __shared__ __attribute__((aligned(16))) char keys_of[4][KT];
  __shared__ __attribute__((aligned(16))) float merge[4][16 * PITCH];
  __shared__ float wm[4][16], wl[4][16], part_f[16][16];
  __shared__ int scan[4], at_prefix, at_seq, last;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int rows = a.Hk * a.RG, D = FULL ? DC : a.cache.dim, ps = a.cache.page_size;

  // ---- this workgroup's run of units -----------------------------------------
  // (fewer than 2^31 units, rounded up to whole runs: checked by the caller)
  // With long runs a head's beginning and end, which cost what a unit does, are
  // counted as one more in front of its own (`over`): else the workgroup with
  // the short sequences is the last to be done (64 ragged sequences up to 8192,
  // codes: its run of 14 units took 85 us, the median 65).  With short runs the
  // rounding of the runs would cost more.
  // A few units a workgroup: where there are workgroups enough for every head
  // to begin a run of its own (`whole`), its share is rounded up to whole runs,
  // and no workgroup has parts of two heads (16 windows of 4096, 16 heads of
  // 256 fp16: 27.0 -> 24.8 us, with all parts joined at once).
  int U, over, per, u0, u1, b, prefix, length;
  bool whole_runs = false;
  auto share = [&](int units) { return whole_runs ? (units + per - 1) / per * per : units + over; };
  auto runs = [&](int units) {
    over = units >= 8 * a.groups ? 1 : 0;
    U = units + over * rows * a.B;
    per = (U + a.groups - 1) / a.groups;
  };
  auto run = [&]() {
    u0 = (int)blockIdx.x * per;
    u1 = min(U, u0 + per);
  };
  if (a.B <= 64) {  // a sequence a lane, and no wave waits for another
    const int len = lane < a.B ? a.lengths[lane] : 0;
    const int units = Span<UNIT>(a, len).units;
    int mine = lane < a.B ? units * rows : 0;
    int incl = sum_to_lane(mine);
    runs(__builtin_amdgcn_readlane(incl, 63));
    if (per > 1 && over == 0) {
      const int parts = sum_to_lane(lane < a.B ? (units + per - 1) / per * rows : 0);
      const int all = __builtin_amdgcn_readlane(parts, 63);
      whole_runs = all <= a.groups;
      if (whole_runs) U = all * per;
    }
    if (over != 0 || whole_runs) {
      mine = lane < a.B ? share(units) * rows : 0;
      incl = sum_to_lane(mine);
    }
    run();
    if (u0 >= U) return;
    b = __builtin_popcountll(__ballot(lane < a.B && incl <= u0));
    prefix = __builtin_amdgcn_readlane(incl - mine, b);
    length = __builtin_amdgcn_readlane(len, b);
  } else {
    const int each = (a.B + 255) / 256;
    int mine = 0;
    for (int j = 0; j < each; ++j) {
      const int x = tid * each + j;
      if (x < a.B) mine += Span<UNIT>(a, a.lengths[x]).units * rows;
    }
    int incl = sum_to_lane(mine);
    if (lane == 63) scan[wave] = incl;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      incl += w < wave ? scan[w] : 0;
      total += scan[w];
    }
    runs(__builtin_amdgcn_readfirstlane(total));
    run();
    if (u0 >= U) return;
    incl += over * rows * min(a.B, (tid + 1) * each);
    mine += over * rows * max(0, min(each, a.B - tid * each));
    if (incl - mine <= u0 && u0 < incl) {
      int p = incl - mine, x = tid * each;
      for (;; ++x) {
        const int t = (Span<UNIT>(a, a.lengths[x]).units + over) * rows;
        if (u0 < p + t) break;
        p += t;
      }
      at_prefix = p;
      at_seq = x;
    }
    __syncthreads();
    b = __builtin_amdgcn_readfirstlane(at_seq);
    prefix = __builtin_amdgcn_readfirstlane(at_prefix);
    length = load_uniform(a.lengths + b);
  }

  // One head's part of the run: units [i0, i1) of the head's, whose share of
  // the runs begins at `start`.  The last of a run may have none.
  struct Segment {
    Span<UNIT> sp;
    int b, prefix, start, i0, i1, head, q0, G;
  };
  auto segment = [&](int u, int b, int prefix, Span<UNIT> sp) {
    int each = share(sp.units);
    while (u >= prefix + each * rows) {
      prefix += each * rows;
      sp = Span<UNIT>(a, load_uniform(a.lengths + ++b));
      each = share(sp.units);
    }
    const int r = (u - prefix) / each, head = r / a.RG, h0 = (r - head * a.RG) * 16;
    const int start = prefix + r * each, i0 = max(0, u - start - over);
    return Segment{sp, b, prefix, start, i0, min(sp.units, u1 - start - over), head, head * a.G + h0, min(16, a.G - h0)};
  };
  Segment sg = segment(u0, b, prefix, Span<UNIT>(a, length));
  const int first_row = sg.start;

  // rows of the cache: of each block's first token (B16), and of token `lane`
  // (modulo TOK); seen: which tokens (B16: blocks) lie on a page
  struct Rows {
    uint32_t base[BLK], own;
    unsigned long long seen;
  };
  auto locate = [&](const Segment &sg, int t0) {
    Rows w;
    // the row of token t, and whether its page exists (else a row that does)
    auto row_of = [&](uint32_t t, auto load, bool &ok) {
      const int pi = (int)((uint64_t)t * a.magic >> a.shift);
      const int page = load(a.table + ((long long)sg.b * a.ldt + min(pi, a.ldt - 1)));
      ok = pi < a.ldt && page >= 0 && page < a.cache.pages;
      return (uint32_t)((ok ? page : 0) * a.cache.heads + sg.head) * ps + (t - pi * ps);
    };
    bool ok;
    if constexpr (B16) {
      w.seen = 0;
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk) {
        w.base[blk] = row_of(t0 + 16 * blk, load_uniform, ok);
        w.seen |= ok ? 0xffffull << 16 * blk : 0ull;
      }
      if constexpr (S8)
        w.own = (lane & 32 ? lane & 16 ? w.base[3] : w.base[2] : lane & 16 ? w.base[1] : w.base[0]) + n;
    } else {
      w.own = row_of(t0 + lane % TOK, [](const int *p) { return *p; }, ok);
      w.seen = __ballot(ok) & (~0ull >> (64 - TOK));
    }
    return w;
  };
  char *const kt = keys_of[wave];
  typedef uint32_t piece __attribute__((ext_vector_type(VW)));
  piece vf[BLK][4][HALVES];
  float ks = 0.0f, vs = 0.0f;  // of token `lane`
  // K's tile, straight into LDS: an instruction takes 64 pieces of 16 bytes,
  // whole rows next to each other in the page (loaded as the products want
  // them, 16 rows at a time, lines are asked for in halves: 5% slower).
  // Piece c of row r is at place c ^ turn(r), so that the 16 rows that a
  // ds_read_b128 takes in a cycle are in different banks.
  auto load_keys = [&](const Rows &w) {
#pragma unroll
    for (int i = 0; i < BLK * CP / 4; ++i) {
      const int row = (i * 64 + lane) / CP, blk = i / (CP / 4);  // of the tile
      const uint32_t c = (lane % CP) ^ key_turn<CP>(row % 16);
      const uint32_t at = (FULL && DC == DP) || 16 * c < (uint32_t)(D * ES) ? 16 * c : 0u;
      const char *keys = static_cast<const char *>(a.cache.K);
      if constexpr (B16)
        load_lds16(make_rsrc(keys + (uint64_t)w.base[blk] * (D * ES)), (row % 16) * (D * ES) + at, kt + i * 1024);
      else
        load_lds16(keys + (uint64_t)(uint32_t)__shfl((int)w.own, row, 64) * (D * ES) + at, kt + i * 1024);
    }
    if constexpr (S8) ks = a.cache.scaleK[w.own];
  };
  auto key = [&](int blk, int j) {
    return *reinterpret_cast<const u32x4 *>(kt + (16 * blk + n) * (CP * 16) + 16 * ((4 * j + g) ^ key_turn<CP>(n)));
  };
  auto load_values = [&](const Rows &w) {
    const char *values = static_cast<const char *>(a.cache.V);
    uint32_t col[HALVES];
#pragma unroll
    for (int hf = 0; hf < HALVES; ++hf) {
      const uint32_t d = hf * 16 * CPL + n * CPL;
      col[hf] = FULL || d < (uint32_t)D ? d * ES : 0u;
    }
#pragma unroll
    for (int blk = 0; blk < BLK; ++blk) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const char *row;
        if constexpr (B16)
          row = values + (uint64_t)w.base[blk] * (D * ES) + (uint32_t)(4 * g * (D * ES)) + k * (D * ES);
        else
          row = values + (uint64_t)(uint32_t)__shfl((int)w.own, 16 * blk + 4 * g + k, 64) * (D * ES);
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf) {
          if constexpr (VW == 3) {  // (a vector of three is loaded as four, which would pass the cache's end)
            const u32x2 two = __builtin_nontemporal_load(reinterpret_cast<const u32x2_words *>(row + col[hf]));
            const uint32_t one = __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(row + col[hf]) + 2);
            vf[blk][k][hf] = piece{two[0], two[1], one};
          } else {
            vf[blk][k][hf] = __builtin_nontemporal_load(reinterpret_cast<const piece *>(row + col[hf]));
          }
        }
      }
    }
    if constexpr (S8) vs = a.cache.scaleV[w.own];
  };

  // The query's values as they are in memory, then its operand: 16 values of
  // piece j for codes, 16 bytes else.
  typedef uint32_t raw __attribute__((ext_vector_type(S8 ? 4 * sizeof(T) : 4)));
  typedef raw raw_anywhere __attribute__((aligned(2)));
  raw qr[KF];
  auto load_query = [&](const Segment &sg) {
    const T *q = static_cast<const T *>(a.Q) + (long long)sg.b * a.ldq + (sg.q0 + (n < sg.G ? n : 0)) * D;
#pragma unroll
    for (int j = 0; j < KF; ++j) {
      const int d = j * (64 / ES) + g * (16 / ES);
      qr[j] = *reinterpret_cast<const raw_anywhere *>(q + (d < D ? d : 0));
      if (n >= sg.G || d >= D) qr[j] = raw{};
    }
  };
  u32x4 qf[QDIG * KF];
  float qscale;
  auto turn_query = [&]() {
    qscale = a.scale2;
    if constexpr (S8) {
      typedef T sixteen __attribute__((ext_vector_type(16)));
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < KF; ++j) {
        const sixteen x = __builtin_bit_cast(sixteen, qr[j]);
#pragma unroll
        for (int e = 0; e < 16; ++e) top = nan_max(top, __builtin_fabsf((float)x[e]));
      }
      top = nanmax_groups(top);
      // rows below 2^-64 are taken times 2^80, which keeps 1 / top finite
      const float lift = top < 0x1p-64f ? 0x1p80f : 1.0f;
      const float inv = top > 0.0f ? kTop / (top * lift) : 0.0f;
      qscale *= top < __builtin_inff() ? top * (1.0f / kTop) : __builtin_nanf("");  // shows in every score
#pragma unroll
      for (int j = 0; j < KF; ++j) {
        const sixteen x = __builtin_bit_cast(sixteen, qr[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f[4] = {(float)x[4 * e] * lift, (float)x[4 * e + 1] * lift, (float)x[4 * e + 2] * lift,
                              (float)x[4 * e + 3] * lift};
          uint32_t w[QDIG];
          digits4(f, inv, w);
#pragma unroll
          for (int k = 0; k < QDIG; ++k) qf[k * KF + j][e] = w[k];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < KF; ++j) qf[j] = qr[j];
    }
  };

  // A tile's keys are asked for when the one before has given its scores, its
  // values when the one before is added up: one tile's bytes are always on the
  // way while a wave computes, in the place that it has just read.  (Without
  // B16 the next tile's table entries are asked for behind V and needed for its
  // keys, so V has landed by then: 64 ragged to 8192 on codes, pages of 24 instead
  // of 64, 83.4 -> 92.9 us.)  A head's
  // query and first tile are asked for before the head in front of it is joined;
  // so far the compiler also waits for them there (the query is masked behind
  // the branch around the tile's loads, and the join's first barrier waits for
  // what goes into LDS), so a change of head costs a trip to memory.
  Rows at;
  int t0, tend;
  auto begin = [&](const Segment &sg, auto first) {
    t0 = sg.sp.base + sg.i0 * UNIT + wave * TOK;
    tend = min(sg.sp.n, sg.sp.base + sg.i1 * UNIT);
    load_query(sg);
    if (t0 < tend) {
      at = locate(sg, t0);
      keep_order();
      load_keys(at);
      keep_order();
      load_values(at);
      keep_order();
      if constexpr (decltype(first)::value) turn_query();  // while they are on the way
    }
  };
  begin(sg, Flag<true>{});
  for (;;) {

    // ---- the tokens ------------------------------------------------------------
    float m = kNegInf, l = 0.0f;
    floatx4 o[HALVES * CPL];  // [column c of a lane's piece][i]: column (4 g + i) CPL + c
#pragma unroll
    for (int c = 0; c < HALVES * CPL; ++c) o[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    auto tile = [&](auto goes_on) {
      constexpr bool more = decltype(goes_on)::value;
      // which tokens are seen, by their place in the tile
      unsigned long long seen = at.seen;
      if (t0 < sg.sp.lo) seen &= ~0ull << (sg.sp.lo - t0);  // fewer than 64 before the window: base is that near
      if (t0 + 63 >= sg.sp.n) seen &= ~0ull >> (63 - (sg.sp.n - 1 - t0));
      const bool whole = seen == ~0ull >> (64 - TOK);
      if constexpr (more) at = locate(sg, t0 + UNIT);

      // K's tile has landed when no more than V's loads, which were asked for
      // behind it (keep_order), are on the way.  (The compiler does not see what the loads
      // into LDS write, so it need not wait for them by itself.)
      wait_loads<BLK * 4 * HALVES * ((VW + 3) / 4)>();

      // scores, in powers of two
      float s[BLK][4];
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk) {
        if constexpr (S8) {
          u32x4 kf[KF];
#pragma unroll
          for (int j = 0; j < KF; ++j) kf[j] = key(blk, j);
          const floatx4 v = digit_product<KF>(kf, qf);
#pragma unroll
          for (int k = 0; k < 4; ++k) s[blk][k] = v[k] * (__shfl(ks, 16 * blk + 4 * g + k, 64) * qscale);
        } else {
          floatx4 acc = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < KF; ++j) {
            u32x4 x = key(blk, j);
            if (!FULL && j * 64 + g * 16 >= D * ES) x = u32x4{0, 0, 0, 0};
            if constexpr (ES == 2) {
              acc = mfma16<T>(x, qf[j], acc);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__builtin_bit_cast(float, (uint32_t)x[e]),
                                                           __builtin_bit_cast(float, (uint32_t)qf[j][e]), acc, 0, 0, 0);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) s[blk][k] = acc[k] * qscale;
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // K's tile has been read
      keep_order();
      if constexpr (more) load_keys(at);
      keep_order();
      if (!whole) {
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const bool in = (uint32_t)(seen >> 16 * blk) >> (4 * g + k) & 1;
            s[blk][k] = in ? s[blk][k] : kNegInf;
            if constexpr (!S8) {
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf)
                if (!in) vf[blk][k][hf] = piece{};
            }
          }
      }

      // running maximum and sum; a NaN does not become the maximum, it shows in the sum
      float top = kNegInf;
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
        for (int k = 0; k < 4; ++k) top = __builtin_fmaxf(top, s[blk][k]);
      top = __builtin_fmaxf(m, fmax_groups(top));
      if (__any(top > m)) {
        const float shrink = top > m ? __builtin_amdgcn_exp2f(m - top) : 1.0f;
        l *= shrink;
#pragma unroll
        for (int c = 0; c < HALVES * CPL; ++c) o[c] *= shrink;
        m = top;
      }
      constexpr float lift = __is_same(T, _Float16) && !S8 ? (float)kScoreBias16 : 0.0f;
      const float from = m == kNegInf ? 0.0f : m - lift;
      float p[BLK][4];
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          p[blk][k] = __builtin_amdgcn_exp2f(s[blk][k] - from);
          l += p[blk][k];
        }

      // ---- weights times V -------------------------------------------------------
      if constexpr (S8) {
        float big = 0.0f;
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            p[blk][k] *= __shfl(vs, 16 * blk + 4 * g + k, 64);
            if (!whole && !((uint32_t)(seen >> 16 * blk) >> (4 * g + k) & 1)) p[blk][k] = 0.0f;
            big = nan_max(big, __builtin_fabsf(p[blk][k]));
          }
        big = nanmax_groups(big);
        // below 2^-100 the digits end at 2^-123; NaN and infinity go on into the outputs
        big = big < 0x1p-100f ? 0x1p-100f : big;
        const float inv = kTop / big, factor = big * (1.0f / kTop);
        u32x4 pd[kDigits];
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
          uint32_t w[kDigits];
          digits4(p[blk], inv, w);
#pragma unroll
          for (int k = 0; k < kDigits; ++k) pd[k][blk] = w[k];
        }
#pragma unroll
        for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
          for (int x = 0; x < CPL / 4; ++x) {
            u32x4 col[4];
#pragma unroll
            for (int blk = 0; blk < BLK; ++blk) {
              const uint32_t a0 = vf[blk][0][hf][x], a1 = vf[blk][1][hf][x], a2 = vf[blk][2][hf][x],
                             a3 = vf[blk][3][hf][x];
              const uint32_t t0_ = __builtin_amdgcn_perm(a1, a0, 0x05010400u);
              const uint32_t t1_ = __builtin_amdgcn_perm(a1, a0, 0x07030602u);
              const uint32_t u0_ = __builtin_amdgcn_perm(a3, a2, 0x05010400u);
              const uint32_t u1_ = __builtin_amdgcn_perm(a3, a2, 0x07030602u);
              col[0][blk] = __builtin_amdgcn_perm(u0_, t0_, 0x05040100u);
              col[1][blk] = __builtin_amdgcn_perm(u0_, t0_, 0x07060302u);
              col[2][blk] = __builtin_amdgcn_perm(u1_, t1_, 0x05040100u);
              col[3][blk] = __builtin_amdgcn_perm(u1_, t1_, 0x07060302u);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const u32x4 one[1] = {col[c]};
              const floatx4 v = digit_product<1>(one, pd);
              floatx4 &out = o[hf * CPL + 4 * x + c];
#pragma unroll
              for (int k = 0; k < 4; ++k) out[k] = __builtin_fmaf(factor, v[k], out[k]);
            }
            __builtin_amdgcn_sched_barrier(0);  // else all columns' sums are in registers at once
          }
      } else {
        if constexpr (ES == 2) {
          u32x4 ph, pl;
#pragma unroll
          for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              typedef T two __attribute__((ext_vector_type(2)));
              const two hi = {(T)p[blk][k], (T)p[blk][k + 1]};
              const two lo = {(T)(p[blk][k] - (float)hi[0]), (T)(p[blk][k + 1] - (float)hi[1])};
              ph[2 * blk + k / 2] = __builtin_bit_cast(uint32_t, hi);
              pl[2 * blk + k / 2] = __builtin_bit_cast(uint32_t, lo);
            }
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
              u32x4 col;
              const uint32_t pick = c & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
              for (int blk = 0; blk < BLK; ++blk) {
                col[2 * blk] = __builtin_amdgcn_perm(vf[blk][1][hf][c / 2], vf[blk][0][hf][c / 2], pick);
                col[2 * blk + 1] = __builtin_amdgcn_perm(vf[blk][3][hf][c / 2], vf[blk][2][hf][c / 2], pick);
              }
              o[hf * CPL + c] = mfma16<T>(col, ph, o[hf * CPL + c]);
              o[hf * CPL + c] = mfma16<T>(col, pl, o[hf * CPL + c]);
            }
        } else {
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
            for (int c = 0; c < CPL; ++c)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[hf * CPL + c] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                    __builtin_bit_cast(float, (uint32_t)vf[0][k][hf][c]), p[0][k], o[hf * CPL + c], 0, 0, 0);
        }
      }
      keep_order();
      if constexpr (more) load_values(at);
      keep_order();
    };
    // The last tile asks for no other one.  It has code of its own: with a
    // branch around each of the two loads the compiler would wait for all of
    // them where K's tile is needed.
    if (t0 < tend) {
      for (; t0 + UNIT < tend; t0 += UNIT) tile(Flag<true>{});
      tile(Flag<false>{});
    }

    // ---- the four waves' results, joined ----------------------------------------
    const Segment done = sg;
    const int u = sg.start + over + sg.i1;
    bool more = u < u1 && !whole_runs;
    if (more) {
      sg = segment(u, sg.b, sg.prefix, sg.sp);
      more = sg.i0 < sg.i1;
      if (more) begin(sg, Flag<false>{});
    }
    const int G = done.G;
    l = sum_groups(l);
    __syncthreads();  // merge, wm and wl are free again
    if (g == 0) wm[wave][n] = m, wl[wave][n] = l;
    if (n < G) {
#pragma unroll
      for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int c = 0; c < CPL; c += 4) {
            const int d = hf * 16 * CPL + (4 * g + k) * CPL + c;
            const int x = hf * CPL + c;
            *reinterpret_cast<floatx4 *>(&merge[wave][n * PITCH + d]) =
                floatx4{o[x][k], o[x + 1][k], o[x + 2][k], o[x + 3][k]};
          }
    }
    __syncthreads();
    const bool alone = done.i0 == 0 && done.i1 == done.sp.units;
    const int row_start = done.start, token_start = row_start + over;
    // the head's workgroups, and where their parts of it are: a workgroup's
    // first head is in its first place, its last one, if another, in its second
    const int wa = token_start / per, ns = (token_start + done.sp.units - 1) / per - wa + 1;
    const uint32_t record = (uint32_t)attend_record(min(16, a.G), D) * 4;
    const __amdgpu_buffer_rsrc_t parts = __builtin_amdgcn_make_buffer_rsrc(
        a.part, (short)0, (int)(2 * kAttendGroups * record), kRsrcWord3);
    const int vecs = G * D / 4;  // a part: outputs, maxima, sums
    auto put = [&](int e, floatx4 v) {
      const int row = 4 * e / D, d = 4 * e - row * D;
      typedef T four __attribute__((ext_vector_type(4), aligned(alignof(T))));
      typedef T plain __attribute__((ext_vector_type(4)));
      *reinterpret_cast<four *>(static_cast<T *>(a.O) + (long long)done.b * a.ldo + (done.q0 + row) * D + d) =
          plain{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    };
    constexpr float bias = __is_same(T, _Float16) && !S8 ? (float)kScoreBias16 : 0.0f;
    auto put_lse = [&](int row, float mm, float ll) {
      if (a.lse != nullptr)
        a.lse[(long long)done.b * a.Hq + done.q0 + row] =
            ll == 0.0f ? kNegInf : (mm - bias + __builtin_amdgcn_logf(ll)) * 0.69314718056f;
    };
    const uint32_t mine_at = (uint32_t)(2 * blockIdx.x + (row_start == first_row ? 0 : 1)) * record;
    for (int e = tid; e < vecs; e += 256) {
      const int row = 4 * e / D, d = 4 * e - row * D;
      float mm = kNegInf, ll = 0.0f;
      floatx4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = __builtin_fmaxf(mm, wm[w][row]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = weight_of(wm[w][row], wl[w][row], mm);
        const floatx4 v = *reinterpret_cast<const floatx4 *>(&merge[w][row * PITCH + d]);
        ll = __builtin_fmaf(f, wl[w][row], ll);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] = __builtin_fmaf(f, v[k], sum[k]);
      }
      if (alone) {
        put(e, ll == 0.0f ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : sum / ll);
        if (d == 0) put_lse(row, mm, ll);
      } else {
        store_through(sum, parts, mine_at + 16 * e);
        if (d == 0) {
          store_through(mm, parts, mine_at + 16 * vecs + 4 * row);
          store_through(ll, parts, mine_at + 16 * vecs + 4 * (G + row));
        }
      }
    }
    if (!alone) {
      // Joins `count` parts, `step` bytes apart from `from` (the first `extra`
      // behind that), P of them at most: all outputs are on the way while the
      // parts' weights are found (thread: part tid / 16, head tid % 16; a
      // wave's four parts by lane exchange, the waves' in LDS).  Parts behind
      // the last read as zero, past the end of the buffer.  The result goes out,
      // or into the first part's place; where registers are short, in rounds of
      // the outputs from e0, the maxima with the one that `ends`.
      auto join = [&](auto most_parts, auto most_vecs, int e0, uint32_t from, uint32_t step, uint32_t extra,
                      int count, bool out, bool ends) {
        constexpr int P = decltype(most_parts)::value, OWN = decltype(most_vecs)::value;
        const int row = tid & 15, sub = tid >> 4;
        const bool in = row < G && sub < count;
        const uint32_t p = from + sub * step + (sub == 0 ? extra : 0) + 16 * vecs + 4 * row;
        float pm = load_through(parts, in ? p : kOob);
        const float pl = load_through(parts, in ? p + 4 * G : kOob);
        floatx4 v[OWN][P];
#pragma unroll
        for (int x = 0; x < OWN; ++x)
#pragma unroll
          for (int w = 0; w < P; ++w)
            v[x][w] = load_through4(parts, e0 + 256 * x < vecs && w < count
                                               ? from + w * step + (w == 0 ? extra : 0) + 16 * (e0 + 256 * x)
                                               : kOob);
        pm = in ? pm : kNegInf;
        const float wave_m = fmax_groups(pm);
        if (g == 0) wm[wave][row] = wave_m;
        __syncthreads();
        float mm = wm[0][row];
#pragma unroll
        for (int w = 1; w < 4; ++w) mm = __builtin_fmaxf(mm, wm[w][row]);
        const float f = weight_of(pm, pl, mm), wave_l = sum_groups(f * pl);
        part_f[sub][row] = f;
        if (g == 0) wl[wave][row] = wave_l;
        __syncthreads();
        auto total = [&](int row) { return (wl[0][row] + wl[1][row]) + (wl[2][row] + wl[3][row]); };
#pragma unroll
        for (int x = 0; x < OWN; ++x) {
          const int e = e0 + 256 * x, rr = min(4 * e / D, 15);
          floatx4 acc = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int w = 0; w < P; ++w)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[k] = __builtin_fmaf(part_f[w][rr], v[x][w][k], acc[k]);
          if (e >= vecs) continue;
          const float sum = total(rr);
          if (!out)
            store_through(acc, parts, from + extra + 16 * e);
          else
            put(e, sum == 0.0f ? floatx4{0.0f, 0.0f, 0.0f, 0.0f} : acc / sum);
        }
        if (sub == 0 && row < G && ends) {  // (nobody reads the maxima any more)
          if (!out) {
            store_through(mm, parts, p);
            store_through(total(row), parts, p + 4 * G);
          } else {
            put_lse(row, mm, total(row));
          }
        }
      };
      // One CU reads parts at some 28 KB a us, 2 to 3 us at a time with the counter:
      // as many at once as its registers take on the way, and for more parts two
      // or three steps of as equal sizes as that allows.  Against the last to
      // arrive reading all: 128 parts of 16 KB (32768 tokens, 16 heads x 256
      // fp16) 76 -> 23 us, 128 of 8 KB 28.6 -> 16.9, 64 of 264 bytes 17.1 -> 11.8,
      // 17 of 16 KB (16 windows of 4096) 24.7 -> 22.2; 16 parts of 2 KB as before.
      const bool small = DC <= 64 || vecs <= 256;
      const int most = small ? 16 : 8;
      int F = ns;
      if (ns > most) {
        F = 2;
        while (F * F < ns) ++F;
        if (F > most) {
          F = 2;
          while (F * F * F < ns) ++F;
        }
      }
      const uint32_t extra = wa * per >= row_start ? 0 : record;  // of part 0
      // part `mine` of the head, of parts `apart` workgroups from each other
      int mine = (int)blockIdx.x - wa, apart = 1, field = 0;
      for (;;) {
        const int first = mine / (F * apart) * (F * apart), all = (ns + apart - 1) / apart;
        const int count = min(F, all - first / apart);
        if (count > 1) {
          asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
          __syncthreads();
          if (tid == 0)
            last = (__hip_atomic_fetch_add(&a.cnt[wa + first], 1u << field, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) >>
                        field & 31) == (unsigned)(count - 1);
          __syncthreads();
          if (!__builtin_amdgcn_readfirstlane(last)) break;
          asm volatile("" ::: "memory");
          const uint32_t from = (uint32_t)(2 * (wa + first)) * record, step = (uint32_t)(2 * apart) * record;
          const uint32_t late = first == 0 ? extra : 0;
          // (fp32: more outputs at once are in the way of the next head's first tile)
          constexpr int OWN = ES == 4 ? DP / 128 : DC / 64;
          if (small)
            join(Number<16>(), Number<1>(), tid, from, step, late, count, all <= F, true);
          else if constexpr (256 * OWN >= 4 * DC)
            join(Number<8>(), Number<OWN>(), tid, from, step, late, count, all <= F, true);
          else if constexpr (OWN > 0)
            for (int x = 0; x < vecs; x += 256 * OWN)
              join(Number<8>(), Number<OWN>(), tid + x, from, step, late, count, all <= F, x + 256 * OWN >= vecs);
          if (tid == 0)
            __hip_atomic_fetch_sub(&a.cnt[wa + first], (unsigned)count << field, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
        if (all <= F) break;
        mine = first, apart *= F, field += 5;
      }
    }
    if (!more) break;
    turn_query();
  }
}

template <class T, bool S8, int DP, int DC = DP> hipError_t launch_attend_dim(const AttendArgs &all, hipStream_t s) {
  AttendArgs a = all;
  // two workgroups a CU, one where heads past 128 values take the registers of both
  if (DP > 128 && a.groups > 256) a.groups = 256;
  const bool blocks = a.cache.page_size % 16 == 0;
  if (a.cache.dim == DC) {
    if (blocks) attend_kernel<T, S8, DP, DC, true, true><<<a.groups, 256, 0, s>>>(a);
    else attend_kernel<T, S8, DP, DC, false, true><<<a.groups, 256, 0, s>>>(a);
  } else if constexpr (DC == DP) {
    if (blocks) attend_kernel<T, S8, DP, DP, true, false><<<a.groups, 256, 0, s>>>(a);
    else attend_kernel<T, S8, DP, DP, false, false><<<a.groups, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}
template <class T, bool S8> hipError_t launch_attend(const AttendArgs &a, hipStream_t s) {
  if (a.cache.dim <= 64) return launch_attend_dim<T, S8, 64>(a, s);
  if (a.cache.dim <= 128) return launch_attend_dim<T, S8, 128>(a, s);
  if (a.cache.dim == 192) return launch_attend_dim<T, S8, 256, 192>(a, s);
  return launch_attend_dim<T, S8, 256>(a, s);
}

}  // namespace
}  // namespace fp32gemm
