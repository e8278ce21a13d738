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
// share is joined by the last of them to arrive, in the order of its tokens
// (partial results and arrival counter as in gemv_split.hip: agent-scope
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
//    own largest, in signed 8-bit digits: three (23 bits) for fp32 operands,
//    two (15 bits) for 16-bit ones.  Two leave an error of 2^-16 of a row's
//    largest q in each product, 3e-5 of a score of unit spread, and 2^-16 of
//    a tile's largest weight: below a hundredth of the output's rounding.  No
//    code of the cache is converted.
//  16-bit floats: products of the type, sums in fp32.  A weight goes in as two
//    numbers of the type (its rounding and what that left), 16 bits or more.
//  fp32: fp32 matrix instructions.
//
// Masked tokens get a score of minus infinity and weight 0 by selection; where
// V is floats their values are selected away too, so whatever unwritten pages
// hold does no harm.
#pragma once

#include "kv_common.h"

namespace fp32gemm {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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

// Signed 8-bit digits of numbers in [-1, 1] times inv: the integer plus
// 0x80 in every digit, whose bytes, 0x80 taken off again, are the digits.
template <int DIG> struct Fixed {
  static constexpr float top = DIG == 3 ? 8355000.0f : 32600.0f;
  static constexpr float bias = DIG == 3 ? 8421504.0f : 32896.5f;  // above 2^23 the addition itself rounds
};
template <int DIG> __device__ __forceinline__ void digits4(const float (&v)[4], float inv, uint32_t (&w)[DIG]) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = (uint32_t)__builtin_fmaf(v[e], inv, Fixed<DIG>::bias);
  const uint32_t t = __builtin_amdgcn_perm(u[1], u[0], 0x05010400u);
  const uint32_t s = __builtin_amdgcn_perm(u[3], u[2], 0x05010400u);
  w[0] = __builtin_amdgcn_perm(s, t, 0x05040100u) ^ 0x80808080u;
  w[1] = __builtin_amdgcn_perm(s, t, 0x07060302u) ^ 0x80808080u;
  if constexpr (DIG == 3) {
    const uint32_t t2 = __builtin_amdgcn_perm(u[1], u[0], 0x0c0c0602u);
    const uint32_t s2 = __builtin_amdgcn_perm(u[3], u[2], 0x0c0c0602u);
    w[2] = __builtin_amdgcn_perm(s2, t2, 0x05040100u) ^ 0x80808080u;
  }
}

// What a product's digits add up to.
template <int DIG> __device__ __forceinline__ float digit_sum(const intx4 (&acc)[DIG], int r) {
  if constexpr (DIG == 3)
    return __builtin_fmaf(256.0f, (float)((acc[2][r] << 8) + acc[1][r]), (float)acc[0][r]);
  else
    return (float)((acc[1][r] << 8) + acc[0][r]);  // below 2^31: 256 products of 127 and 128, or 64
}

template <class T, bool S8> struct Kind;
template <class T> struct Kind<T, true> {
  static constexpr int ES = 1, TOK = 64, DIG = sizeof(T) == 4 ? 3 : 2;
};
template <> struct Kind<float, false> { static constexpr int ES = 4, TOK = 16, DIG = 1; };
template <class T> struct Kind<T, false> { static constexpr int ES = 2, TOK = 32, DIG = 2; };

template <class T> __device__ __forceinline__ floatx4 mfma16(u32x4 a, u32x4 b, floatx4 c) {
  typedef T frag __attribute__((ext_vector_type(8)));
  if constexpr (__is_same(T, _Float16))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(frag, a), __builtin_bit_cast(frag, b), c, 0, 0, 0);
}

// A sequence's units and where its tokens start: lo .. n are seen.
template <int UNIT> struct Span {
  int lo, n, base, units;
  __device__ __forceinline__ Span(const AttendArgs &a, int b) {
    const int most = a.ldt * a.cache.page_size;  // fits: checked by the caller
    n = a.lengths[b];
    n = n < 0 ? 0 : n > most ? most : n;
    lo = a.window > 0 && n > a.window ? n - a.window : 0;
    base = lo & ~63;
    units = (n - base + UNIT - 1) / UNIT;
    units = units < 1 ? 1 : units;  // an empty sequence's outputs are written too
  }
};

// B16: a page holds whole blocks of 16 tokens, so a block's address is the
// wave's; else every token has its own.
template <class T, bool S8, int DP, bool B16>
__global__ void __launch_bounds__(256, DP > 128 ? 1 : 2) attend_kernel(AttendArgs a) {
  typedef Kind<T, S8> KD;
  constexpr int ES = KD::ES, TOK = KD::TOK, DIG = KD::DIG, UNIT = 4 * TOK, BLK = TOK / 16;
  constexpr int CPL = DP >= 128 ? 8 : 4;       // columns of V of a lane, next to each other
  constexpr int HALVES = DP / (16 * CPL);      // of which there are 16 lanes
  constexpr int KF = DP * ES / 64;             // 16-byte pieces of a token's K in a lane
  constexpr int VW = CPL * ES / 4;             // words of a token's V piece
  constexpr int NP = HALVES * CPL * 16 * 16;   // outputs of a wave: 16 heads x DP
  static_assert(NP == 16 * DP, "");

  __shared__ __attribute__((aligned(16))) float merge[4 * NP > kAttendGroups * 16 ? 4 * NP : kAttendGroups * 16];
  __shared__ float wm[4][16], wl[4][16], red[2][16][16];
  __shared__ long long scan[4];
  __shared__ long long at_prefix;
  __shared__ int at_seq, last;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int rows = a.Hk * a.RG, D = a.cache.dim, ps = a.cache.page_size;

  // ---- this workgroup's run of units -----------------------------------------
  const int each = (a.B + 255) / 256;
  long long mine = 0;
  for (int j = 0; j < each; ++j) {
    const int b = tid * each + j;
    if (b < a.B) mine += (long long)Span<UNIT>(a, b).units * rows;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const long long t = __shfl_up(incl, d, 64);
    if (lane >= d) incl += t;
  }
  if (lane == 63) scan[wave] = incl;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    before += w < wave ? scan[w] : 0;
    total += scan[w];
  }
  // (the caller has checked that the units are fewer than 2^31)
  const int U = (int)total, per = (U + a.groups - 1) / a.groups;
  const int u0 = (int)blockIdx.x * per;
  if (u0 >= U) return;
  const int u1 = min(U, u0 + per);
  incl += before;
  if (incl - mine <= u0 && u0 < incl) {
    long long p = incl - mine;
    int b = tid * each;
    for (;; ++b) {
      const long long t = (long long)Span<UNIT>(a, b).units * rows;
      if (u0 < p + t) break;
      p += t;
    }
    at_prefix = p;
    at_seq = b;
  }
  __syncthreads();
  int b = __builtin_amdgcn_readfirstlane(at_seq);
  int prefix = __builtin_amdgcn_readfirstlane((int)at_prefix);
  Span<UNIT> sp(a, b);
  const int first_row = prefix + (u0 - prefix) / sp.units * sp.units;  // unit where the first head starts

  for (int u = u0; u < u1;) {
    if (u >= prefix + sp.units * rows) {
      prefix += sp.units * rows;
      sp = Span<UNIT>(a, ++b);
      continue;
    }
    const int r = (u - prefix) / sp.units, i0 = u - prefix - r * sp.units;
    const int i1 = min(sp.units, i0 + u1 - u);
    const int head = r / a.RG, h0 = (r - head * a.RG) * 16;
    const int G = min(16, a.G - h0);  // query heads here
    const int q0 = head * a.G + h0;   // the first of them

    // ---- the query's operand -------------------------------------------------
    const T *q = static_cast<const T *>(a.Q) + (long long)b * a.ldq + (q0 + (n < G ? n : 0)) * D;
    u32x4 qf[S8 ? DIG * KF : KF];
    float qscale = a.scale2;
    if constexpr (S8) {
      typedef T eight __attribute__((ext_vector_type(8), aligned(alignof(T))));
      float v[KF][16];
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < KF; ++j) {
        const int d = j * 64 + g * 16;
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          eight x = *reinterpret_cast<const eight *>(q + (d < D ? d + e : 0));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            v[j][e + k] = n < G && d < D ? (float)x[k] : 0.0f;
            top = nan_max(top, __builtin_fabsf(v[j][e + k]));
          }
        }
      }
      top = nanmax_groups(top);
      // rows below 2^-64 are taken times 2^80, which keeps 1 / top finite
      const float lift = top < 0x1p-64f ? 0x1p80f : 1.0f;
      const float inv = top > 0.0f ? Fixed<DIG>::top / (top * lift) : 0.0f;
      qscale *= top < __builtin_inff() ? top * (1.0f / Fixed<DIG>::top) : __builtin_nanf("");  // shows in every score
#pragma unroll
      for (int j = 0; j < KF; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f[4] = {v[j][4 * e] * lift, v[j][4 * e + 1] * lift, v[j][4 * e + 2] * lift,
                              v[j][4 * e + 3] * lift};
          uint32_t w[DIG];
          digits4<DIG>(f, inv, w);
#pragma unroll
          for (int k = 0; k < DIG; ++k) qf[k * KF + j][e] = w[k];
        }
    } else {
      typedef u32x4 anywhere __attribute__((aligned(2)));
#pragma unroll
      for (int j = 0; j < KF; ++j) {
        const int d = j * (64 / ES) + g * (16 / ES);
        const u32x4 x = *reinterpret_cast<const anywhere *>(q + (d < D ? d : 0));
        qf[j] = n < G && d < D ? x : u32x4{0, 0, 0, 0};
      }
    }

    // ---- the tokens ------------------------------------------------------------
    float m = kNegInf, l = 0.0f;
    floatx4 o[HALVES * CPL];  // [column c of a lane's piece][i]: column (4 g + i) CPL + c
#pragma unroll
    for (int c = 0; c < HALVES * CPL; ++c) o[c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};

    for (int i = i0; i < i1; ++i) {
      const int t0 = sp.base + i * UNIT + wave * TOK;
      if (t0 >= sp.n) break;
      // rows of the cache: of K's token 16 blk + n, of V's tokens 16 blk + 4 g + i
      uint32_t krow[BLK], vrow[BLK][4];
      uint32_t seen = 0;  // by blk: whether the block's (B16) or the token's page exists; bits 4 blk + i
      if constexpr (B16) {
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
          const uint32_t t = t0 + 16 * blk;
          const int pi = (int)((uint64_t)t * a.magic >> a.shift);
          const int page = pi < a.ldt ? a.table[(long long)b * a.ldt + pi] : -1;
          const bool ok = page >= 0 && page < a.cache.pages;
          const uint32_t base = ((ok ? page : 0) * a.cache.heads + head) * ps + (t - pi * ps);
          seen |= ok ? 0xfu << 4 * blk : 0u;
          krow[blk] = base + n;
#pragma unroll
          for (int k = 0; k < 4; ++k) vrow[blk][k] = base + 4 * g + k;
        }
      } else {
        // lane t < TOK looks its token's row up, the others ask it
        const uint32_t t = t0 + lane % TOK;
        const int pi = (int)((uint64_t)t * a.magic >> a.shift);
        const int page = pi < a.ldt ? a.table[(long long)b * a.ldt + pi] : -1;
        const bool ok = page >= 0 && page < a.cache.pages;
        const uint32_t row = ((ok ? page : 0) * a.cache.heads + head) * ps + (t - pi * ps);
        const unsigned long long oks = __ballot(ok);
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
          krow[blk] = (uint32_t)__shfl((int)row, 16 * blk + n, 64);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            vrow[blk][k] = (uint32_t)__shfl((int)row, 16 * blk + 4 * g + k, 64);
            seen |= (uint32_t)(oks >> (16 * blk + 4 * g + k) & 1) << (4 * blk + k);
          }
        }
      }
      const uint32_t every = BLK == 8 ? ~0u : (1u << 4 * BLK) - 1;
      const bool whole = t0 >= sp.lo && t0 + TOK <= sp.n && __all(seen == every);
      if (!whole) {
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int t = t0 + 16 * blk + 4 * g + k;
            if (t < sp.lo || t >= sp.n) seen &= ~(1u << (4 * blk + k));
          }
      }

      u32x4 kf[BLK][KF];
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
        for (int j = 0; j < KF; ++j) {
          const int d = j * 64 + g * 16;  // bytes
          const char *p = static_cast<const char *>(a.cache.K) + (uint64_t)krow[blk] * (D * ES);
          kf[blk][j] = *reinterpret_cast<const u32x4 *>(p + (d < D * ES ? d : 0));
        }
      typedef uint32_t piece __attribute__((ext_vector_type(VW)));
      piece vf[BLK][4][HALVES];
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int hf = 0; hf < HALVES; ++hf) {
            const int d = hf * 16 * CPL + n * CPL;
            const char *p = static_cast<const char *>(a.cache.V) + (uint64_t)vrow[blk][k] * (D * ES);
            vf[blk][k][hf] = *reinterpret_cast<const piece *>(p + (d < D ? d * ES : 0));
          }
      float ks[BLK][4], vs[BLK][4];
      if constexpr (S8) {
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
          if constexpr (B16) {
            typedef floatx4 anywhere __attribute__((aligned(4)));
            const floatx4 x = *reinterpret_cast<const anywhere *>(a.cache.scaleK + vrow[blk][0]);
            const floatx4 y = *reinterpret_cast<const anywhere *>(a.cache.scaleV + vrow[blk][0]);
#pragma unroll
            for (int k = 0; k < 4; ++k) ks[blk][k] = x[k], vs[blk][k] = y[k];
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) ks[blk][k] = a.cache.scaleK[vrow[blk][k]], vs[blk][k] = a.cache.scaleV[vrow[blk][k]];
          }
        }
      }

      // scores, in powers of two
      float s[BLK][4];
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk) {
        if constexpr (S8) {
          intx4 acc[DIG];
#pragma unroll
          for (int k = 0; k < DIG; ++k) {
            acc[k] = intx4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < KF; ++j)
              acc[k] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, kf[blk][j]),
                                                             __builtin_bit_cast(intx4, qf[k * KF + j]), acc[k], 0, 0, 0);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) s[blk][k] = digit_sum<DIG>(acc, k) * (ks[blk][k] * qscale);
        } else {
          floatx4 acc = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int j = 0; j < KF; ++j) {
            u32x4 x = kf[blk][j];
            if (D != DP && j * 64 + g * 16 >= D * ES) x = u32x4{0, 0, 0, 0};
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
      if (!whole) {
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!(seen >> (4 * blk + k) & 1)) s[blk][k] = kNegInf;
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
            p[blk][k] = seen >> (4 * blk + k) & 1 ? p[blk][k] * vs[blk][k] : 0.0f;
            big = nan_max(big, __builtin_fabsf(p[blk][k]));
          }
        big = nanmax_groups(big);
        // below 2^-100 the digits end at 2^-123; NaN and infinity go on into the outputs
        big = big < 0x1p-100f ? 0x1p-100f : big;
        const float inv = Fixed<DIG>::top / big, factor = big * (1.0f / Fixed<DIG>::top);
        u32x4 pd[DIG];
#pragma unroll
        for (int blk = 0; blk < BLK; ++blk) {
          uint32_t w[DIG];
          digits4<DIG>(p[blk], inv, w);
#pragma unroll
          for (int k = 0; k < DIG; ++k) pd[k][blk] = w[k];
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
              intx4 acc[DIG];
#pragma unroll
              for (int k = 0; k < DIG; ++k)
                acc[k] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(intx4, col[c]),
                                                               __builtin_bit_cast(intx4, pd[k]), intx4{0, 0, 0, 0}, 0, 0, 0);
              floatx4 &out = o[hf * CPL + 4 * x + c];
#pragma unroll
              for (int k = 0; k < 4; ++k) out[k] = __builtin_fmaf(factor, digit_sum<DIG>(acc, k), out[k]);
            }
          }
      } else {
        if (!whole) {
#pragma unroll
          for (int blk = 0; blk < BLK; ++blk)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int hf = 0; hf < HALVES; ++hf)
                if (!(seen >> (4 * blk + k) & 1)) vf[blk][k][hf] = piece{};
        }
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
    }

    // ---- the four waves' results, joined ----------------------------------------
    l = sum_groups(l);
    __syncthreads();  // merge, wm, wl and red are free again
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
            *reinterpret_cast<floatx4 *>(&merge[wave * NP + n * DP + d]) =
                floatx4{o[x][k], o[x + 1][k], o[x + 2][k], o[x + 3][k]};
          }
    }
    __syncthreads();
    const bool alone = i0 == 0 && i1 == sp.units;
    const int row_start = prefix + r * sp.units;
    const int wa = row_start / per, wb = (row_start + sp.units - 1) / per;  // workgroups of this head
    const size_t record = (size_t)min(16, a.G) * (D + 2);
    float *part = a.part + (size_t)(2 * blockIdx.x + (row_start == first_row ? 0 : 1)) * record;
    auto put = [&](int row, int d, float value) {
      static_cast<T *>(a.O)[(long long)b * a.ldo + (q0 + row) * D + d] = (T)value;
    };
    constexpr float bias = __is_same(T, _Float16) && !S8 ? (float)kScoreBias16 : 0.0f;
    auto put_lse = [&](int row, float mm, float ll) {
      if (a.lse != nullptr)
        a.lse[(long long)b * a.Hq + q0 + row] =
            ll == 0.0f ? kNegInf : (mm - bias + __builtin_amdgcn_logf(ll)) * 0.69314718056f;
    };
    for (int e = tid; e < G * D; e += 256) {
      const int row = e / D, d = e - row * D;
      float mm = kNegInf, ll = 0.0f, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) mm = __builtin_fmaxf(mm, wm[w][row]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = wm[w][row] == kNegInf && wl[w][row] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(wm[w][row] - (mm == kNegInf ? 0.0f : mm));
        ll = __builtin_fmaf(f, wl[w][row], ll);
        sum = __builtin_fmaf(f, merge[w * NP + row * DP + d], sum);
      }
      if (alone) {
        put(row, d, ll == 0.0f ? 0.0f : sum / ll);
        if (d == 0) put_lse(row, mm, ll);
      } else {
        __hip_atomic_store(part + row * D + d, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (d == 0) {
          __hip_atomic_store(part + G * D + row, mm, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          __hip_atomic_store(part + G * D + G + row, ll, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
      }
    }
    if (!alone) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (tid == 0)
        last = __hip_atomic_fetch_add(&a.cnt[wa], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (unsigned)(wb - wa);
      __syncthreads();
      if (last) {
        asm volatile("" ::: "memory");
        const int ns = wb - wa + 1;
        // workgroup wa has this head in its first place only if its run starts here
        auto src = [&](int w) {
          return a.part + (size_t)(2 * (wa + w) + (w == 0 && wa * per != row_start ? 1 : 0)) * record;
        };
        // weights of the parts, in LDS
        const int row = tid & 15, sub = tid >> 4;
        float mm = kNegInf;
        if (row < G)
          for (int w = sub; w < ns; w += 16)
            mm = __builtin_fmaxf(mm, __hip_atomic_load(src(w) + G * D + row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
        red[0][sub][row] = mm;
        __syncthreads();
        for (int w = 0; w < 16; ++w) mm = __builtin_fmaxf(mm, red[0][w][row]);
        float ll = 0.0f;
        if (row < G)
          for (int w = sub; w < ns; w += 16) {
            const float pm = __hip_atomic_load(src(w) + G * D + row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const float pl = __hip_atomic_load(src(w) + G * D + G + row, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const float f = pm == kNegInf && pl == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(pm - (mm == kNegInf ? 0.0f : mm));
            merge[w * 16 + row] = f;
            ll = __builtin_fmaf(f, pl, ll);
          }
        red[1][sub][row] = ll;
        __syncthreads();
        for (int e = tid; e < G * D; e += 256) {
          const int rr = e / D, d = e - rr * D;
          float sum = 0.0f, all = 0.0f;
          for (int w = 0; w < 16; ++w) all += red[1][w][rr];
          int w = 0;
          for (; w + 8 <= ns; w += 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[k] = __hip_atomic_load(src(w + k) + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = __builtin_fmaf(merge[(w + k) * 16 + rr], v[k], sum);
          }
          for (; w < ns; ++w)
            sum = __builtin_fmaf(merge[w * 16 + rr],
                                 __hip_atomic_load(src(w) + e, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), sum);
          put(rr, d, all == 0.0f ? 0.0f : sum / all);
          if (d == 0) {
            float top = kNegInf;
            for (int k = 0; k < 16; ++k) top = __builtin_fmaxf(top, red[0][k][rr]);
            put_lse(rr, top, all);
          }
        }
        if (tid == 0) __hip_atomic_store(&a.cnt[wa], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    u += i1 - i0;
  }
}

template <class T, bool S8, int DP> hipError_t launch_attend_dim(const AttendArgs &a, hipStream_t s) {
  if (a.cache.page_size % 16 == 0)
    attend_kernel<T, S8, DP, true><<<a.groups, 256, 0, s>>>(a);
  else
    attend_kernel<T, S8, DP, false><<<a.groups, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <class T, bool S8> hipError_t launch_attend(const AttendArgs &a, hipStream_t s) {
  if (a.cache.dim <= 64) return launch_attend_dim<T, S8, 64>(a, s);
  if (a.cache.dim <= 128) return launch_attend_dim<T, S8, 128>(a, s);
  return launch_attend_dim<T, S8, 256>(a, s);
}

}  // namespace
}  // namespace fp32gemm
