// Heads of queries, keys and values, row by row: the root-mean-square norm and
// the position rotation (qk_norm_rope), the same with keys and values going
// into the paged cache (qkv_rope_write), the cache alone (kv_write), and the
// cache's rows as floats (kv_read).
//
// A row is one token's D values of one head.
//   norm:      n_d = x_d / sqrt(sum x_d^2 / D + eps) * w_d
//   rotation:  angle_i = position freq_i;  a' = a cos - b sin, b' = b cos + a sin
//              for the pairs i < R / 2 (a, b): d = i and i + R / 2, or 2 i and
//              2 i + 1
//   codes:     those of s8_quantize, of the row rounded to fp32
// All of it is computed in 64 bits and rounded to fp32 once.  The angle of
// position 10^6 has 20 bits before its point, which 32 bits would take from
// those behind it; and a key's code is then the same whatever order the sum
// of squares is added in, but for values within 1e-15 of a half.  On this card
// 64-bit fused multiplications run at the rate of 32-bit ones.
//
// A wave has some rows of one token and one kind (queries, keys or values), a
// group of L lanes a row at a time, each lane four pairs of it: the rotation
// needs no other lane, and sines, cosines and weights stay in registers from
// row to row.  No wave waits for another.
//
// Bound by memory, with the 64-bit arithmetic close behind it (vector units 82%
// busy): 8192 tokens of 32 + 8 heads of 128 bf16 take 38.6 us, 4.4 TB/s of the
// 5.1 that a large copy reaches (61 us with a row a wave, which computed each
// token's sines for every row); with the cache in codes 48-53 us, in bf16 46.
// Few rows are bound by the launch and one trip to memory: one token 3.5 us.
#include <initializer_list>

#include "kv_common.h"

namespace fp32gemm {
namespace {

constexpr int NT = 256;  // threads of a workgroup

template <class T> struct Four {
  typedef T type __attribute__((ext_vector_type(4)));
  typedef T anywhere __attribute__((ext_vector_type(4), aligned(alignof(T))));
};

// Elements [0, n) of p, zero behind them; and back.
template <class T, bool WHOLE, class V> __device__ __forceinline__ void load4(const T *p, int n, V *v) {
  if (WHOLE || n == 4) {
    const typename Four<T>::type c = *reinterpret_cast<const typename Four<T>::anywhere *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (V)c[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < n ? (V)p[e] : (V)0.0f;
  }
}
template <class T, bool WHOLE> __device__ __forceinline__ void store4(T *p, int n, const float *v, bool past_caches) {
  if (WHOLE || n == 4) {
    typename Four<T>::type c;
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = (T)v[e];
    typename Four<T>::anywhere *to = reinterpret_cast<typename Four<T>::anywhere *>(p);
    if (past_caches) {
      asm volatile("");  // (the compiler makes one plain store of the two, else)
      __builtin_nontemporal_store(c, to);
      asm volatile("");
    } else {
      *to = c;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) p[e] = (T)v[e];
  }
}

// sin and cos of an angle below 2^50 in magnitude: the nearest multiple of
// pi / 2 is taken off in three parts of it (Cody and Waite; the fused
// multiplication leaves no error in the first), the rest, within pi / 4, goes
// into the two Taylor series, whose next terms are below 2^-55.
struct SinCos {
  double s, c;
};
__device__ __forceinline__ SinCos sin_cos(double x) {
  const double n = __builtin_rint(x * 0x1.45f306dc9c883p-1);
  double r = __builtin_fma(-n, 0x1.921fb54442d18p+0, x);
  r = __builtin_fma(-n, 0x1.1a62633145c07p-54, r);
  r = __builtin_fma(-n, -0x1.f1976b7ed8fbcp-110, r);
  const double z = r * r;
  double s = 1.0 / 355687428096000.0;  // 17!
  s = __builtin_fma(s, z, -1.0 / 1307674368000.0);
  s = __builtin_fma(s, z, 1.0 / 6227020800.0);
  s = __builtin_fma(s, z, -1.0 / 39916800.0);
  s = __builtin_fma(s, z, 1.0 / 362880.0);
  s = __builtin_fma(s, z, -1.0 / 5040.0);
  s = __builtin_fma(s, z, 1.0 / 120.0);
  s = __builtin_fma(s, z, -1.0 / 6.0);
  s = __builtin_fma(s * z, r, r);
  double c = -1.0 / 6402373705728000.0;  // 18!
  c = __builtin_fma(c, z, 1.0 / 20922789888000.0);
  c = __builtin_fma(c, z, -1.0 / 87178291200.0);
  c = __builtin_fma(c, z, 1.0 / 479001600.0);
  c = __builtin_fma(c, z, -1.0 / 3628800.0);
  c = __builtin_fma(c, z, 1.0 / 40320.0);
  c = __builtin_fma(c, z, -1.0 / 720.0);
  c = __builtin_fma(c, z, 1.0 / 24.0);
  c = __builtin_fma(c, z, -0.5);
  c = __builtin_fma(c, z, 1.0);
  const int q = (int)((long long)n & 3);
  const double u = q & 1 ? c : s, v = q & 1 ? s : c;
  return {q & 2 ? -u : u, (q + 1) & 2 ? -v : v};
}

__device__ __forceinline__ void rotate(double &a, double &b, const SinCos &t) {
  const double u = a * t.c - b * t.s;
  b = b * t.c + a * t.s;
  a = u;
}

// The value of another lane of the row: in step S the other of the pair, the
// other pair of the quad, and from there on a lane of the other half of 8, 16,
// 32 and 64 lanes, whose lanes all hold the same by then.
template <int S> __device__ __forceinline__ uint32_t across(uint32_t v) {
  constexpr int kDpp[4] = {0xb1, 0x4e, 0x141, 0x140};
  if constexpr (S < 4) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kDpp[S < 4 ? S : 0], 0xf, 0xf, false);
  } else {
    const auto p = S == 4 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                          : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return (threadIdx.x & (S == 4 ? 16 : 32)) ? p[0] : p[1];
  }
}
template <int S> __device__ __forceinline__ double across(double v) {
  const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
  const uint32_t lo = across<S>((uint32_t)b), hi = across<S>((uint32_t)(b >> 32));
  return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
__device__ __forceinline__ double both(double a, double b) { return a + b; }
__device__ __forceinline__ uint32_t both(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Sum (of doubles) or maximum (of words) over a row's L lanes, in all of them.
template <int L, class V> __device__ __forceinline__ V over_row(V v) {
  v = both(v, across<0>(v));
  v = both(v, across<1>(v));
  v = both(v, across<2>(v));
  if constexpr (L > 8) v = both(v, across<3>(v));
  if constexpr (L > 16) v = both(v, across<4>(v));
  if constexpr (L > 32) v = both(v, across<5>(v));
  return v;
}

// 1 / sqrt(x): the hardware's estimate (23 bits) and two Newton steps; of
// infinity the estimate itself, 0, where a step would make a NaN.
__device__ __forceinline__ double rsqrt64(double x) {
  const double estimate = __builtin_amdgcn_rsq(x);
  double y = estimate;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double h = 0.5 * y;
    y = __builtin_fma(h, __builtin_fma(-x * y, y, 1.0), y);
  }
  return x < __builtin_inf() ? y : estimate;
}

// Where a slot's row starts, in rows; -1 for slots outside the cache.
__device__ __forceinline__ long long cache_row(const KvCache &c, int slot, int head) {
  if (slot < 0 || slot >= c.pages * c.page_size) return -1;
  const int page = slot / c.page_size;
  return ((long long)page * c.heads + head) * c.page_size + (slot - page * c.page_size);
}

// CACHE: 0 none, 1 in the operands' type, 2 codes.  WHOLE: every lane's four
// pairs exist, or none of them.  A step is 64 / L rows of one kind; a token's
// steps are its queries', keys' and values', and a wave takes `steps` of them
// behind each other.
template <class T, int L, bool WHOLE, int CACHE>
__global__ void __launch_bounds__(NT) kv_rows_kernel(KvRowArgs a, int steps) {
  constexpr int RPS = 64 / L;  // rows of a step
  __shared__ SinCos turns_of[NT / 64][4 * L];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sq = (a.Hq + RPS - 1) / RPS, sk = (a.Hk + RPS - 1) / RPS, sv = (a.Hv + RPS - 1) / RPS;
  const int pieces = (sq + sk + sv + steps - 1) / steps;
  const int unit = blockIdx.x * (NT / 64) + wave;
  const int t = unit / pieces, s0 = (unit - t * pieces) * steps;
  if (t >= a.T) return;  // a wave by itself: nothing is shared
  int s1 = min(s0 + steps, sq + sk + sv);
  long long row0 = 0;
  if (CACHE > 0 && s1 > sq) {
    row0 = cache_row(a.cache, a.slots[t], 0);
    if (row0 < 0) s1 = min(s1, sq);
  }
  const int half = a.R / 2;

  // the lane's four pairs of a row
  const int c = lane % L, group = lane / L;
  int pa, pb, n;
  bool turns;
  if (a.style == 0) {
    const int c1 = (half + 3) / 4;
    turns = c < c1;
    const int cc = turns ? c : c - c1, hh = turns ? half : a.D / 2 - half;
    pa = (turns ? 0 : 2 * half) + 4 * cc;
    pb = pa + hh;
    n = min(4, hh - 4 * cc);
  } else {
    // two pairs of each half of the row, so that the lanes' stores lie next to
    // each other (with four pairs in a run, 8192 tokens of 32 + 8 heads of 128
    // fp32 took 77 us, past the caches 146; now 67, as halves do)
    pa = 4 * c;
    pb = a.D / 2 + 4 * c;
    turns = 2 * c < half;  // pb's pairs are behind pa's
    n = 8 * c < a.D ? 4 : 0;
  }
  auto pair = [&](int e) { return a.style == 0 ? 4 * c + e : (e < 2 ? pa : pb) / 2 + e % 2; };
  SinCos turn[4];
  if (half > 0 && s0 < sq + sk) {
    SinCos *mine = turns_of[wave];
    const double position = (double)a.pos[t];
    for (int e = lane; e < half; e += 64) mine[e] = sin_cos(position * a.freq[e]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's own LDS is in order
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = pair(e);
      turn[e] = turns && i < half ? mine[i] : SinCos{0.0, 1.0};
    }
  }

  // a step's row, asked for a step before it is used
  struct Row {
    T v[8];
  };
  auto load = [&](int s) {
    const bool query = s < sq, value = s >= sq + sk;
    const int h = (s - (query ? 0 : value ? sq + sk : sq)) * RPS + group;
    const T *x = static_cast<const T *>(query ? a.Q : value ? a.V : a.K) +
                 (long long)t * (query ? a.ldq : value ? a.ldv : a.ldk) + h * a.D;
    Row r = {};
    if (s < s1 && h < (query ? a.Hq : value ? a.Hv : a.Hk) && n > 0) {
      load4<T, WHOLE>(x + pa, n, r.v);
      load4<T, WHOLE>(x + pb, n, r.v + 4);
    }
    return r;
  };
  int kind = -1;  // of the weights in g
  float g[8];
  Row next = load(s0);
  for (int s = s0; s < s1; ++s) {
    const bool query = s < sq, value = s >= sq + sk;
    const int now = query ? 0 : value ? 2 : 1;
    const int h = (s - (query ? 0 : value ? sq + sk : sq)) * RPS + group;
    const T *w = static_cast<const T *>(query ? a.Wq : value ? nullptr : a.Wk);
    const bool has = h < (query ? a.Hq : value ? a.Hv : a.Hk) && n > 0;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)next.v[e];
    next = load(s + 1);
    if (now != kind) {
      kind = now;
      if (w != nullptr && n > 0) {
        load4<T, WHOLE>(w + pa, n, g);
        load4<T, WHOLE>(w + pb, n, g + 4);
      }
    }
    if (!value && (w != nullptr || half > 0)) {
      double v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (double)f[e];
      if (w != nullptr) {
        double ss = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fma(v[e], v[e], ss);
        const double rstd = rsqrt64(__builtin_fma(over_row<L>(ss), a.inv_dim, (double)a.eps));
        if (n > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= rstd * (double)g[e];
        }
      }
      if (turns) {
        if (a.style == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) rotate(v[e], v[e + 4], turn[e]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (pair(e) < half) rotate(v[2 * e], v[2 * e + 1], turn[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
    }
    if (CACHE == 2 && !query) {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, abs_bits(f[e]));
      top = over_row<L>(top);
      if (has) {
        const float scale = row_scale(top), inv = quick_inv(scale);
        const long long row = row0 + (long long)h * a.cache.page_size;
        int8_t *q = static_cast<int8_t *>(value ? a.cache.V : a.cache.K) + row * a.D;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float u[4] = {f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]};
          const uint32_t word = code_word(u, inv, scale);
          int8_t *p = q + (k ? pb : pa);
          if (WHOLE || n == 4) {
            typedef uint32_t anywhere __attribute__((aligned(1)));
            *reinterpret_cast<anywhere *>(p) = word;
          } else {
            for (int e = 0; e < n; ++e) p[e] = (int8_t)(word >> 8 * e);
          }
        }
        if (c == 0) (value ? a.cache.scaleV : a.cache.scaleK)[row] = scale;
      }
    } else if (has) {
      T *y;
      if (query)
        y = static_cast<T *>(a.Yq) + (long long)t * a.ldyq + h * a.D;
      else if (CACHE == 0)
        y = static_cast<T *>(a.Yk) + (long long)t * a.ldyk + h * a.D;
      else
        y = static_cast<T *>(value ? a.cache.V : a.cache.K) + (row0 + (long long)h * a.cache.page_size) * a.D;
      store4<T, WHOLE>(y + pa, n, f, a.past_caches);
      store4<T, WHOLE>(y + pb, n, f + 4, a.past_caches);
    }
  }
}

// Whether the halves of 128-byte lines come from different stores in half of a
// row's lines or more.  A row of 16-bit values is written by two stores, whose
// runs, which end at `ends`, take turns.
bool halved_lines(int D, std::initializer_list<int> ends) {
  if (2 * D % 128 != 0) return false;
  int halved = 0;
  for (int line = 0; line < 2 * D; line += 128) {
    int turn[2] = {0, 0};
    bool whole = true;
    for (int half = 0; half < 2; ++half)
      for (int e : ends) {
        const int past = 2 * e - (line + 64 * half);
        if (past <= 0) turn[half] ^= 1;
        if (past > 0 && past < 64) whole = false;
      }
    halved += whole && turn[0] != turn[1];
  }
  return 4 * 64 * halved >= 2 * D;
}

// Floats of this many bytes, as much as the XCDs' caches hold, are stored past
// them: whatever reads them next finds them in memory anyway.  8192 tokens of
// 32 + 8 heads of 128 bf16 39.7 -> 37.7 us, with codes for the cache 47.5 ->
// 45.4; 4096 of fp32 40.4 -> 36.4.  But not where that writes to memory in parts:
//
//  fp32, where the two stores of a row, whose runs end at `ends`, often share 64
//    bytes: 64 values of which 16 turn 46.7 us with the caches and 61.6 past them
//    (2 of a row's 4 pieces of 64 bytes), 128 of which 16 turn 42.2 and 46.5 (2
//    of 8), 192 of which 16 turn 41.8 and 38.8 (2 of 12).
//  16 bits, where lines are halved, from 75 MB on, with rows next to each other
//    (bf16, 32 + 8 heads, with the caches and past them, us): 64 of 128 turn, 36
//    MB 18.0 and 16.8, 72 MB 33.8 and 31.0, 84 MB 39.1 and 42.5, 120 MB 52.2 and
//    53.1, 250 MB equal; 64 of 64 in pairs at 84 MB 39.9 and 42.9, 64 of 256 (2 of
//    4 lines) 39.0 and 40.3, 64 of 192 (1 of 3) 46.8 and 46.0.  46 other layouts of
//    16 to 256 values, and rows from any address, are 3% slower to 15% faster past
//    the caches, all of them 7% and more at 60 MB; the rows of a cache 5% slower to
//    14% faster, what is read from one 11 to 39% faster.
bool past_caches(long long values, int size, int D, std::initializer_list<int> ends, bool aligned, bool next_to_each_other) {
  if (values * size < 32 << 20) return false;
  if (size == 2) return !(next_to_each_other && aligned && values * size >= 75 << 20 && halved_lines(D, ends));
  int shared = 0;
  for (int e : ends)
    if (!aligned || e * size % 64 != 0) ++shared;
  return 80 * (shared + !aligned) < D;
}

// Lanes of a row: the power of two that holds its groups of four pairs.
int lanes_of(const KvRowArgs &a) {
  const int groups = a.style == 0 ? (a.R / 2 + 3) / 4 + ((a.D - a.R) / 2 + 3) / 4 : a.D / 8;
  return groups <= 8 ? 8 : groups <= 16 ? 16 : groups <= 32 ? 32 : 64;
}

template <class T, int L, bool WHOLE> hipError_t launch_lanes(const KvRowArgs &a, hipStream_t s) {
  auto steps_of = [](int heads) { return (heads + 64 / L - 1) / (64 / L); };
  const int all = steps_of(a.Hq) + steps_of(a.Hk) + steps_of(a.Hv);
  // Several steps a wave share the token's sines; one at a time fills the GPU
  // with fewer tokens.  bf16, 32 + 8 heads of 128, steps of 1 / 2 / 5 / 10: 128
  // tokens 4.3 / 4.8 / 6.8 / 10.2 us, 1024 11.1 / 9.1 / 10.4 / 13.3, 8192 61 /
  // 46 / 39.6 / 43.  A token's pieces are made alike.
  int steps = (int)(((long long)a.T * all + 3000) / 6000);
  steps = steps < 1 ? 1 : steps > 6 ? 6 : steps;
  const int pieces = (all + steps - 1) / steps;
  steps = (all + pieces - 1) / pieces;
  const long long units = (long long)a.T * ((all + steps - 1) / steps);
  const int grid = (int)((units + NT / 64 - 1) / (NT / 64));
  if (a.cache.type < 0)
    kv_rows_kernel<T, L, WHOLE, 0><<<grid, NT, 0, s>>>(a, steps);
  else if (a.cache.type == kTypeS8)
    kv_rows_kernel<T, L, WHOLE, 2><<<grid, NT, 0, s>>>(a, steps);
  else
    kv_rows_kernel<T, L, WHOLE, 1><<<grid, NT, 0, s>>>(a, steps);
  return hipGetLastError();
}

template <class T> hipError_t launch_type(const KvRowArgs &all, hipStream_t s) {
  const int RT = all.Hq + all.Hk + all.Hv;
  if (RT == 0) return hipSuccess;
  const int L = lanes_of(all);
  const int floats = all.Hq + (all.cache.type == kTypeS8 ? 0 : all.Hk + all.Hv);
  const bool whole = all.style != 0 || all.R % 8 == 0;
  auto in64 = [](const void *p, int ld) { return ((uintptr_t)p | (uintptr_t)ld * sizeof(T)) % 64 == 0; };
  const bool aligned = in64(all.Yq, all.ldyq) && in64(all.Yk, all.ldyk) &&
                       (all.cache.type < 0 || (in64(all.cache.K, 0) && in64(all.cache.V, 0)));
  const long long values = (long long)all.T * floats * all.D;
  const bool rows = all.Hq > 0 || all.cache.type < 0;  // next to each other, not only those of a cache
  const bool past = all.style == 0
                        ? past_caches(values, sizeof(T), all.D, {all.R / 2, all.R, (all.D + all.R) / 2}, aligned, rows)
                        : past_caches(values, sizeof(T), all.D, {all.D / 2}, aligned, rows);
  // a launch's threads stay below 2^31
  const int most = (1 << 24) / RT > 0 ? (1 << 24) / RT : 1;
  for (long long t0 = 0; t0 < all.T; t0 += most) {
    KvRowArgs a = all;
    a.T = (int)(all.T - t0 < most ? all.T - t0 : most);
    a.past_caches = past;
    a.Q = static_cast<const T *>(all.Q) + t0 * all.ldq;
    a.K = static_cast<const T *>(all.K) + t0 * all.ldk;
    a.V = static_cast<const T *>(all.V) + t0 * all.ldv;
    a.Yq = static_cast<T *>(all.Yq) + t0 * all.ldyq;
    a.Yk = static_cast<T *>(all.Yk) + t0 * all.ldyk;
    a.pos = all.pos + t0;
    a.slots = all.slots + t0;
    hipError_t e;
    if (whole)
      e = L == 8 ? launch_lanes<T, 8, true>(a, s) : L == 16 ? launch_lanes<T, 16, true>(a, s)
                                                            : launch_lanes<T, 32, true>(a, s);
    else
      e = L == 8 ? launch_lanes<T, 8, false>(a, s)
          : L == 16 ? launch_lanes<T, 16, false>(a, s)
          : L == 32 ? launch_lanes<T, 32, false>(a, s)
                    : launch_lanes<T, 64, false>(a, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Rows of the cache as floats: L lanes a row, eight values a lane, which is 16
// bytes of 16-bit outputs and 8 of codes.  Bound by memory: 8192 tokens of 2 x 8
// heads of 128, codes to bf16, 11.0 us (4.6 TB/s).
template <class T, int L, bool CODES> __global__ void __launch_bounds__(NT) kv_read_kernel(KvReadArgs a) {
  const int heads = a.cache.heads, D = a.cache.dim;
  // eight values of 16 bits in a run, or twice four of 32, so that stores lie next to each other
  constexpr bool kTwo = sizeof(T) == 4;
  const int i = blockIdx.x * (NT / L) + (int)threadIdx.x / L, c = threadIdx.x % L;
  const int d = c * (kTwo ? 4 : 8), d1 = kTwo ? D / 2 + d : d + 4;
  const int t = i / (2 * heads);
  if (t >= a.T || 8 * c >= D) return;
  const int h = i - t * 2 * heads;
  const bool value = h >= heads;
  const int head = value ? h - heads : h;
  const long long row = cache_row(a.cache, a.slots[t], head);
  if (row < 0) return;
  T *y = value ? static_cast<T *>(a.V) + (long long)t * a.ldv : static_cast<T *>(a.K) + (long long)t * a.ldk;
  y += head * D;
  const void *src = value ? a.cache.V : a.cache.K;
  float f[8];
  if constexpr (CODES) {
    typedef int8_t codes __attribute__((ext_vector_type(4)));
    const int8_t *q = static_cast<const int8_t *>(src) + row * D;
    const codes lo = *reinterpret_cast<const codes *>(q + d), hi = *reinterpret_cast<const codes *>(q + d1);
    const float scale = (value ? a.cache.scaleV : a.cache.scaleK)[row];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = (float)lo[e] * scale, f[4 + e] = (float)hi[e] * scale;
  } else {
    load4<T, true>(static_cast<const T *>(src) + row * D + d, 4, f);
    load4<T, true>(static_cast<const T *>(src) + row * D + d1, 4, f + 4);
  }
  if constexpr (kTwo) {
    store4<T, true>(y + d, 4, f, a.past_caches);
    store4<T, true>(y + d1, 4, f + 4, a.past_caches);
  } else {
    typedef T eight __attribute__((ext_vector_type(8)));
    typedef T anywhere __attribute__((ext_vector_type(8), aligned(alignof(T))));
    eight v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (T)f[e];
    if (a.past_caches) {
      asm volatile("");  // as in store4
      __builtin_nontemporal_store(v, reinterpret_cast<anywhere *>(y + d));
      asm volatile("");
    } else {
      *reinterpret_cast<anywhere *>(y + d) = v;
    }
  }
}

template <class T> hipError_t launch_read(const KvReadArgs &all, hipStream_t s) {
  const int rows = 2 * all.cache.heads, lanes = all.cache.dim / 8;
  const int L = lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
  const int most = (1 << 24) / rows > 0 ? (1 << 24) / rows : 1;
  const int D = all.cache.dim;
  const bool aligned =
      ((uintptr_t)all.K | (uintptr_t)all.V | (uintptr_t)all.ldk * sizeof(T) | (uintptr_t)all.ldv * sizeof(T)) % 64 == 0;
  const bool past = past_caches((long long)all.T * rows * D, sizeof(T), D, {sizeof(T) == 4 ? D / 2 : D}, aligned, true);
  for (long long t0 = 0; t0 < all.T; t0 += most) {
    KvReadArgs a = all;
    a.T = (int)(all.T - t0 < most ? all.T - t0 : most);
    a.past_caches = past;
    a.slots = all.slots + t0;
    a.K = static_cast<T *>(all.K) + t0 * all.ldk;
    a.V = static_cast<T *>(all.V) + t0 * all.ldv;
    const int grid = (a.T * rows + NT / L - 1) / (NT / L);
    if (a.cache.type == kTypeS8) {
      if (L == 8) kv_read_kernel<T, 8, true><<<grid, NT, 0, s>>>(a);
      else if (L == 16) kv_read_kernel<T, 16, true><<<grid, NT, 0, s>>>(a);
      else kv_read_kernel<T, 32, true><<<grid, NT, 0, s>>>(a);
    } else {
      if (L == 8) kv_read_kernel<T, 8, false><<<grid, NT, 0, s>>>(a);
      else if (L == 16) kv_read_kernel<T, 16, false><<<grid, NT, 0, s>>>(a);
      else kv_read_kernel<T, 32, false><<<grid, NT, 0, s>>>(a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_kv_rows(const KvRowArgs &a, int type, hipStream_t s) {
  if (type == kTypeF32) return launch_type<float>(a, s);
  if (type == kTypeF16) return launch_type<_Float16>(a, s);
  return launch_type<__bf16>(a, s);
}

hipError_t launch_kv_read(const KvReadArgs &a, int type, hipStream_t s) {
  if (type == kTypeF32) return launch_read<float>(a, s);
  if (type == kTypeF16) return launch_read<_Float16>(a, s);
  return launch_read<__bf16>(a, s);
}

}  // namespace fp32gemm
