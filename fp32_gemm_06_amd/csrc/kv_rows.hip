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
// A group of L lanes has a row, each lane four pairs of it, so the rotation
// needs no other lane; sine and cosine of the workgroup's tokens are computed
// once, into LDS, for all their heads.
#include "kv_common.h"

namespace fp32gemm {
namespace {

constexpr int NT = 256;  // threads of a workgroup

template <class T> struct Four {
  typedef T type __attribute__((ext_vector_type(4)));
  typedef T anywhere __attribute__((ext_vector_type(4), aligned(alignof(T))));
};

// Elements [0, n) of p, zero behind them; and back.
template <class T, bool WHOLE> __device__ __forceinline__ void load4(const T *p, int n, float *v) {
  if (WHOLE || n == 4) {
    const typename Four<T>::type c = *reinterpret_cast<const typename Four<T>::anywhere *>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)c[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < n ? (float)p[e] : 0.0f;
  }
}
template <class T, bool WHOLE> __device__ __forceinline__ void store4(T *p, int n, const float *v) {
  if (WHOLE || n == 4) {
    typename Four<T>::type c;
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = (T)v[e];
    *reinterpret_cast<typename Four<T>::anywhere *>(p) = c;
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

template <int L> __device__ __forceinline__ double row_sum(double v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
template <int L> __device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) {
    const uint32_t t = (uint32_t)__shfl_xor((int)v, d, 64);
    v = t > v ? t : v;
  }
  return v;
}

// Where a slot's row starts, in rows; -1 for slots outside the cache.
__device__ __forceinline__ long long cache_row(const KvCache &c, int slot, int head) {
  if (slot < 0 || slot >= c.pages * c.page_size) return -1;
  const int page = slot / c.page_size;
  return ((long long)page * c.heads + head) * c.page_size + (slot - page * c.page_size);
}

// CACHE: 0 none, 1 in the operands' type, 2 codes.  WHOLE: every lane's four
// pairs exist, or none of them.
template <class T, int L, bool WHOLE, int CACHE>
__global__ void __launch_bounds__(NT) kv_rows_kernel(KvRowArgs a) {
  constexpr int RP = NT / L;  // rows of a workgroup
  __shared__ SinCos turn[4 * NT];  // a workgroup's tokens times R / 2: at most RP (4 L)
  const int RT = a.Hq + a.Hk + a.Hv;
  const int rows = a.T * RT, first = blockIdx.x * RP;
  const int half = a.R / 2;
  const int t0 = first / RT;
  if (half > 0) {
    const int t1 = min(first + RP, rows) - 1;
    const int entries = (t1 / RT - t0 + 1) * half;
    for (int e = threadIdx.x; e < entries; e += NT) {
      const int t = e / half;
      turn[e] = sin_cos((double)a.pos[t0 + t] * a.freq[e - t * half]);
    }
  }

  const int i = first + (int)threadIdx.x / L, c = threadIdx.x % L;
  const bool live = i < rows;
  const int t = live ? i / RT : t0;
  int h = live ? i - t * RT : 0;
  // the row, its norm, and where it goes
  const T *x, *w;
  T *y = nullptr;
  long long row = -1;
  bool value = false;
  if (h < a.Hq) {
    x = static_cast<const T *>(a.Q) + (long long)t * a.ldq + h * a.D;
    w = static_cast<const T *>(a.Wq);
    y = static_cast<T *>(a.Yq) + (long long)t * a.ldyq + h * a.D;
  } else {
    h -= a.Hq;
    value = h >= a.Hk;
    h -= value ? a.Hk : 0;
    x = value ? static_cast<const T *>(a.V) + (long long)t * a.ldv + h * a.D
              : static_cast<const T *>(a.K) + (long long)t * a.ldk + h * a.D;
    w = value ? nullptr : static_cast<const T *>(a.Wk);
    if constexpr (CACHE == 0) {
      y = static_cast<T *>(a.Yk) + (long long)t * a.ldyk + h * a.D;
    } else if (live) {
      row = cache_row(a.cache, a.slots[t], h);
      if constexpr (CACHE == 1)
        if (row >= 0) y = static_cast<T *>(value ? a.cache.V : a.cache.K) + row * a.D;
    }
  }
  const bool codes = CACHE == 2 && y == nullptr;
  // the lane's pairs
  int pa, pb, n;
  bool turns;
  if (a.style == 0) {
    const int c1 = (half + 3) / 4;
    turns = c < c1;
    const int cc = turns ? c : c - c1, hh = turns ? half : (a.D - a.R) / 2;
    pa = (turns ? 0 : a.R) + 4 * cc;
    pb = pa + hh;
    n = min(4, hh - 4 * cc);
  } else {
    turns = 4 * c < half;
    pa = 8 * c;
    pb = pa + 4;
    n = 8 * c < a.D ? 4 : 0;
  }
  turns = turns && !value;
  const bool has = live && n > 0 && (y != nullptr || (codes && row >= 0));

  float f[8] = {}, g[8];
  if (has) {
    load4<T, WHOLE>(x + pa, n, f);
    load4<T, WHOLE>(x + pb, n, f + 4);
  }
  if (w != nullptr && has) {
    load4<T, WHOLE>(w + pa, n, g);
    load4<T, WHOLE>(w + pb, n, g + 4);
  }
  double v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (double)f[e];
  if (a.Wq != nullptr || a.Wk != nullptr) {
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fma(v[e], v[e], ss);
    ss = row_sum<L>(ss);
    if (w != nullptr && has) {
      const double rstd = 1.0 / __builtin_sqrt(ss / a.D + (double)a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= rstd * (double)g[e];
    }
  }
  if (half > 0) {
    __syncthreads();
    if (turns && has) {
      const SinCos *sc = turn + (t - t0) * half + 4 * c;
if (a.style == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (WHOLE || e < n) rotate(v[e], v[e + 4], sc[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (4 * c + e < half) rotate(v[2 * e], v[2 * e + 1], sc[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
  if constexpr (CACHE == 2) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, abs_bits(f[e]));
    top = row_max<L>(top);
    if (codes && has) {
      const float scale = row_scale(top), inv = quick_inv(scale);
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
  }
  if (has && y != nullptr) {
    store4<T, WHOLE>(y + pa, n, f);
    store4<T, WHOLE>(y + pb, n, f + 4);
  }
}

// Lanes of a row: the power of two that holds its groups of four pairs.
int lanes_of(const KvRowArgs &a) {
  const int groups = a.style == 0 ? (a.R / 2 + 3) / 4 + ((a.D - a.R) / 2 + 3) / 4 : a.D / 8;
  return groups <= 8 ? 8 : groups <= 16 ? 16 : groups <= 32 ? 32 : 64;
}

template <class T, int L, bool WHOLE> hipError_t launch_lanes(const KvRowArgs &a, hipStream_t s) {
  const int rows = a.T * (a.Hq + a.Hk + a.Hv), grid = (rows + NT / L - 1) / (NT / L);
  if (a.cache.type < 0)
    kv_rows_kernel<T, L, WHOLE, 0><<<grid, NT, 0, s>>>(a);
  else if (a.cache.type == kTypeS8)
    kv_rows_kernel<T, L, WHOLE, 2><<<grid, NT, 0, s>>>(a);
  else
    kv_rows_kernel<T, L, WHOLE, 1><<<grid, NT, 0, s>>>(a);
  return hipGetLastError();
}

template <class T> hipError_t launch_type(const KvRowArgs &all, hipStream_t s) {
  const int RT = all.Hq + all.Hk + all.Hv;
  if (RT == 0) return hipSuccess;
  const int L = lanes_of(all);
  const bool whole = all.style != 0 || all.R % 8 == 0;
  // a launch's threads stay below 2^31
  const int most = (1 << 24) / RT > 0 ? (1 << 24) / RT : 1;
  for (long long t0 = 0; t0 < all.T; t0 += most) {
    KvRowArgs a = all;
    a.T = (int)(all.T - t0 < most ? all.T - t0 : most);
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

// Rows of the cache as floats: L lanes a row, eight values a lane.
template <class T, int L, bool CODES> __global__ void __launch_bounds__(NT) kv_read_kernel(KvReadArgs a) {
  const int heads = a.cache.heads, D = a.cache.dim;
  const int i = blockIdx.x * (NT / L) + (int)threadIdx.x / L, d = threadIdx.x % L * 8;
  const int t = i / (2 * heads);
  if (t >= a.T || d >= D) return;
  const int h = i - t * 2 * heads;
  const bool value = h >= heads;
  const int head = value ? h - heads : h;
  const long long row = cache_row(a.cache, a.slots[t], head);
  if (row < 0) return;
  T *y = value ? static_cast<T *>(a.V) + (long long)t * a.ldv : static_cast<T *>(a.K) + (long long)t * a.ldk;
  y += head * D + d;
  const void *src = value ? a.cache.V : a.cache.K;
  float f[8];
  if constexpr (CODES) {
    typedef int8_t codes __attribute__((ext_vector_type(8)));
    const codes c = *reinterpret_cast<const codes *>(static_cast<const int8_t *>(src) + row * D + d);
    const float scale = (value ? a.cache.scaleV : a.cache.scaleK)[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)c[e] * scale;
  } else {
    load4<T, true>(static_cast<const T *>(src) + row * D + d, 4, f);
    load4<T, true>(static_cast<const T *>(src) + row * D + d + 4, 4, f + 4);
  }
  store4<T, true>(y, 4, f);
  store4<T, true>(y + 4, 4, f + 4);
}

template <class T> hipError_t launch_read(const KvReadArgs &all, hipStream_t s) {
  const int rows = 2 * all.cache.heads, lanes = all.cache.dim / 8;
  const int L = lanes <= 8 ? 8 : lanes <= 16 ? 16 : 32;
  const int most = (1 << 24) / rows > 0 ? (1 << 24) / rows : 1;
  for (long long t0 = 0; t0 < all.T; t0 += most) {
    KvReadArgs a = all;
    a.T = (int)(all.T - t0 < most ? all.T - t0 : most);
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
