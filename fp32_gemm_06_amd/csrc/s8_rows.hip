// Rows of floats to 8-bit codes with a scale each: s8_quantize, and s8_rmsnorm
// with the residual's addition in front of it.
//
//   quantize:  v_k = x_k
//   rmsnorm:   h_k = x_k + r_k rounded to the operands' type (what the
//              residual stream keeps), v_k = fl32(h_k w_k),
//              rstd = 1 / sqrt(sum h_k^2 / K + eps)
//   both:      step = fl32(max |v_k| / 127), code_k = round(v_k / step)
//   scale:     step, or fl32(step rstd)
//
// rstd is one positive number for the whole row, so the codes of v are those
// of the normalised row: the maximum and the sum of squares come from one
// pass, and no value is normalised before it is coded.  The row stays in
// registers between that pass and the codes, so memory is read once.  The
// sum of squares is kept in 64 bits: squares of float32 values pass its range.
#include "s8_common.h"

namespace fp32gemm {
namespace {

constexpr int E = 8;  // elements per thread and step

// E elements from an address aligned to the element only.
template <class T> struct Chunk {
  T v[E];
};
template <class T> __device__ __forceinline__ Chunk<T> load_chunk(const T *p) {
  Chunk<T> c;
  __builtin_memcpy(&c, p, sizeof(c));
  return c;
}

// Elements [k, k + E) of a row of K, zero past its end.
template <class T>
__device__ __forceinline__ void load_row(const T *row, int k, int K, float (&v)[E]) {
  if (k + E <= K) {
    const Chunk<T> c = load_chunk(row + k);
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = (float)c.v[e];
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = k + e < K ? (float)row[k + e] : 0.0f;
  }
}

template <class T>
__device__ __forceinline__ void store_row(T *row, int k, int K, const T (&v)[E]) {
  if (k + E <= K) {
    __builtin_memcpy(row + k, v, sizeof(v));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < K) row[k + e] = v[e];
  }
}

struct RowStat {
  uint32_t top;  // bits of the largest |v|
  double ss;     // sum of h^2
};

__device__ __forceinline__ RowStat wave_stat(RowStat s, bool norm) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t t = (uint32_t)__shfl_xor((int)s.top, d, 64);
    s.top = t > s.top ? t : s.top;
    if (norm) s.ss += __shfl_xor(s.ss, d, 64);
  }
  return s;
}

// v (and h, stored) of one chunk, and its part of the row's statistics.
template <class T, bool NORM>
__device__ __forceinline__ void chunk_values(const S8RowArgs &a, const T *x, const T *r, const T *w,
                                             T *hout, int k, float (&v)[E], RowStat &st) {
  load_row(x, k, a.K, v);
  if constexpr (NORM) {
    if (r != nullptr) {
      float q[E];
      load_row(r, k, a.K, q);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = (float)(T)(v[e] + q[e]);
    }
    if (hout != nullptr) {
      T h[E];
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = (T)v[e];
      store_row(hout, k, a.K, h);
    }
    float g[E];
    load_row(w, k, a.K, g);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      st.ss = __builtin_fma((double)v[e], (double)v[e], st.ss);
      v[e] *= g[e];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t b = abs_bits(v[e]);
    st.top = b > st.top ? b : st.top;
  }
}

__device__ __forceinline__ void chunk_codes(const S8RowArgs &a, int8_t *qrow, int k,
                                            const float (&v)[E], const RowStep &rs) {
  int8_t c[E];
#pragma unroll
  for (int e = 0; e < E; ++e) c[e] = (int8_t)row_code(v[e], rs);
  store_row(qrow, k, a.K, c);
}

// NT threads a row (a wave or more), ROWS rows a workgroup; NV chunks of a
// row in each thread's registers.  NV = 0: rows of any length, whose chunks
// are read again for the codes (from the stored sum, where there is one).
template <class T, bool NORM, int NT, int ROWS, int NV>
__global__ void __launch_bounds__(NT *ROWS) rows_kernel(S8RowArgs a) {
  constexpr int WAVES = NT / 64;
  __shared__ uint32_t tops[ROWS * WAVES];
  __shared__ double sums[ROWS * WAVES];
  const int tid = threadIdx.x % NT, sub = threadIdx.x / NT;
  const long long row = (long long)blockIdx.x * ROWS + sub;
  const bool live = row < a.M;
  const long long i = live ? row : a.M - 1;  // a row to read; nothing is written for it
  const T *x = static_cast<const T *>(a.X) + i * a.ldx;
  const T *r = a.R ? static_cast<const T *>(a.R) + i * a.ldr : nullptr;
  const T *w = static_cast<const T *>(a.W);
  T *hout = a.H && live ? static_cast<T *>(a.H) + i * a.ldh : nullptr;
  int8_t *q = a.Q + i * a.ldq;

  RowStat st = {0u, 0.0};
  float v[NV > 0 ? NV : 1][E];
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (tid + j * NT) * E;
      if (k < a.K) chunk_values<T, NORM>(a, x, r, w, hout, k, v[j], st);
    }
  } else {
    for (int k = tid * E; k < a.K; k += NT * E) chunk_values<T, NORM>(a, x, r, w, hout, k, v[0], st);
  }
  st = wave_stat(st, NORM);
  if constexpr (WAVES > 1) {
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0) {
      tops[wave] = st.top;
      sums[wave] = st.ss;
    }
    __syncthreads();
    st = {0u, 0.0};
#pragma unroll
    for (int u = 0; u < WAVES; ++u) {
      const uint32_t t = tops[sub * WAVES + u];
      st.top = t > st.top ? t : st.top;
      st.ss += sums[sub * WAVES + u];
    }
  }
  const float step = row_scale(st.top);
  if (live && tid == 0) {
    float scale = step;
    if (NORM && step > 0.0f) scale = (float)((double)step / __builtin_sqrt(st.ss / a.K + (double)a.eps));
    a.scales[i] = scale;
  }
  if (!live) return;
  const RowStep rs = row_step(step);
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (tid + j * NT) * E;
      if (k < a.K) chunk_codes(a, q, k, v[j], rs);
    }
  } else {
    // With an H the sum is read back from it (by the thread that wrote it),
    // since X or R may be the same memory.
    const T *src = hout ? hout : x;
    S8RowArgs b = a;
    RowStat none = {0u, 0.0};
    for (int k = tid * E; k < a.K; k += NT * E) {
      chunk_values<T, NORM>(b, src, hout ? nullptr : r, w, nullptr, k, v[0], none);
      chunk_codes(a, q, k, v[0], rs);
    }
  }
}

template <class T, bool NORM> hipError_t launch_rows(const S8RowArgs &a, hipStream_t s) {
  auto go = [&](auto kernel, int threads, int rows) {
    kernel<<<(a.M + rows - 1) / rows, threads, 0, s>>>(a);
    return hipGetLastError();
  };
  if (a.K <= 512) return go(rows_kernel<T, NORM, 64, 4, 1>, 256, 4);
  if (a.K <= 4096) return go(rows_kernel<T, NORM, 256, 1, 2>, 256, 1);
  if (a.K <= 8192) return go(rows_kernel<T, NORM, 256, 1, 4>, 256, 1);
  if (a.K <= 16384) return go(rows_kernel<T, NORM, 512, 1, 4>, 512, 1);
  return go(rows_kernel<T, NORM, 1024, 1, 0>, 1024, 1);
}

// Columns of X stored K x M, to rows of codes.  A workgroup takes CB columns
// over all of K: their largest values first, then 64 k at a time through LDS,
// where the codes turn from k-major to column-major.
constexpr int CB = 32;
constexpr int CT = 512;

template <class T>
__global__ void __launch_bounds__(CT) columns_kernel(S8RowArgs a) {
  constexpr int KR = CT / CB;  // k read at a time
  constexpr int KT = 64;       // k per turn through LDS
  __shared__ uint32_t tops[KR][CB];
  __shared__ int8_t turn[CB][KT + 4];
  const int c = threadIdx.x % CB, kr = threadIdx.x / CB;
  const long long col0 = (long long)blockIdx.x * CB;
  const bool live = col0 + c < a.M;
  const T *x = static_cast<const T *>(a.X) + (live ? col0 + c : a.M - 1);
  uint32_t top = 0;
  for (int k = kr; k < a.K; k += KR) {
    const uint32_t b = abs_bits((float)x[(long long)k * a.ldx]);
    top = b > top ? b : top;
  }
  tops[kr][c] = top;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < KR; ++u) top = tops[u][c] > top ? tops[u][c] : top;
  const float step = row_scale(top);
  if (live && kr == 0) a.scales[col0 + c] = step;
  const RowStep rs = row_step(step);
  for (int k0 = 0; k0 < a.K; k0 += KT) {
#pragma unroll
    for (int u = 0; u < KT / KR; ++u) {
      const int k = k0 + u * KR + kr;
      const float v = k < a.K ? (float)x[(long long)k * a.ldx] : 0.0f;
      turn[c][u * KR + kr] = (int8_t)row_code(v, rs);
    }
    __syncthreads();
    for (int f = threadIdx.x; f < CB * (KT / 4); f += CT) {
      const int cc = f / (KT / 4), k4 = f % (KT / 4) * 4;
      if (col0 + cc < a.M) {
        int8_t *q = a.Q + (col0 + cc) * a.ldq + k0 + k4;
        if (k0 + k4 + 4 <= a.K) {
          __builtin_memcpy(q, &turn[cc][k4], 4);
        } else {
          for (int e = 0; e < 4; ++e)
            if (k0 + k4 + e < a.K) q[e] = turn[cc][k4 + e];
        }
      }
    }
    __syncthreads();
  }
}

template <class T> hipError_t launch_columns(const S8RowArgs &a, hipStream_t s) {
  columns_kernel<T><<<(a.M + CB - 1) / CB, CT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_s8_rows(const S8RowArgs &a, int type, hipStream_t s) {
  const bool norm = a.W != nullptr;
  if (type == kTypeF32)
    return norm ? launch_rows<float, true>(a, s) : launch_rows<float, false>(a, s);
  if (type == kTypeF16)
    return norm ? launch_rows<_Float16, true>(a, s) : launch_rows<_Float16, false>(a, s);
  return norm ? launch_rows<__bf16, true>(a, s) : launch_rows<__bf16, false>(a, s);
}

hipError_t launch_s8_columns(const S8RowArgs &a, int type, hipStream_t s) {
  if (type == kTypeF32) return launch_columns<float>(a, s);
  if (type == kTypeF16) return launch_columns<_Float16>(a, s);
  return launch_columns<__bf16>(a, s);
}

}  // namespace fp32gemm
