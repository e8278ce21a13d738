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
// Bound by memory: 8192 x 4096 bf16 with residual 43.9 us, 5.35 TB/s (a copy of
// 1 GiB 5.16).  One row is one workgroup's latency, from the loads through the
// reduction to the codes (1 x 4096, eight waves: 3.1 us, launch and all, in a
// captured run of calls).
#include "s8_common.h"

namespace fp32gemm {
namespace {

constexpr int E = 8;  // elements of a thread's chunk of a row

// E elements in registers, and at any address of an element (the hardware
// takes wide accesses at any alignment).
template <class T> struct ChunkOf {
  typedef T type __attribute__((ext_vector_type(E)));
  typedef T anywhere __attribute__((ext_vector_type(E), aligned(alignof(T))));
};

// Elements [k, k + E) of a row of K, zero past its end; and back.  WHOLE: K is
// a multiple of E, and no chunk ends past it.
template <class T, bool WHOLE>
__device__ __forceinline__ typename ChunkOf<T>::type load_chunk(const T *row, int k, int K) {
  typename ChunkOf<T>::type c = {};
  if (WHOLE || k + E <= K) {
    c = *reinterpret_cast<const typename ChunkOf<T>::anywhere *>(row + k);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < K) c[e] = row[k + e];
  }
  return c;
}
template <class T, bool WHOLE>
__device__ __forceinline__ void store_chunk(T *row, int k, int K, typename ChunkOf<T>::type c) {
  if (WHOLE || k + E <= K) {
    *reinterpret_cast<typename ChunkOf<T>::anywhere *>(row + k) = c;
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < K) row[k + e] = c[e];
  }
}

struct RowStat {
  uint32_t top;  // bits of the largest |v|
  double ss;     // sum of h^2
};

// Sum and maximum over the wave's lanes, by cross-lane moves in the vector
// unit (towards lane 63, then to all).
template <int CTRL, int ROWS> __device__ __forceinline__ int lanes(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS, bool NORM> __device__ __forceinline__ void fold(RowStat &s) {
  const uint32_t t = (uint32_t)lanes<CTRL, ROWS>((int)s.top);
  s.top = t > s.top ? t : s.top;
  if constexpr (NORM) {
    const unsigned long long b = __builtin_bit_cast(unsigned long long, s.ss);
    const uint32_t lo = (uint32_t)lanes<CTRL, ROWS>((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)lanes<CTRL, ROWS>((int)(uint32_t)(b >> 32));
    s.ss += __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
  }
}
template <bool NORM> __device__ __forceinline__ RowStat wave_stat(RowStat s) {
  fold<0x111, 0xf, NORM>(s);  // from 1, 2, 4, 8 lanes below in a row of 16
  fold<0x112, 0xf, NORM>(s);
  fold<0x114, 0xf, NORM>(s);
  fold<0x118, 0xf, NORM>(s);
  fold<0x142, 0xa, NORM>(s);  // lane 15 of a row to the next row
  fold<0x143, 0xc, NORM>(s);  // lane 31 to the upper half
  s.top = (uint32_t)__builtin_amdgcn_readlane((int)s.top, 63);
  if constexpr (NORM) {
    const unsigned long long b = __builtin_bit_cast(unsigned long long, s.ss);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
    s.ss = __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
  }
  return s;
}

// A chunk as it is read: X, and for the norm R and W.
template <class T> struct Raw {
  typename ChunkOf<T>::type x, r, w;
};
template <class T, bool NORM, bool WHOLE>
__device__ __forceinline__ void read_raw(Raw<T> &c, const T *x, const T *r, const T *w, int k, int K) {
  c.x = load_chunk<T, WHOLE>(x, k, K);
  if constexpr (NORM) {
    if (r != nullptr) c.r = load_chunk<T, WHOLE>(r, k, K);
    c.w = load_chunk<T, WHOLE>(w, k, K);
  }
}

// v (and h, stored) of one chunk, and its part of the row's statistics.
template <class T, bool NORM, bool WHOLE>
__device__ __forceinline__ void chunk_values(const Raw<T> &c, bool residual, T *hout, int k, int K,
                                             float (&v)[E], RowStat &st) {
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = (float)c.x[e];
  if constexpr (NORM) {
    typename ChunkOf<T>::type h = c.x;
    if (residual) {
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = (T)(v[e] + (float)c.r[e]);
    }
    if (hout != nullptr) store_chunk<T, WHOLE>(hout, k, K, h);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float f = (float)h[e];
      st.ss = __builtin_fma((double)f, (double)f, st.ss);
      v[e] = f * (float)c.w[e];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const uint32_t b = abs_bits(v[e]);
    st.top = b > st.top ? b : st.top;
  }
}

// Codes of one chunk of a row with this scale.
template <bool WHOLE>
__device__ __forceinline__ void chunk_codes(int8_t *qrow, int k, int K, const float (&v)[E], float inv,
                                            float scale) {
  uint32_t w[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const float f[4] = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
    w[g] = code_word(f, inv, scale);
  }
  if (WHOLE || k + E <= K) {
    typedef uint32_t words __attribute__((ext_vector_type(2)));
    typedef uint32_t anywhere __attribute__((ext_vector_type(2), aligned(1)));
    *reinterpret_cast<anywhere *>(qrow + k) = words{w[0], w[1]};
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (k + e < K) qrow[k + e] = (int8_t)(w[e / 4] >> 8 * (e % 4));
  }
}

// A row for each blockDim.x / ROWS threads; NV chunks of it in each thread's
// registers, all read before the first is used.  NV = 0: rows of any length,
// whose chunks are read again for the codes (from the stored sum, where there
// is one).  More than one row a workgroup: one wave each.
template <class T, bool NORM, int ROWS, int NV, bool WHOLE>
__global__ void __launch_bounds__(ROWS > 1 ? 64 * ROWS : 1024) rows_kernel(S8RowArgs a) {
  __shared__ uint32_t tops[16];
  __shared__ double sums[16];
  const int nt = ROWS > 1 ? 64 : blockDim.x;
  const int tid = ROWS > 1 ? threadIdx.x & 63 : threadIdx.x;
  const long long i = (long long)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x >> 6 : 0);
  if (i >= a.M) return;  // whole waves, and only where there is no barrier
  const int K = a.K;
  const T *x = static_cast<const T *>(a.X) + i * a.ldx;
  const T *r = a.R ? static_cast<const T *>(a.R) + i * a.ldr : nullptr;
  const T *w = static_cast<const T *>(a.W);
  T *hout = a.H ? static_cast<T *>(a.H) + i * a.ldh : nullptr;
  int8_t *q = a.Q + i * a.ldq;

  RowStat st = {0u, 0.0};
  float v[NV > 0 ? NV : 1][E];
  if constexpr (NV > 0) {
    Raw<T> raw[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (tid + j * nt) * E;
      if (k < K) read_raw<T, NORM, WHOLE>(raw[j], x, r, w, k, K);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (tid + j * nt) * E;
      if (k < K) chunk_values<T, NORM, WHOLE>(raw[j], r != nullptr, hout, k, K, v[j], st);
    }
  } else {
    for (int k = tid * E; k < K; k += nt * E) {
      Raw<T> raw;
      read_raw<T, NORM, WHOLE>(raw, x, r, w, k, K);
      chunk_values<T, NORM, WHOLE>(raw, r != nullptr, hout, k, K, v[0], st);
    }
  }
  st = wave_stat<NORM>(st);
  if constexpr (ROWS == 1) {
    const int waves = nt / 64;
    if (tid % 64 == 0) {
      tops[tid / 64] = st.top;
      if constexpr (NORM) sums[tid / 64] = st.ss;
    }
    __syncthreads();
    st = {0u, 0.0};
    for (int u = 0; u < waves; ++u) {
      st.top = tops[u] > st.top ? tops[u] : st.top;
      if constexpr (NORM) st.ss += sums[u];
    }
  }
  const float step = row_scale(st.top);
  const float inv = quick_inv(step);
  if constexpr (NV > 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = (tid + j * nt) * E;
      if (k < K) chunk_codes<WHOLE>(q, k, K, v[j], inv, step);
    }
  } else {
    // With an H the sum is read back from it (by the thread that wrote it),
    // since X or R may be the same memory.
    const T *src = hout ? hout : x;
    const T *add = hout ? nullptr : r;
    RowStat none = {0u, 0.0};
    for (int k = tid * E; k < K; k += nt * E) {
      Raw<T> raw;
      read_raw<T, NORM, WHOLE>(raw, src, add, w, k, K);
      chunk_values<T, NORM, WHOLE>(raw, add != nullptr, static_cast<T *>(nullptr), k, K, v[0], none);
      chunk_codes<WHOLE>(q, k, K, v[0], inv, step);
    }
  }
  if (tid == 0) {
    float scale = step;
    if (NORM && step > 0.0f) scale = (float)((double)step / __builtin_sqrt(st.ss / K + (double)a.eps));
    a.scales[i] = scale;
  }
}

// Rows of one launch: keeps the grid's threads below 2^32 for any M.
constexpr int kMaxLaunchRows = 1 << 21;

template <class T, bool NORM, bool WHOLE> hipError_t launch_rows(const S8RowArgs &all, hipStream_t s) {
  const int chunks = (all.K + E - 1) / E;
  for (long long m0 = 0; m0 < all.M; m0 += kMaxLaunchRows) {
    S8RowArgs a = all;
    a.M = (int)(all.M - m0 < kMaxLaunchRows ? all.M - m0 : kMaxLaunchRows);
    a.X = static_cast<const T *>(all.X) + m0 * all.ldx;
    if (all.R) a.R = static_cast<const T *>(all.R) + m0 * all.ldr;
    if (all.H) a.H = static_cast<T *>(all.H) + m0 * all.ldh;
    a.Q += m0 * all.ldq;
    a.scales += m0;
    // Whole waves of threads with NV chunks each.  With a row or less for each
    // CU its latency counts, and one chunk a thread is the quicker (bf16 norm,
    // 128 x 4096: 3.6 against 4.5 us); with many rows two chunks in flight
    // are (8192 x 4096: 43.8 against 45.1).  In between one would still be the
    // quicker by 5 to 10% (512 x 4096: 5.7 against 6.0).  Four spill in fp32.
    auto threads = [&](int nv) { return (chunks + 64 * nv - 1) / (64 * nv) * 64; };
    if (chunks <= 64)
      rows_kernel<T, NORM, 4, 1, WHOLE><<<(a.M + 3) / 4, 256, 0, s>>>(a);
    else if (chunks <= 128)
      rows_kernel<T, NORM, 4, 2, WHOLE><<<(a.M + 3) / 4, 256, 0, s>>>(a);
    else if (chunks <= 1024 && a.M <= 256)
      rows_kernel<T, NORM, 1, 1, WHOLE><<<a.M, threads(1), 0, s>>>(a);
    else if (chunks <= 2048)
      rows_kernel<T, NORM, 1, 2, WHOLE><<<a.M, threads(2), 0, s>>>(a);
    else
      rows_kernel<T, NORM, 1, 0, WHOLE><<<a.M, 1024, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Columns of X stored K x M, to rows of codes.  A workgroup takes 64 bytes of
// each row of X, 1024 k at a time: four lanes read a row's 64 bytes, a thread
// four consecutive k, whose codes of a column make a word.  The words turn in
// LDS from k-major to column-major.
constexpr int CT = 1024, CK = 1024;

template <class T> struct Columns {
  static constexpr int VE = 16 / sizeof(T);  // columns of a thread
  static constexpr int CB = 4 * VE;          // of the workgroup
  static constexpr int PITCH = CK / 4 + 4;   // words of a column in LDS: 4 columns apart are 16 banks apart
  typedef T vec __attribute__((ext_vector_type(VE)));
  typedef T anywhere __attribute__((ext_vector_type(VE), aligned(alignof(T))));

  const S8RowArgs &a;
  int col0, c, g, cols;  // the workgroup's columns; the thread's, its word of 4 k, its columns in X
  const T *x;

  __device__ __forceinline__ Columns(const S8RowArgs &a_, int block, int blocks) : a(a_) {
    // neighbouring columns, which share lines of X, to the same XCD
    const int xcd = block & 7, lid = xcd * (blocks >> 3) + min(xcd, blocks & 7) + (block >> 3);
    col0 = lid * CB;
    c = threadIdx.x % 4 * VE;
    g = threadIdx.x / 4;
    cols = a.M - col0 - c;
    x = static_cast<const T *>(a.X) + col0 + c;
  }
  __device__ __forceinline__ vec load(int k) const {
    vec v = {};
    if (k < a.K) {
      const T *p = x + (long long)k * a.ldx;
      if (cols >= VE) {
        v = *reinterpret_cast<const anywhere *>(p);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (e < cols) v[e] = p[e];
      }
    }
    return v;
  }
  __device__ __forceinline__ void load4(int k0, vec (&v)[4]) const {
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = load(k0 + 4 * g + u);
  }
  __device__ __forceinline__ void see(const vec (&v)[4], uint32_t (&top)[VE]) const {
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const uint32_t b = abs_bits((float)v[u][e]);
        top[e] = b > top[e] ? b : top[e];
      }
  }
  // The workgroup's largest bits of column `threadIdx.x` (below CB).
  __device__ __forceinline__ uint32_t fold(uint32_t (&top)[VE], uint32_t (*tops)[CB]) const {
#pragma unroll
    for (int e = 0; e < VE; ++e) {
#pragma unroll
      for (int d = 4; d < 64; d <<= 1) {
        const uint32_t t = (uint32_t)__shfl_xor((int)top[e], d, 64);
        top[e] = t > top[e] ? t : top[e];
      }
      if (threadIdx.x % 64 < 4) tops[threadIdx.x / 64][c + e] = top[e];
    }
    __syncthreads();
    uint32_t t = 0;
    if (threadIdx.x < CB) {
#pragma unroll
      for (int w = 0; w < CT / 64; ++w) t = tops[w][threadIdx.x] > t ? tops[w][threadIdx.x] : t;
    }
    return t;
  }
  // Codes of 1024 k from k0: scales by column in LDS, 1 / step in registers.
  __device__ __forceinline__ void put(const vec (&v)[4], int k0, uint32_t *words, const float *scale,
                                      const float (&inv)[VE]) const {
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float f[4] = {(float)v[0][e], (float)v[1][e], (float)v[2][e], (float)v[3][e]};
      words[(c + e) * PITCH + g] = code_word(f, inv[e], scale[c + e]);
    }
    __syncthreads();
    const int left = a.K - k0;
    for (int f = threadIdx.x; f < CB * (CK / 16); f += CT) {
      const int col = f / (CK / 16), k = f % (CK / 16) * 16;
      if (col0 + col >= a.M || k >= left) continue;
      int8_t *q = a.Q + (long long)(col0 + col) * a.ldq + k0 + k;
      const uint32_t *from = words + col * PITCH + k / 4;
      if (k + 16 <= left) {
        typedef uint32_t four __attribute__((ext_vector_type(4)));
        typedef uint32_t four_anywhere __attribute__((ext_vector_type(4), aligned(1)));
        *reinterpret_cast<four_anywhere *>(q) = *reinterpret_cast<const four *>(from);
      } else {
        for (int e = 0; e < left - k; ++e) q[e] = (int8_t)(from[e / 4] >> 8 * (e % 4));
      }
    }
  }
};

// All of K in one workgroup.  The first HELD times 1024 k stay in registers
// between the columns' largest values and their codes; the rest is read twice.
template <class T, int HELD>
__global__ void __launch_bounds__(CT) columns_kernel(S8RowArgs a) {
  typedef Columns<T> C;
  __shared__ uint32_t tops[CT / 64][C::CB];
  __shared__ float scale[C::CB];
  __shared__ __attribute__((aligned(16))) uint32_t turn[2][C::CB * C::PITCH];
  const C o(a, blockIdx.x, gridDim.x);
  uint32_t top[C::VE] = {};
  typename C::vec held[HELD][4];
#pragma unroll
  for (int h = 0; h < HELD; ++h) o.load4(h * CK, held[h]);
#pragma unroll
  for (int h = 0; h < HELD; ++h) o.see(held[h], top);
  for (int k0 = HELD * CK; k0 < a.K; k0 += CK) {
    typename C::vec v[4];
    o.load4(k0, v);
    o.see(v, top);
  }
  const uint32_t t = o.fold(top, tops);
  if (threadIdx.x < C::CB) {
    scale[threadIdx.x] = row_scale(t);
    if (o.col0 + (int)threadIdx.x < a.M) a.scales[o.col0 + threadIdx.x] = row_scale(t);
  }
  __syncthreads();
  float inv[C::VE];
#pragma unroll
  for (int e = 0; e < C::VE; ++e) inv[e] = quick_inv(scale[o.c + e]);
  // one half of `turn` is written while the other may still be read: two
  // barriers lie between two writes of the same half
#pragma unroll
  for (int h = 0; h < HELD; ++h)
    if (h * CK < a.K) o.put(held[h], h * CK, turn[h & 1], scale, inv);
  for (int k0 = HELD * CK; k0 < a.K; k0 += CK) {
    typename C::vec v[4];
    o.load4(k0, v);
    o.put(v, k0, turn[k0 / CK & 1], scale, inv);
  }
}

// K over workgroups (blockIdx.y takes 1024 k), for few columns: the columns'
// largest bits by atomic maxima in `scales` (whole numbers: any order gives
// the same), then the codes, then the scales in place of the bits.
__global__ void columns_clear_kernel(float *scales, int M) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < M) scales[i] = 0.0f;
}
template <class T> __global__ void __launch_bounds__(CT) columns_top_kernel(S8RowArgs a) {
  typedef Columns<T> C;
  __shared__ uint32_t tops[CT / 64][C::CB];
  const C o(a, blockIdx.x, gridDim.x);
  uint32_t top[C::VE] = {};
  typename C::vec v[4];
  o.load4(blockIdx.y * CK, v);
  o.see(v, top);
  const uint32_t t = o.fold(top, tops);
  if (threadIdx.x < C::CB && o.col0 + (int)threadIdx.x < a.M)
    atomicMax(reinterpret_cast<uint32_t *>(a.scales) + o.col0 + threadIdx.x, t);
}
template <class T> __global__ void __launch_bounds__(CT) columns_code_kernel(S8RowArgs a) {
  typedef Columns<T> C;
  __shared__ float scale[C::CB];
  __shared__ __attribute__((aligned(16))) uint32_t turn[C::CB * C::PITCH];
  const C o(a, blockIdx.x, gridDim.x);
  typename C::vec v[4];
  o.load4(blockIdx.y * CK, v);
  if (threadIdx.x < C::CB)
    scale[threadIdx.x] = o.col0 + (int)threadIdx.x < a.M
                             ? row_scale(reinterpret_cast<const uint32_t *>(a.scales)[o.col0 + threadIdx.x])
                             : 0.0f;
  __syncthreads();
  float inv[C::VE];
#pragma unroll
  for (int e = 0; e < C::VE; ++e) inv[e] = quick_inv(scale[o.c + e]);
  o.put(v, blockIdx.y * CK, turn, scale, inv);
}
__global__ void columns_scale_kernel(float *scales, int M) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < M) scales[i] = row_scale(reinterpret_cast<const uint32_t *>(scales)[i]);
}

template <class T> hipError_t launch_columns(const S8RowArgs &a, hipStream_t s) {
  constexpr int CB = Columns<T>::CB;
  const int groups = (a.M - 1) / CB + 1, chunks = (a.K + CK - 1) / CK;
  // With half the CUs or fewer busy, K over workgroups and four launches (12 us
  // at least) are the quicker once K is long: fp32, 100 columns of 16384, 14.2
  // against 69.7 us, 1000 of 5000 18.1 against 23.8, of 3000 14.4 against 15.0;
  // bf16, whose workgroups have twice the columns, 4096 of 4096 25.5 against
  // 29.6, of 2000 18.2 against 16.4.  The rule is coarse on both sides (fp32,
  // 100 of 4096 would take 11.6 split and takes 15.9; 2048 of 5000 18.2 unsplit
  // and takes 22.8).
  if (groups <= 128 && chunks > (sizeof(T) == 4 ? 4 : 2)) {
    const int small = (a.M - 1) / 256 + 1;
    columns_clear_kernel<<<small, 256, 0, s>>>(a.scales, a.M);
    columns_top_kernel<T><<<dim3(groups, chunks), CT, 0, s>>>(a);
    columns_code_kernel<T><<<dim3(groups, chunks), CT, 0, s>>>(a);
    columns_scale_kernel<<<small, 256, 0, s>>>(a.scales, a.M);
    return hipGetLastError();
  }
  // Registers for 4096 k of fp32 save the second reading, and cost the second
  // workgroup of a CU (11008 columns of 4096: 67.4 us, holding 1024 k 72.3);
  // up to K = 1024, and for 16-bit values, whose second reading is half as
  // long, the two workgroups are worth more (16384 of 1024: 17.4 against
  // 23.2; bf16, 11008 of 4096: 61.5 against 65.0, but 16384 of 4096 82.1
  // against 77.8).  X from memory; from the last-level cache 48 and 61, and 49
  // and 53.
  if constexpr (sizeof(T) == 4) {
    if (a.K > CK) {
      columns_kernel<T, 4><<<groups, CT, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  columns_kernel<T, 1><<<groups, CT, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

template <class T> hipError_t rows_of(const S8RowArgs &a, hipStream_t s) {
  if (a.W != nullptr)
    return a.K % E == 0 ? launch_rows<T, true, true>(a, s) : launch_rows<T, true, false>(a, s);
  return a.K % E == 0 ? launch_rows<T, false, true>(a, s) : launch_rows<T, false, false>(a, s);
}

hipError_t launch_s8_rows(const S8RowArgs &a, int type, hipStream_t s) {
  if (type == kTypeF32) return rows_of<float>(a, s);
  if (type == kTypeF16) return rows_of<_Float16>(a, s);
  return rows_of<__bf16>(a, s);
}

hipError_t launch_s8_columns(const S8RowArgs &a, int type, hipStream_t s) {
  if (type == kTypeF32) return launch_columns<float>(a, s);
  if (type == kTypeF16) return launch_columns<_Float16>(a, s);
  return launch_columns<__bf16>(a, s);
}

}  // namespace fp32gemm
