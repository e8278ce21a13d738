// The 8-bit product for few rows (M <= 128): the time is one pass over W's
// codes.
//
// A workgroup owns 16 TN rows of W (columns of C) and every row of A.  Its
// waves split K into consecutive runs of 64-byte steps; a lane loads the 16
// bytes of W that it feeds to v_mfma_i32_16x16x64_i8 straight from memory, a
// step of 16 rows in one instruction (the next step reads the other half of
// the same 128-byte lines), and A's the same way, out of L2.  A batch of U
// steps is in flight while the one before is multiplied.  The waves' sums
// meet in LDS; they are integers, so their order does not matter.
#include "s8_kernel.h"

namespace fp32gemm {
namespace {

template <int TM_, int TN_, int WAVES_, int U_> struct Skinny {
  static constexpr int TM = TM_, TN = TN_, WAVES = WAVES_, U = U_;
  static constexpr int NT = WAVES * 64;
  static constexpr int ROWS = 16 * TM, COLS = 16 * TN;
};

template <class T, bool WIDE>
__global__ void __launch_bounds__(T::NT) s8_skinny_kernel(S8Args a) {
  constexpr int TM = T::TM, TN = T::TN, WAVES = T::WAVES, U = T::U;
  __shared__ intx4 part[WAVES][TM * TN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * T::COLS;
  const int cols = a.N - n0;
  const int steps = (a.K + 63) / 64;
  const int per = (steps + WAVES - 1) / WAVES;
  const int s0 = wave * per, s1 = min(s0 + per, steps);

  const int8_t *Bg = a.B + (size_t)n0 * a.ldb;
  const __amdgpu_buffer_rsrc_t rs_a = make_rsrc(a.A), rs_b = make_rsrc(Bg);
  uint32_t offa[TM], offb[TN];  // of the lane's chunk in step 0
#pragma unroll
  for (int i = 0; i < TM; ++i)
    offa[i] = 16 * i + lr < a.M ? (uint32_t)((16 * i + lr) * a.lda + 16 * lq) : kOob;
#pragma unroll
  for (int j = 0; j < TN; ++j)
    offb[j] = 16 * j + lr < cols ? (uint32_t)((16 * j + lr) * a.ldb + 16 * lq) : kOob;

  struct Batch {
    intx4 a[U][TM], b[U][TN];
  };
  auto load = [&](Batch &f, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 64 + 16 * lq;  // the lane's first k
      const bool in = s + u < s1 && k < a.K;
      const uint32_t step = (uint32_t)(s + u) * 64;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        if constexpr (WIDE)
          f.b[u][j] = __builtin_bit_cast(
              intx4, __builtin_amdgcn_raw_buffer_load_b128(rs_b, in ? offb[j] + step : kOob, 0, 0));
        else
          f.b[u][j] = s8_load16(Bg + (size_t)(16 * j + lr) * a.ldb + k,
                                s + u < s1 && 16 * j + lr < cols ? a.K - k : 0);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        if constexpr (WIDE)
          f.a[u][i] = __builtin_bit_cast(
              intx4, __builtin_amdgcn_raw_buffer_load_b128(rs_a, in ? offa[i] + step : kOob, 0, 0));
        else
          f.a[u][i] = s8_load16(a.A + (size_t)(16 * i + lr) * a.lda + k,
                                s + u < s1 && 16 * i + lr < a.M ? a.K - k : 0);
      }
    }
  };
  intx4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = intx4{0, 0, 0, 0};
  auto multiply = [&](Batch &f, int s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (WIDE && (a.K & 15) != 0 && s + u == steps - 1) {
        // the chunk that K ends in: what lies past it is not A's
        const int valid = a.K - (s + u) * 64 - 16 * lq;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int keep = valid - 4 * d;
            f.a[u][i][d] = keep >= 4 ? f.a[u][i][d]
                                     : keep <= 0 ? 0 : f.a[u][i][d] & (int)((1u << (8 * keep)) - 1);
          }
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.b[u][j], f.a[u][i], acc[i][j], 0, 0, 0);
    }
  };
  Batch f0, f1;
  load(f0, s0);
  for (int s = s0; s < s1; s += 2 * U) {
    load(f1, s + U);
    multiply(f0, s);
    load(f0, s + 2 * U);
    multiply(f1, s + U);
  }

#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) part[wave][i * TN + j][lane] = acc[i][j];
  __syncthreads();
  // Thread t adds up four columns of one row: those of lane t % 64 in block t / 64.
  const bool whole = s8_whole_runs(a, 4);
  for (int t = threadIdx.x; t < TM * TN * 64; t += T::NT) {
    const int blk = t >> 6;
    const int m = 16 * (blk / TN) + lr, n = n0 + 16 * (blk % TN) + 4 * lq;
    if (m >= a.M || n >= a.N) continue;
    intx4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) sum += part[w][blk][lane];
    s8_finish4(a, m, n, sum, whole);
  }
}

template <class T> hipError_t launch(const S8Args &a, hipStream_t s) {
  const int groups = (a.N + T::COLS - 1) / T::COLS;
  if (s8_dma_ok(a)) s8_skinny_kernel<T, true><<<groups, T::NT, 0, s>>>(a);
  else s8_skinny_kernel<T, false><<<groups, T::NT, 0, s>>>(a);
  return hipGetLastError();
}

template <int TN> hipError_t by_rows(const S8Args &a, hipStream_t s) {
  if (a.M <= 16) return launch<Skinny<1, TN, 8, 4>>(a, s);
  if (a.M <= 32) return launch<Skinny<2, TN, 8, 4>>(a, s);
  if (a.M <= 64) return launch<Skinny<4, TN, 8, 2>>(a, s);
  return launch<Skinny<8, TN, 8, 1>>(a, s);
}

}  // namespace

hipError_t launch_s8_skinny16(const S8Args &a, hipStream_t s) { return by_rows<1>(a, s); }
hipError_t launch_s8_skinny32(const S8Args &a, hipStream_t s) { return by_rows<2>(a, s); }

}  // namespace fp32gemm
