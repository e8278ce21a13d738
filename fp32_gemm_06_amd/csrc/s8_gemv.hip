// The 8-bit product for one to four rows: a dot product of every row of W
// with every row of A.  The time is one pass over W's codes, and with few of
// them the way to the first and from the last.
//
// A wave takes R rows of W and walks K in blocks of 1024: a lane loads 16
// codes of each, a whole 1 KB of a row with one instruction, and the same k of
// A's rows, which stay in L2, and adds four four-way dot products for each
// pair.  The loads of UNROLL blocks are in flight together.  KW waves of a
// workgroup share the same rows and split K.  The lanes' sums meet by
// cross-lane additions, the waves' in LDS; they are integers, so the order
// does not matter.  W from memory: 1 x 11008 x 4096 9.2 us, 4.9 TB/s (16-row
// tiles 13.9); 1 x 4096 x 4096 4.9 (6.0), most of it the launch; 1 x 128256 x
// 4096 84.7, 6.2 TB/s; four rows 11.8, 6.3 and 99.  From the last-level cache
// the first two take 8.2 and 4.7, four rows 9.6 and 5.5.  Two rows of W a wave:
// with one, A is read as often as W, with four too few waves remain (from the
// cache, 4 x 11008 x 4096: 9.6, 9.6 and 14.0 us; 1 x 11007 x 4095 without
// alignment 9.7, 9.9 and 10.4).
#include "s8_kernel.h"

namespace fp32gemm {
namespace {

constexpr int kWaves = 4;

// Sum over the wave's lanes, in lane 63.
__device__ __forceinline__ int lane_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

template <int MR, int R, int KW>
__global__ void __launch_bounds__(64 * kWaves) s8_gemv_kernel(S8Args a) {
  constexpr int GROUPS = kWaves / KW, COLS = GROUPS * R;
  constexpr int UNROLL = MR * R <= 4 ? 4 : 2;
  __shared__ int part[kWaves][MR * R];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = blockIdx.y * MR;
  const int n0 = blockIdx.x * COLS;
  // rows past the end are the last one again; their sums are not stored
  const int8_t *x[MR], *w[R];
#pragma unroll
  for (int i = 0; i < MR; ++i) x[i] = a.A + (size_t)min(m0 + i, a.M - 1) * a.lda + 16 * lane;
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = a.B + (size_t)min(n0 + wave / KW * R + r, a.N - 1) * a.ldb + 16 * lane;
  const int blocks = (a.K + 1023) / 1024, each = (blocks + KW - 1) / KW;
  const int b0 = wave % KW * each, b1 = min(b0 + each, blocks);

  int acc[MR][R];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) acc[i][r] = 0;
  auto block = [&](int k, int valid) {
    intx4 xv[MR], wv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) wv[r] = s8_load16(w[r] + k, valid, a.K);
#pragma unroll
    for (int i = 0; i < MR; ++i) xv[i] = s8_load16(x[i] + k, valid, a.K);
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[i][r] = __builtin_amdgcn_sdot4(xv[i][d], wv[r][d], acc[i][r], false);
  };
  const int whole = min(b1, a.K / 1024);
  int b = b0;
#pragma unroll UNROLL
  for (; b < whole; ++b) block(b * 1024, 16);
  if (b < b1) block(b * 1024, a.K - b * 1024 - 16 * lane);  // the block that K ends in

#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int s = lane_sum(acc[i][r]);
      if (lane == 63) part[wave][i * R + r] = s;
    }
  __syncthreads();
  const int t = threadIdx.x;
  if (t >= MR * COLS) return;
  const int i = t / COLS, c = t % COLS;
  const int m = m0 + i, n = n0 + c;
  if (m >= a.M || n >= a.N) return;
  int sum = 0;
#pragma unroll
  for (int q = 0; q < KW; ++q) sum += part[c / R * KW + q][i * R + c % R];
  const float v = s8_scaled<true>(sum, a.sA[m], a.sB[n], a.bias != nullptr ? a.bias[n] : 0.0f);
  const size_t at = (size_t)m * a.ldc + n;
  if (a.type == kTypeF32) s8_finish_one(a, static_cast<float *>(a.C) + at, v);
  else if (a.type == kTypeF16) s8_finish_one(a, static_cast<_Float16 *>(a.C) + at, v);
  else s8_finish_one(a, static_cast<__bf16 *>(a.C) + at, v);
}

template <int MR, int R, int KW> hipError_t launch(const S8Args &a, hipStream_t s) {
  constexpr int COLS = kWaves / KW * R;
  s8_gemv_kernel<MR, R, KW>
      <<<dim3((a.N + COLS - 1) / COLS, (a.M + MR - 1) / MR), 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}

template <int R, int KW> hipError_t by_rows(const S8Args &a, hipStream_t s) {
  if (a.M == 1) return launch<1, R, KW>(a, s);
  if (a.M == 2) return launch<2, R, KW>(a, s);
  return launch<4, R, KW>(a, s);
}

}  // namespace

hipError_t launch_s8_gemv_r2(const S8Args &a, hipStream_t s) { return by_rows<2, 1>(a, s); }
hipError_t launch_s8_gemv_r2k4(const S8Args &a, hipStream_t s) { return by_rows<2, 4>(a, s); }

}  // namespace fp32gemm
