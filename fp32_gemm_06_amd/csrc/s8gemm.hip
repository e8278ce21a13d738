// The 8-bit product's kernels, their choice by shape, and the launch.
#include <math.h>

#include "s8_kernel.h"

namespace fp32gemm {
namespace {

// Rows of one launch: keeps the grid's threads below 2^32 for any M.
constexpr int kMaxLaunchRows = 1 << 22;

// A configuration, and its time on a shape in microseconds (M, N large against
// the tile):  fixed + each * rounds + (first + more * (rounds - 1)) * K / 1000,
// rounds = the tiles that a CU gets, ceil(tiles / 256).
struct S8Config {
  const char *name;
  int BM, BN;
  float fixed, each, first, more;
  hipError_t (*launch)(const S8Args &, hipStream_t);
};

// BMxBN_kKS_sNST: KS slices of K a stage, NST stages in LDS.  The small tiles
// split K over their waves and fill the CUs for few rows or columns; the
// large ones move fewer bytes for each product.  The four numbers are fitted
// to each configuration's times over 508 shapes (M 1 .. 4096, N 64 .. 11008,
// K 128 .. 11008, bf16 out), and the shortest fitted time chosen: over those
// shapes it is 2.8% above the best of them (geometric mean; 64x64_k1_s4 alone
// 42%).
#define S8_TILE(name, BM, BN, WM, WN, KS, NST, ...) \
  {name, BM, BN, __VA_ARGS__, s8_launch<S8Tile<BM, BN, WM, WN, KS, NST>>}
const S8Config kConfigs[] = {
    S8_TILE("16x16_k8_s4", 16, 16, 16, 16, 8, 4, 1.80f, 2.19f, 0.32f, 0.33f),
    S8_TILE("16x16_k4_s4", 16, 16, 16, 16, 4, 4, 2.45f, 0.97f, 0.40f, 0.29f),
    S8_TILE("16x32_k4_s4", 16, 32, 16, 32, 4, 4, 1.82f, 2.12f, 0.51f, 0.55f),
    S8_TILE("32x32_k4_s4", 32, 32, 32, 32, 4, 4, 2.24f, 2.79f, 0.58f, 0.73f),
    S8_TILE("64x32_k4_s3", 64, 32, 64, 32, 4, 3, 1.63f, 4.53f, 0.92f, 1.11f),
    S8_TILE("64x64_k2_s4", 64, 64, 32, 32, 2, 4, 1.65f, 3.58f, 1.33f, 1.72f),
    S8_TILE("64x64_k1_s4", 64, 64, 32, 32, 1, 4, 3.05f, 1.43f, 2.06f, 1.50f),
    S8_TILE("128x64_k2_s3", 128, 64, 64, 32, 2, 3, 1.25f, 5.01f, 2.22f, 2.76f),
    S8_TILE("128x128_k1_s4", 128, 128, 64, 32, 1, 4, 0.65f, 5.11f, 3.27f, 4.51f),
    S8_TILE("256x128_k1_s3", 256, 128, 64, 64, 1, 3, 0.03f, 6.76f, 5.41f, 7.42f),
    S8_TILE("256x256_k1_s2", 256, 256, 128, 64, 1, 2, 0.00f, 9.01f, 9.40f, 15.11f),
};
#undef S8_TILE
constexpr int kNumConfigs = sizeof(kConfigs) / sizeof(kConfigs[0]);

int pick(int M, int N, int K) {
  int best = 0;
  float least = 0.0f;
  for (int c = 0; c < kNumConfigs; ++c) {
    const S8Config &f = kConfigs[c];
    const float tiles = (float)((M + f.BM - 1) / f.BM) * (float)((N + f.BN - 1) / f.BN);
    const float rounds = ceilf(tiles / 256.0f);
    const float t = f.fixed + f.each * rounds + (f.first + f.more * (rounds - 1.0f)) * K * 1e-3f;
    if (c == 0 || t < least) {
      best = c;
      least = t;
    }
  }
  return best;
}

__global__ void s8_epilogue_kernel(S8Args a) {
  const long long n = (long long)a.M * a.N;
  for (long long f = blockIdx.x * (long long)blockDim.x + threadIdx.x; f < n;
       f += (long long)gridDim.x * blockDim.x) {
    const size_t i = f / a.N, j = f % a.N;
    const size_t at = i * a.ldc + j;
    auto put = [&](auto *c) {
      float v = 0.0f;
      if (a.beta != 0.0f) v = a.beta * (float)c[at];
      if (a.bias != nullptr) v += a.bias[j];
      c[at] = (std::remove_reference_t<decltype(c[at])>)apply_act(v, a.act);
    };
    if (a.type == kTypeF32) put(static_cast<float *>(a.C));
    else if (a.type == kTypeF16) put(static_cast<_Float16 *>(a.C));
    else put(static_cast<__bf16 *>(a.C));
  }
}

}  // namespace

int s8_num_configs() { return kNumConfigs; }
const char *s8_config_name(int cfg) {
  return cfg >= 0 && cfg < s8_num_configs() ? kConfigs[cfg].name : nullptr;
}
int select_s8_config(int M, int N, int K) { return pick(M > 0 ? M : 1, N > 0 ? N : 1, K > 0 ? K : 1); }

hipError_t launch_s8(int cfg, const S8Args &a, hipStream_t s) {
  if (cfg < 0) cfg = pick(a.M, a.N, a.K);
  const size_t size = a.type == kTypeF32 ? 4 : 2;
  for (int m0 = 0; m0 < a.M; m0 += kMaxLaunchRows) {
    S8Args b = a;
    b.M = a.M - m0 < kMaxLaunchRows ? a.M - m0 : kMaxLaunchRows;
    b.A = a.A + (size_t)m0 * a.lda;
    b.sA = a.sA + m0;
    b.C = static_cast<char *>(a.C) + (size_t)m0 * a.ldc * size;
    const hipError_t e = kConfigs[cfg].launch(b, s);
    if (e != hipSuccess) return e;
    if (b.M == a.M - m0) break;  // m0 + the step may pass the int range
  }
  return hipSuccess;
}

hipError_t launch_s8_epilogue_only(const S8Args &a, hipStream_t s) {
  const long long n = (long long)a.M * a.N;
  const long long groups = (n + 255) / 256;
  s8_epilogue_kernel<<<(int)(groups < 4096 ? groups : 4096), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace fp32gemm
