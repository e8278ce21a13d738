// The 8-bit product's kernels, their choice by shape, and the launch.
#include <math.h>

#include "s8_kernel.h"

namespace fp32gemm {
namespace {

// Rows of one launch: keeps the grid's threads below 2^32 for any M.
constexpr int kMaxLaunchRows = 1 << 22;

// A configuration, and its time on a shape in microseconds:
//   each * rounds + fixed + (first + full * fill + more * (rounds - 1)) K / 1000
// with rounds = ceil(tiles / 256), the tiles that a CU gets, and fill = the
// share of those places that have one (a full chip shares L2 and power).
struct S8Config {
  const char *name;
  int BM, BN;
  float fixed, each, first, full, more;
  hipError_t (*launch)(const S8Args &, hipStream_t);
};

// BMxBN_kKS_sNST: KS slices of K a stage, NST stages in LDS.  The small tiles
// split K over their waves and fill the CUs for few rows or columns; the
// large ones move fewer bytes for each product.  Sixteen waves where a CU
// holds one workgroup: a wave's loads reach LDS at 8 to 13 bytes/ns, and more
// waves move more (256 x 128 tiles, 1536 x 4096 x 4096: 31.8 us with 16
// waves, 35.7 with 8).  The five numbers are fitted to each configuration's
// times on 4339 shapes (M 1 .. 4096, N and K 64 .. 11008, most of them drawn,
// bf16 out), and the shortest fitted time is chosen: 1.5% above the best of
// the fourteen (geometric mean), 0.8% on the shapes that take 20 us or more.
// 64x64_k1_s4, the best one by itself, is 31% above.  On rows without
// alignment (1902 shapes) the same choice is 5% above.
#define S8_TILE(name, BM, BN, WM, WN, KS, NST, AHEAD, ...) \
  {name, BM, BN, __VA_ARGS__,                                               \
   s8_launch<S8Tile<BM, BN, WM, WN, KS, NST, AHEAD>, S8Tile<BM, BN, WM, WN, KS, NST, AHEAD>>}
const S8Config kConfigs[] = {
    S8_TILE("16x16_k8_s4", 16, 16, 16, 16, 8, 4, true, 3.65f, 1.46f, 0.09f, 0.22f, 0.49f),
    S8_TILE("16x16_k4_s4", 16, 16, 16, 16, 4, 4, true, 4.58f, 0.43f, 0.14f, 0.14f, 0.39f),
    S8_TILE("16x32_k4_s4", 16, 32, 16, 32, 4, 4, true, 3.40f, 1.66f, 0.28f, 0.31f, 0.63f),
    S8_TILE("32x32_k4_s4", 32, 32, 32, 32, 4, 4, true, 2.55f, 2.68f, 0.44f, 0.40f, 0.77f),
    S8_TILE("64x32_k4_s3", 64, 32, 32, 32, 4, 3, true, 1.90f, 3.65f, 0.82f, 0.39f, 1.15f),
    S8_TILE("64x64_k2_s4", 64, 64, 16, 32, 2, 4, true, 1.76f, 3.61f, 1.16f, 0.64f, 1.64f),
    S8_TILE("64x64_k1_s4", 64, 64, 16, 32, 1, 4, true, 3.50f, 1.37f, 1.39f, 0.55f, 1.41f),
    S8_TILE("96x64_k2_s3", 96, 64, 48, 32, 2, 3, true, 0.77f, 4.98f, 1.66f, 0.61f, 1.99f),
    S8_TILE("128x64_k1_s3", 128, 64, 32, 32, 1, 3, true, 2.93f, 2.11f, 1.85f, 0.97f, 2.01f),
    S8_TILE("128x128_k1_s4", 128, 128, 32, 32, 1, 4, true, 0.00f, 5.65f, 2.32f, 2.23f, 3.55f),
    S8_TILE("192x128_k1_s2", 192, 128, 96, 32, 1, 2, false, 0.28f, 5.07f, 4.93f, 2.94f, 3.14f),
    S8_TILE("256x128_k1_s3", 256, 128, 64, 32, 1, 3, true, 0.00f, 6.13f, 3.94f, 3.39f, 6.64f),
    S8_TILE("256x192_k1_s2", 256, 192, 64, 96, 1, 2, false, 0.00f, 7.47f, 7.80f, 3.96f, 10.63f),
    // 16 waves have no registers left for the path through them
    {"256x256_k1_s2", 256, 256, 0.00f, 6.82f, 8.54f, 6.08f, 12.60f,
     s8_launch<S8Tile<256, 256, 64, 64, 1, 2, false>, S8Tile<256, 256, 64, 128, 1, 2, true>>},
};
#undef S8_TILE
constexpr int kNumConfigs = sizeof(kConfigs) / sizeof(kConfigs[0]);

int pick(int M, int N, int K) {
  int best = 0;
  float least = 0.0f;
  for (int c = 0; c < kNumConfigs; ++c) {
    const S8Config &f = kConfigs[c];
    const float tiles = (float)((M + f.BM - 1) / f.BM) * (float)((N + f.BN - 1) / f.BN);
    const float rounds = ceilf(tiles / 256.0f), fill = tiles / (256.0f * rounds);
    const float t = f.fixed + f.each * rounds +
                    (f.first + f.full * fill + f.more * (rounds - 1.0f)) * (float)K * 1e-3f;
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
