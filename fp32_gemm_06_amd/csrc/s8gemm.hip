// The 8-bit product's kernels, their choice by shape, and the launch.
#include <limits.h>

#include "s8_kernel.h"

namespace fp32gemm {
namespace {

// Rows of one launch: keeps the grid's threads below 2^32 for any M.
constexpr int kMaxLaunchRows = 1 << 22;

struct S8Config {
  const char *name;
  int max_rows;
  hipError_t (*launch)(const S8Args &, hipStream_t);
};

#define S8_TILE(name, ...) {name, INT_MAX, s8_launch<S8Tile<__VA_ARGS__>>}
const S8Config kConfigs[] = {
    S8_TILE("16x16_k8_s4", 16, 16, 16, 16, 16, 8, 4),
    S8_TILE("16x16_k4_s4", 16, 16, 16, 16, 16, 4, 4),
    S8_TILE("16x32_k8_s3", 16, 32, 16, 32, 16, 8, 3),
    S8_TILE("16x32_k4_s4", 16, 32, 16, 32, 16, 4, 4),
    S8_TILE("16x64_k4_s3", 16, 64, 16, 64, 16, 4, 3),
    S8_TILE("32x16_k8_s3", 32, 16, 32, 16, 16, 8, 3),
    S8_TILE("32x32_k4_s4", 32, 32, 32, 32, 16, 4, 4),
    S8_TILE("32x32_k8_s2", 32, 32, 32, 32, 16, 8, 2),
    S8_TILE("32x64_k4_s3", 32, 64, 32, 64, 16, 4, 3),
    S8_TILE("64x16_k4_s3", 64, 16, 64, 16, 16, 4, 3),
    S8_TILE("64x32_k4_s3", 64, 32, 64, 32, 16, 4, 3),
    S8_TILE("64x64_k2_s4", 64, 64, 32, 32, 16, 2, 4),
    S8_TILE("64x64_k4o_s2", 64, 64, 64, 64, 16, 4, 2),
    S8_TILE("64x64_k1_s4", 64, 64, 32, 32, 16, 1, 4),
    S8_TILE("128x64_k1_s4", 128, 64, 64, 32, 16, 1, 4),
    S8_TILE("128x64_k2_s3", 128, 64, 64, 32, 16, 2, 3),
    S8_TILE("128x128_w64x64_s2", 128, 128, 64, 64, 16, 1, 2),
    S8_TILE("128x128_w64x64_s4", 128, 128, 64, 64, 16, 1, 4),
    S8_TILE("128x128_w64x32_s4", 128, 128, 64, 32, 16, 1, 4),
    S8_TILE("128x256_w64x64_s3", 128, 256, 64, 64, 16, 1, 3),
    S8_TILE("256x128_w64x64_s3", 256, 128, 64, 64, 16, 1, 3),
    S8_TILE("256x256_w128x64_s2", 256, 256, 128, 64, 16, 1, 2),
    {"skinny16", kS8SkinnyRows, launch_s8_skinny16},
};

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

int pick(int M, int N, int K) {
  (void)N;
  (void)K;
  return M <= 128 ? 1 : M <= 256 ? 11 : 21;
}

}  // namespace

int s8_num_configs() { return (int)(sizeof(kConfigs) / sizeof(kConfigs[0])); }
const char *s8_config_name(int cfg) {
  return cfg >= 0 && cfg < s8_num_configs() ? kConfigs[cfg].name : nullptr;
}
int s8_config_max_rows(int cfg) {
  return cfg >= 0 && cfg < s8_num_configs() ? kConfigs[cfg].max_rows : -1;
}
int select_s8_config(int M, int N, int K) { return pick(M, N, K); }

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
