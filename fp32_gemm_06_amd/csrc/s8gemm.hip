// The 8-bit product's kernels, their choice by shape, and the launch.
#include <math.h>

#include "s8_kernel.h"

namespace fp32gemm {
namespace {

// Tiles of one launch: keeps the grid's threads below 2^32.
constexpr long long kMaxLaunchTiles = 1 << 21;

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

// gemv_rR: dot products, R rows of W a wave (kKW: KW waves split K).
// BMxBN_kKS_sNST: KS slices of K a stage, NST stages in LDS.  The small tiles
// split K over their waves and fill the CUs for few rows or columns; the
// large ones move fewer bytes for each product.  Sixteen waves where a CU
// holds one workgroup: a wave's loads reach LDS at 8 to 13 bytes/ns, and more
// waves move more (256 x 128 tiles, 1536 x 4096 x 4096: 31.8 us with 16
// waves, 35.7 with 8).  The five numbers are fitted to each configuration's
// times on 6831 shapes (M 1 .. 4096, N and K 64 .. 11008, most of them drawn,
// bf16 out) and 1722 large ones, with three copies of the operands in turn, so
// that a small W comes from the last-level cache.  The shortest fitted time is
// chosen: 2.1% above the best of the sixteen (geometric mean; at most 50%),
// 0.4% on the shapes that take 20 us or more and 0.3% on the large ones.
// 64x64_k1_s4, the best one by itself, is 40% above.  On rows without
// alignment (4618 shapes) the same choice is 3.5% and 1.2% above (at most 78%),
// with W from memory (1 to 16 rows, N to 128256, K to 28672) 3% (at most 37%,
// four rows of a wide W with a short K).  Beyond those sizes it is
// extrapolated.
#define S8_TILE(name, BM, BN, WM, WN, KS, NST, AHEAD, ...) \
  {name, BM, BN, __VA_ARGS__,                                               \
   s8_launch<S8Tile<BM, BN, WM, WN, KS, NST, AHEAD>, S8Tile<BM, BN, WM, WN, KS, NST, AHEAD>>}
const S8Config kConfigs[] = {
    {"gemv_r2", 4, 8, 3.03f, 0.00f, 0.23f, 0.09f, 0.27f, launch_s8_gemv_r2},
    {"gemv_r2k4", 4, 2, 3.34f, 0.11f, 0.03f, 0.00f, 0.06f, launch_s8_gemv_r2k4},
    S8_TILE("16x16_k8_s4", 16, 16, 16, 16, 8, 4, true, 3.43f, 1.35f, 0.09f, 0.25f, 0.54f),
    S8_TILE("16x16_k4_s4", 16, 16, 16, 16, 4, 4, true, 2.91f, 0.83f, 0.28f, 0.20f, 0.35f),
    S8_TILE("16x32_k4_s4", 16, 32, 16, 32, 4, 4, true, 2.80f, 1.60f, 0.31f, 0.48f, 0.62f),
    S8_TILE("32x32_k4_s4", 32, 32, 32, 32, 4, 4, true, 2.49f, 2.29f, 0.43f, 0.44f, 0.81f),
    S8_TILE("64x32_k4_s3", 64, 32, 32, 32, 4, 3, true, 1.90f, 3.10f, 0.84f, 0.32f, 1.18f),
    S8_TILE("64x64_k2_s4", 64, 64, 16, 32, 2, 4, true, 2.06f, 2.86f, 1.04f, 0.57f, 1.54f),
    S8_TILE("64x64_k1_s4", 64, 64, 16, 32, 1, 4, true, 3.57f, 1.01f, 1.20f, 0.55f, 1.52f),
    S8_TILE("96x64_k2_s3", 96, 64, 48, 32, 2, 3, true, 0.48f, 4.54f, 1.60f, 0.67f, 2.02f),
    S8_TILE("128x64_k1_s3", 128, 64, 32, 32, 1, 3, true, 3.23f, 1.40f, 1.74f, 0.93f, 2.17f),
    S8_TILE("128x128_k1_s4", 128, 128, 32, 32, 1, 4, true, 0.92f, 4.18f, 2.05f, 2.03f, 3.75f),
    S8_TILE("192x128_k1_s2", 192, 128, 96, 32, 1, 2, false, 1.19f, 3.44f, 5.52f, 1.44f, 3.99f),
    S8_TILE("256x128_k1_s3", 256, 128, 64, 32, 1, 3, true, 0.00f, 5.75f, 3.73f, 3.05f, 6.18f),
    S8_TILE("256x192_k1_s2", 256, 192, 64, 96, 1, 2, false, 0.36f, 7.13f, 7.28f, 3.12f, 9.02f),
    // 16 waves have no registers left for the path through them
    {"256x256_k1_s2", 256, 256, 0.00f, 7.67f, 7.83f, 4.90f, 10.44f,
     s8_launch<S8Tile<256, 256, 64, 64, 1, 2, false>, S8Tile<256, 256, 64, 128, 1, 2, true>>},
};
#undef S8_TILE
constexpr int kNumConfigs = sizeof(kConfigs) / sizeof(kConfigs[0]);

// Where the fitted times decide between the dot products and the tiles, and
// where they do not.  They come from N and K up to 11008 with W's codes in the
// last-level cache, and what they say of few rows fails outside that: a round
// of dot products costs nothing in them (gemv_r2's `each`), wide weights put one
// row on 64 x 64 tiles.  So, measured with W from memory too:
//   1 and 2 rows are dot products (1 x 32000 x 4096: 20.9 us, the best tiles
//   30.6; 1 x 16384 x 4096 12.0 and 17.4; 1 x 28672 x 8192 36.4 and 43.6; over
//   the 1981 fitted shapes of one and two rows the quicker dot products are 0.3
//   to 0.9% above the best, the quickest tiles 8 to 16%);
//   3 and 4 are either, by the fitted times, which are not always right (4 x
//   11008 x 4096 11.6 and 13.4; 4 x 28672 x 8192 51.3 and 43.9; 4 x 32000 x 4096
//   26.8 and 30.7, and tiles are chosen);
//   5 to 8 read W twice, and are either up to this N (8 x 131 x 10653 4.5 and
//   6.6), tiles above (8 x 10931 x 443 10.2 and 5.2; 8 x 28672 x 8192 83.5 and
//   44.3);
//   from 9 rows on the tiles are always the quicker.
constexpr int kGemvRows = 4, kGemvTwiceN = 2048;
bool stands(bool dots, int M, int N) {
  if (dots) return M <= kGemvRows || (M <= 2 * kGemvRows && N <= kGemvTwiceN);
  return M > 2;
}

int pick(int M, int N, int K) {
  int best = -1;
  float least = 0.0f;
  for (int c = 0; c < kNumConfigs; ++c) {
    const S8Config &f = kConfigs[c];
    if (!stands(f.BM == kGemvRows, M, N)) continue;
    const float tiles = (float)((M - 1) / f.BM + 1) * (float)((N - 1) / f.BN + 1);
    const float rounds = ceilf(tiles / 256.0f), fill = tiles / (256.0f * rounds);
    const float t = f.fixed + f.each * rounds +
                    (f.first + f.full * fill + f.more * (rounds - 1.0f)) * (float)K * 1e-3f;
    if (best < 0 || t < least) {
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
  const S8Config &c = kConfigs[cfg];
  const size_t size = a.type == kTypeF32 ? 4 : 2;
  const long long across = (a.N + c.BN - 1) / c.BN;
  long long down = kMaxLaunchTiles / across;  // at least 4: N is at most 2^20
  if (c.BM == kGemvRows && down > 65535) down = 65535;  // rows are their grid's second dimension
  for (long long m0 = 0; m0 < a.M; m0 += down * c.BM) {
    S8Args b = a;
    b.M = (int)(a.M - m0 < down * c.BM ? a.M - m0 : down * c.BM);
    b.A = a.A + m0 * a.lda;
    b.sA = a.sA + m0;
    b.C = static_cast<char *>(a.C) + (size_t)m0 * a.ldc * size;
    const hipError_t e = c.launch(b, s);
    if (e != hipSuccess) return e;
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
