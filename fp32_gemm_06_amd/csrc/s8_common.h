// Declarations of the 8-bit linear layer: the integer product s8gemm and the
// operators that make its codes, s8_quantize and s8_rmsnorm.
#pragma once

#include "common.h"

namespace fp32gemm {

typedef int intx4 __attribute__((ext_vector_type(4)));

// Element types of the float operands (the header's FP32GEMM_TYPE_*).
constexpr int kTypeF32 = 0, kTypeF16 = 1, kTypeBf16 = 2;

// One C <- act(sA sB (A B^T) + beta C + bias) call, already validated: A is
// M x K, B is N x K, both 8-bit codes with k contiguous.
struct S8Args {
  int M, N, K;
  const int8_t *A;
  const int8_t *B;
  const float *sA;
  const float *sB;
  float beta;
  int type;  // of C
  void *C;
  int lda, ldb, ldc;
  const float *bias;  // NULL: none
  int act;
};

// The product (s8gemm.hip), with the configuration that suits the shape
// (cfg < 0) or the one asked for.
hipError_t launch_s8(int cfg, const S8Args &a, hipStream_t s);
int s8_num_configs();
const char *s8_config_name(int cfg);
int select_s8_config(int M, int N, int K);

// Dot products for few rows (s8_gemv.hip).
hipError_t launch_s8_gemv_r2(const S8Args &a, hipStream_t s);
hipError_t launch_s8_gemv_r2k4(const S8Args &a, hipStream_t s);

// C <- act(beta C + bias): the product over an empty K.
hipError_t launch_s8_epilogue_only(const S8Args &a, hipStream_t s);

// One s8_quantize or s8_rmsnorm call, already validated.
struct S8RowArgs {
  int M, K;
  const void *X;
  int ldx;
  const void *R;  // NULL: no residual
  int ldr;
  void *H;  // NULL: the sum is not stored
  int ldh;
  const void *W;  // NULL: quantize, no norm
  float eps;
  int8_t *Q;
  int ldq;
  float *scales;
};

hipError_t launch_s8_rows(const S8RowArgs &a, int type, hipStream_t s);
// X stored K x M, the codes of its columns.
hipError_t launch_s8_columns(const S8RowArgs &a, int type, hipStream_t s);

// ---- float types ------------------------------------------------------------
template <int TYPE> struct FloatOf { typedef float type; };
template <> struct FloatOf<kTypeF16> { typedef _Float16 type; };
template <> struct FloatOf<kTypeBf16> { typedef __bf16 type; };

// ---- codes ------------------------------------------------------------------
// A row's largest magnitude travels as the bits of |v|: they order as the
// magnitudes do, with infinity and then every NaN above the finite values.
constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu;
}

// What a row's codes are computed from.  step = fl32(top / 127).  Steps
// below 2^-60 and the values with them are taken times 2^80, which is exact
// and keeps 1 / step and the residual below out of the subnormal range; a row
// without codes (all zero, a step that underflows to zero, or a value that
// is not finite) has step 0 here, which code() maps to 0.
struct RowStep {
  float step, inv, lift;
};

__device__ __forceinline__ RowStep row_step(float scale) {
  RowStep r;
  const bool none = !(scale > 0.0f) || !(scale < __builtin_inff());
  r.lift = scale < 0x1p-60f ? 0x1p80f : 1.0f;
  r.step = none ? 0.0f : scale * r.lift;
  r.inv = none ? 0.0f : 1.0f / r.step;
  return r;
}

// The scale of a row whose largest magnitude has these bits: fl32(top / 127),
// NaN when the row holds an infinity or a NaN (its codes are zero, and
// whatever is multiplied by that scale shows it).
__device__ __forceinline__ float row_scale(uint32_t top) {
  return top >= kInfBits ? __builtin_nanf("") : __builtin_bit_cast(float, top) / 127.0f;
}

// round(v / step), halves to even, as if the quotient were exact.  v * inv is
// within 3e-5 of it, so its nearest integer q is wrong only next to a half;
// the residual v - q step is exact there (a multiple of half an ulp of step
// below 2^24 of them), and says on which side of the half v lies.
__device__ __forceinline__ int row_code(float v, const RowStep &r) {
  const float x = v * r.lift;
  const float q = __builtin_rintf(x * r.inv);
  const float e = 2.0f * __builtin_fmaf(-q, r.step, x);
  const float m = __builtin_fabsf(e);
  const int qi = (int)q;
  const bool off = m > r.step || (m == r.step && (qi & 1));
  const int c = qi + (off ? (e > 0.0f ? 1 : -1) : 0);
  return r.step > 0.0f ? (c > 127 ? 127 : c < -127 ? -127 : c) : 0;
}

}  // namespace fp32gemm
