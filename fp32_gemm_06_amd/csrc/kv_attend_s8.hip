// Attention over a cache of 8-bit codes.
#include "kv_attend_kernel.h"

namespace fp32gemm {
hipError_t launch_attend_s8(const AttendArgs &a, int type, hipStream_t s) {
  if (type == kTypeF32) return launch_attend<float, true>(a, s);
  if (type == kTypeF16) return launch_attend<_Float16, true>(a, s);
  return launch_attend<__bf16, true>(a, s);
}
}  // namespace fp32gemm
