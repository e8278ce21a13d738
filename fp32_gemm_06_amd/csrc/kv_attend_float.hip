// Attention over a cache in the operands' own type.
#include "kv_attend_kernel.h"

namespace fp32gemm {
hipError_t launch_attend_float(const AttendArgs &a, int type, hipStream_t s) {
  if (type == kTypeF32) return launch_attend<float, false>(a, s);
  if (type == kTypeF16) return launch_attend<_Float16, false>(a, s);
  return launch_attend<__bf16, false>(a, s);
}
}  // namespace fp32gemm
