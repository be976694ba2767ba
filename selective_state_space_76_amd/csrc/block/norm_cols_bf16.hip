// norm_cols_bf16.hip -- norm_cols_kernel.h for x in bf16, hidden in bf16.
#include "norm_cols_kernel.h"

namespace ssm {

hipError_t launch_norm_cols_bf16(const NormParams& p, hipStream_t s) {
  p.residual ? fwd<bf16_t, bf16_t, true>(p, s) : fwd<bf16_t, bf16_t, false>(p, s);
  return hipGetLastError();
}

hipError_t launch_norm_cols_bwd_bf16(const NormParams& p, hipStream_t s) {
  bwd<bf16_t, bf16_t>(p, s);
  return hipGetLastError();
}

}  // namespace ssm
