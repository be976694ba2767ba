// norm_cols_mixed.hip -- norm_cols_kernel.h for x in bf16, hidden in fp32.
#include "norm_cols_kernel.h"

namespace ssm {

hipError_t launch_norm_cols_mixed(const NormParams& p, hipStream_t s) {
  p.residual ? fwd<bf16_t, float, true>(p, s) : fwd<bf16_t, float, false>(p, s);
  return hipGetLastError();
}

hipError_t launch_norm_cols_bwd_mixed(const NormParams& p, hipStream_t s) {
  bwd<bf16_t, float>(p, s);
  return hipGetLastError();
}

}  // namespace ssm
