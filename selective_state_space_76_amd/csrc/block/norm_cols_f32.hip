// norm_cols_f32.hip -- norm_cols_kernel.h for x in fp32, hidden in fp32.
#include "norm_cols_kernel.h"

namespace ssm {

hipError_t launch_norm_cols_f32(const NormParams& p, hipStream_t s) {
  p.residual ? fwd<float, float, true>(p, s) : fwd<float, float, false>(p, s);
  return hipGetLastError();
}

hipError_t launch_norm_cols_bwd_f32(const NormParams& p, hipStream_t s) {
  bwd<float, float>(p, s);
  return hipGetLastError();
}

}  // namespace ssm
