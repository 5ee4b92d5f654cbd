// The backward kernel of the residual norm for fp32 activations.
#include "lst_norm_grad.cuh"

namespace lst {

NormKernel<GradArgs> norm_grad_f32(bool vec, bool wide) {
  if (vec) return wide ? norm_grad_kernel<float, true, 4, false> : norm_grad_kernel<float, true, 2, true>;
  return wide ? norm_grad_kernel<float, false, 4, false> : norm_grad_kernel<float, false, 2, true>;
}

cudaError_t norm_grad_f32_take_error(int* out) { return take_norm_error(out); }

}  // namespace lst
