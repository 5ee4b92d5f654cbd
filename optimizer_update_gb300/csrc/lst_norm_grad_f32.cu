// The backward kernel of the residual norm for fp32 activations.
#include "lst_norm_grad.cuh"

namespace lst {

NormKernel<GradArgs> norm_grad_f32(bool vec, int k) {
  if (vec) return k == 4 ? norm_grad_kernel<float, true, 4, false> : norm_grad_kernel<float, true, 2, true>;
  return k == 4 ? norm_grad_kernel<float, false, 4, false> : k == 2 ? norm_grad_kernel<float, false, 2, true> : norm_grad_kernel<float, false, 1, true>;
}

cudaError_t norm_grad_f32_take_error(int* out) { return take_norm_error(out); }

}  // namespace lst
