// The backward kernel of the residual norm for bf16 activations.
#include "lst_norm_grad.cuh"

namespace lst {

NormKernel<GradArgs> norm_grad_bf16(bool vec, bool wide, int form) {
  if (vec && !wide) {
    switch (form) {
      case 1: return norm_grad_kernel<__nv_bfloat16, true, 2, true, 1>;
      case 2: return norm_grad_kernel<__nv_bfloat16, true, 2, true, 2>;
      case 3: return norm_grad_kernel<__nv_bfloat16, true, 2, true, 3>;
      case 4: return norm_grad_kernel<__nv_bfloat16, true, 2, true, 4>;
      case 5: return norm_grad_kernel<__nv_bfloat16, true, 2, true, 5>;
      case 6: return norm_grad_kernel<__nv_bfloat16, true, 2, true, 6>;
    }
  }
  if (vec) return wide ? norm_grad_kernel<__nv_bfloat16, true, 4, false, 0> : norm_grad_kernel<__nv_bfloat16, true, 2, true, 0>;
  return wide ? norm_grad_kernel<__nv_bfloat16, false, 4, false, 0> : norm_grad_kernel<__nv_bfloat16, false, 2, true, 0>;
}

cudaError_t norm_grad_bf16_take_error(int* out) { return take_norm_error(out); }

}  // namespace lst
