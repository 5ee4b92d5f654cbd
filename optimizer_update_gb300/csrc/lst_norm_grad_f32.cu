// The backward kernel of the residual norm for fp32 activations.
#include "lst_norm_grad.cuh"

namespace lst {

namespace {
template <bool ONE>
NormKernel<GradArgs> rows_kernel(int form) {
  switch (form) {
    case 1: return norm_grad_rows_kernel<float, 0, true, ONE>;
    case 2: return norm_grad_rows_kernel<float, 1, true, ONE>;
    case 3: return norm_grad_rows_kernel<float, 2, true, ONE>;
    case 4: return norm_grad_rows_kernel<float, 0, false, ONE>;
    case 5: return norm_grad_rows_kernel<float, 1, false, ONE>;
    default: return norm_grad_rows_kernel<float, 2, false, ONE>;
  }
}
}  // namespace

NormKernel<GradArgs> norm_grad_f32(bool vec, int k, int form, bool one) {
  if (vec && k == 2 && form) return one ? rows_kernel<true>(form) : rows_kernel<false>(form);
  if (vec) return k == 4 ? norm_grad_kernel<float, true, 4, false> : norm_grad_kernel<float, true, 2, true>;
  return k == 4 ? norm_grad_kernel<float, false, 4, false> : k == 2 ? norm_grad_kernel<float, false, 2, true> : norm_grad_kernel<float, false, 1, true>;
}

cudaError_t norm_grad_f32_take_error(int* out) { return take_norm_error(out); }

}  // namespace lst
