// The backward kernel of the residual norm for bf16 activations.
#include "lst_norm_grad.cuh"

namespace lst {

namespace {
template <int BLOCK, bool ONE>
NormKernel<GradArgs> rows_kernel(int kept) {
  return kept == 0   ? norm_grad_rows_kernel<__nv_bfloat16, 0, BLOCK, ONE>
         : kept == 1 ? norm_grad_rows_kernel<__nv_bfloat16, 1, BLOCK, ONE>
                     : norm_grad_rows_kernel<__nv_bfloat16, 2, BLOCK, ONE>;
}
template <bool ONE>
NormKernel<GradArgs> rows_kernel(int block, int kept) {
  return block == 0 ? rows_kernel<0, ONE>(kept) : block == 1 ? rows_kernel<1, ONE>(kept) : rows_kernel<2, ONE>(kept);
}
}  // namespace

NormKernel<GradArgs> norm_grad_bf16(bool vec, int k, int form, bool one) {
  if (vec && k == 2 && form) return one ? rows_kernel<true>((form - 1) / 3, (form - 1) % 3) : rows_kernel<false>((form - 1) / 3, (form - 1) % 3);
  if (vec) return k == 4 ? norm_grad_kernel<__nv_bfloat16, true, 4, false> : norm_grad_kernel<__nv_bfloat16, true, 2, true>;
  return k == 4 ? norm_grad_kernel<__nv_bfloat16, false, 4, false> : k == 2 ? norm_grad_kernel<__nv_bfloat16, false, 2, true> : norm_grad_kernel<__nv_bfloat16, false, 1, true>;
}

cudaError_t norm_grad_bf16_take_error(int* out) { return take_norm_error(out); }

}  // namespace lst
