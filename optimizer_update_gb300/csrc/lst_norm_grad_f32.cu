// The backward kernel of the residual norm for fp32 activations.
#include "lst_norm_grad.cuh"
#include "lst_norm_split.cuh"

namespace lst {

namespace {
template <int BLOCK, bool ONE>
NormKernel<GradArgs> rows_kernel(int kept) {
  return kept == 0   ? norm_grad_rows_kernel<float, 0, BLOCK, ONE>
         : kept == 1 ? norm_grad_rows_kernel<float, 1, BLOCK, ONE>
                     : norm_grad_rows_kernel<float, 2, BLOCK, ONE>;
}
template <bool ONE>
NormKernel<GradArgs> rows_kernel(int block, int kept) {
  return block == 0 ? rows_kernel<0, ONE>(kept) : block == 1 ? rows_kernel<1, ONE>(kept) : rows_kernel<2, ONE>(kept);
}
}  // namespace

NormKernel<GradArgs> norm_grad_f32(bool vec, int k, int form, bool one) {
  if (form) return one ? rows_kernel<true>((form - 1) / 3, (form - 1) % 3) : rows_kernel<false>((form - 1) / 3, (form - 1) % 3);
  if (vec) return norm_grad_kernel<float, true, 2>;
  return k == 2 ? norm_grad_kernel<float, false, 2> : norm_grad_kernel<float, false, 1>;
}

SplitKernels norm_split_f32(bool vec) {
  return vec ? SplitKernels{norm_stats_kernel<float, true>, norm_apply_kernel<float, true>}
             : SplitKernels{norm_stats_kernel<float, false>, norm_apply_kernel<float, false>};
}

cudaError_t norm_grad_f32_take_error(int* out) { return take_norm_error(out); }

}  // namespace lst
