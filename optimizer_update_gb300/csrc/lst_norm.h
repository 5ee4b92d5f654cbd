// Internal interface of the residual-norm kernels (lst_norm.cu).
#pragma once

#include <cuda_runtime.h>

namespace lst {

// Whether some wait of the backward kernel ran out since the last call on this
// device (synchronises the device).
cudaError_t norm_take_error(int* out);

}  // namespace lst
