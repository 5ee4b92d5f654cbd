// Internal interface of the residual-norm kernels (lst_norm.cu).
#pragma once

#include <cuda_runtime.h>

namespace lst {

// Whether some wait of the residual-norm kernels, forward or backward, ran out since
// the last call on this device (synchronises the device).
cudaError_t norm_take_error(int* out);

}  // namespace lst
