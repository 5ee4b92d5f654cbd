// Argument checks and small device helpers shared by the training operators.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "lst_internal.h"

namespace lst {

inline int64_t ops_round_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
inline int64_t ops_ceil_div(int64_t x, int64_t a) { return (x + a - 1) / a; }
inline int dtype_bytes(int32_t dtype) { return dtype == LST_F32 ? 4 : 2; }

// A matrix argument: non-null, known type, sizes, alignment to its element.
inline lst_status check_matrix(const lst_matrix* m, const char* name, const char* who) {
  if (!m) return fail(LST_ERR_INVALID_ARG, "%s: %s is null", who, name);
  if (m->dtype != LST_BF16 && m->dtype != LST_F32)
    return fail(LST_ERR_INVALID_ARG, "%s: %s has unknown type %d", who, name, (int)m->dtype);
  if (m->rows < 0 || m->cols < 0 || m->rows > (int64_t(1) << 31) - 1 || m->cols > (int64_t(1) << 31) - 1)
    return fail(LST_ERR_INVALID_ARG, "%s: %s: rows or columns outside 0..2^31-1", who, name);
  if (m->stride < m->cols) return fail(LST_ERR_INVALID_ARG, "%s: %s: stride below the column count", who, name);
  if (m->stride > (int64_t(1) << 36)) return fail(LST_ERR_INVALID_ARG, "%s: %s: stride above 2^36", who, name);
  if (m->rows > 0 && m->cols > 0) {
    if (!m->data) return fail(LST_ERR_INVALID_ARG, "%s: %s: data is null", who, name);
    if (reinterpret_cast<uintptr_t>(m->data) % dtype_bytes(m->dtype))
      return fail(LST_ERR_ALIGNMENT, "%s: %s: data not aligned to its element", who, name);
  }
  return LST_OK;
}

inline lst_status check_indices(const lst_indices* t, const char* name, const char* who) {
  if (!t) return fail(LST_ERR_INVALID_ARG, "%s: %s is null", who, name);
  if (t->bits != 32 && t->bits != 64) return fail(LST_ERR_INVALID_ARG, "%s: %s: bits must be 32 or 64", who, name);
  if (t->count < 0 || t->count > (int64_t(1) << 30))
    return fail(LST_ERR_INVALID_ARG, "%s: %s: count outside 0..2^30", who, name);
  if (t->count > 0) {
    if (!t->data) return fail(LST_ERR_INVALID_ARG, "%s: %s: data is null", who, name);
    if (reinterpret_cast<uintptr_t>(t->data) % (t->bits / 8))
      return fail(LST_ERR_ALIGNMENT, "%s: %s: data not aligned to its element", who, name);
  }
  return LST_OK;
}

inline lst_status check_workspace(const void* ws, int64_t bytes, int64_t need, const char* who) {
  if (need == 0) return LST_OK;
  if (!ws) return fail(LST_ERR_INVALID_ARG, "%s: workspace is null", who);
  if (reinterpret_cast<uintptr_t>(ws) % 256) return fail(LST_ERR_ALIGNMENT, "%s: workspace not 256-byte aligned", who);
  if (bytes < need)
    return fail(LST_ERR_INVALID_ARG, "%s: workspace of %lld bytes, at least %lld needed", who, (long long)bytes,
                (long long)need);
  return LST_OK;
}

// Launches of the operators are chained: each kernel may be set up while the one
// before it runs (programmatic stream serialisation), and begins with
// wait_for_previous(), which returns when everything before it on the stream
// has finished and is visible. let_next_start() allows the next launch's setup;
// all kernels call it at once. A chain of small launches goes from about 10 to
// 5 us each this way.
template <class... Params, class... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}
#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

#define LST_TRY(expr)                        \
  do {                                       \
    const lst_status st_ = (expr);           \
    if (st_ != LST_OK) return st_;           \
  } while (0)
#define LST_TRY_CUDA(expr, who)                        \
  do {                                                 \
    const cudaError_t err_ = (expr);                   \
    if (err_ != cudaSuccess) return cuda_fail(err_, who); \
  } while (0)

}  // namespace lst
