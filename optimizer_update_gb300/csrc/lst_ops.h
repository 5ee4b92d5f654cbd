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
