// Newton-Schulz constants and the one-kernel form for small matrices.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace lst {

// The quintic's coefficients, and the powers of two by which fp16 values of each
// kind are stored (lst_muon.cu says why these).
constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr float kScaleX = 16384.0f, kScaleA = 16384.0f, kScaleQ = 8192.0f, kScaleQA = 16384.0f, kScaleR = 4096.0f;

struct NsMomentum {
  float momentum, eps;
  int32_t nesterov;
};

// u of one element from its gradient and updated momentum.
__device__ __forceinline__ float muon_u(float g, float m, const NsMomentum& s) {
  return s.nesterov ? __fadd_rn(g, __fmul_rn(s.momentum, m)) : m;
}
__device__ __forceinline__ float new_momentum(float m, float g, const NsMomentum& s) {
  return __fadd_rn(__fmul_rn(s.momentum, m), g);
}

// Squares in fp32 leave its range from |u| = 1.8e19 on and lose their last bits below
// 1e-23. Where a sum of squares is outside kLeastSum .. kMostSum it is taken again over
// u * pre, with `pre` one of two powers of two; matrices in the ordinary range do not notice.
constexpr float kLeastSum = 0x1p-100f, kMostSum = 0x1p100f;
constexpr float kSmallPre = 0x1p100f;  // of sums below: u is under 2^-50
constexpr float kLargePre = 0x1p-80f;  // of sums above, infinite or NaN
__device__ __forceinline__ bool ordinary_sum(float sum) { return sum >= kLeastSum && sum <= kMostSum; }
__device__ __forceinline__ float other_pre(float sum) { return sum < kLeastSum ? kSmallPre : kLargePre; }

// X_0 = U / (|U|_F + eps) times kScaleX is (u * pre) * inv of every element, from the sum of
// (u * pre)^2. The divisor is 2^-50 at least, or with kSmallPre (zero matrices
// among them) 2^100 times the smallest eps: `inv` is finite.
__device__ __forceinline__ float ns_inv(float sum, float pre, float eps) { return kScaleX / (sqrtf(sum) + eps * pre); }

// One matrix of a launch: the input (a gradient with its momentum, or the matrix
// itself), and where the result goes: a bf16 matrix, or a weight to update.
struct NsSmallItem {
  const void* g;
  float* mom;      // null: g is the matrix
  void* out;       // bf16 result, or the weight
  uint16_t* w16;   // derived bf16 weight (mixed layout)
  int64_t ld, out_ld;
  float step;      // lr * update scale (weights)
};
constexpr int kNsSmallItems = 48;
struct NsSmallCall {
  int64_t rows, cols;
  int32_t f32;      // g is fp32
  int32_t format;   // lst_format of the weight, or -1: bf16 result
  int32_t steps;
  float decay;
  NsMomentum s;
};

// Whether matrices of this shape run in one kernel.
bool ns_small_fits(int64_t rows, int64_t cols);
cudaError_t ns_small(const NsSmallItem* items, int count, const NsSmallCall& call, cudaStream_t stream);
// For m x m Gram matrices with m at most kNsChain: what two steps make of them
// (s <- Q' Q, stored times kScaleR; s holds A times kScaleA), `count` matrices
// `pitch` elements apart with rows `ld` apart (a multiple of 64), on 16 bytes.
constexpr int kNsChain = 256;
cudaError_t ns_chain(__half* s, int64_t m, int64_t ld, int64_t pitch, int64_t count, cudaStream_t stream);
// Whether one of these kernels' waits ran out since the last call (synchronises).
cudaError_t ns_small_take_error(int* out);

}  // namespace lst
