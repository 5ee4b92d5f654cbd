// Host interface of the tensor-core product kernel (lst_gemm.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace lst {

// A 16-bit operand in device memory: `inner` contiguous elements, `outer` rows
// `pitch` elements apart, `batch` such matrices `batch_pitch` elements apart.
// The summed dimension is the inner one, or with `transposed` the outer one.
// Base and pitches are multiples of 16 bytes (a rule of the tile loads).
struct GemmOperand {
  const void* ptr;
  int64_t inner, outer, pitch;
  bool transposed = false;
  int64_t batch = 1, batch_pitch = 0;
};

// out = alpha * acc + beta * c (+ diag on the main diagonal), rounded to fp16
// or bf16; c has out's shape, pitch and type; alpha times *scale where that is
// not null (device memory). `vec`: 16 where out's and
// c's rows start on 16 bytes, otherwise 2.
struct StoreParams {
  void* out;
  const void* c;
  int64_t ld, batch_stride;
  float alpha, beta, diag;
  int32_t bf16, vec;
  const float* scale = nullptr;
};

// w = w * decay - step * acc for the matrices of the batch, with w, the derived
// bf16 weight (or null) and step of matrix b at entry first + b of the launch's
// table. `format`: bf16 w, fp32 w with derived bf16, fp32 w (lst_format).
constexpr int kGemmMaxUpdates = 64;
struct UpdateTable {
  void* w[kGemmMaxUpdates];
  uint16_t* w16[kGemmMaxUpdates];
  float step[kGemmMaxUpdates];
};
struct UpdateParams {
  int64_t ld;
  int32_t first, format, vec;
  float decay;
};

// fp32 partial sums of a K range: out[split][row][col], added to what is there
// when `accumulate` is set. Used in place of StoreParams where out is not null.
struct PartialParams {
  float* out;
  int64_t ld, split_stride;
  int32_t accumulate;
};

// Logits of tokens (rows) against a piece of the vocabulary (columns; the other
// way round for GEMM_BF16_XENT_FEW), reduced on the spot; see lst_xent.cu.
struct XentParams {
  const void* targets;
  float2* stats;    // [token][group of 128, or 32]: (max, sum of exp(l - max))
  float* target_logit;
  uint16_t* q;      // [token][entry]: (max - l) in steps of 2^-11, or null
  int64_t q_ld, stat_ld, first_group, first_column;
  int32_t index_bytes;
};

// out = weight[column] * acc (+ out), bf16 or fp32, on any alignment (`vec`: 16 where its
// rows start on 16 bytes); or partial sums where partial.out is not null.
struct WgradParams {
  void* out;
  int64_t ld;
  const void* weight;
  int32_t f32, weight_f32, accumulate, vec;
  PartialParams partial;
};

enum GemmKind {
  GEMM_F16,         // fp16 operands, StoreParams
  GEMM_F16_UPDATE,  // fp16 operands, UpdateParams
  GEMM_BF16,        // bf16 operands, StoreParams or PartialParams
  GEMM_BF16_XENT,   // bf16 operands, XentParams
  GEMM_BF16_XENT_FEW,
  GEMM_BF16_WGRAD,  // bf16 operands, WgradParams
};

struct GemmProblem {
  GemmOperand a, b;
  int64_t m, n, k, batch = 1;
  bool symmetric = false;  // the result is symmetric: form one triangle of tiles and mirror it
  int splits = 1;          // K ranges (PartialParams)
  int parts = 1;           // GEMM_BF16_WGRAD: B as a sum of so many, k / parts (a multiple of 64) deep each; a is
                           // read again for every part, part i of b is matrix i of its batch
  StoreParams store{};
  PartialParams partial{};
  XentParams xent{};
  UpdateParams update{};
  WgradParams wgrad{};
};

constexpr int kGemmMaxProblems = 8;
constexpr int kGemmTile = 256;

// One launch over up to kGemmMaxProblems independent products of one kind.
cudaError_t launch_gemm(GemmKind kind, const GemmProblem* problems, int count, cudaStream_t stream,
                        const UpdateTable* updates = nullptr);

// K ranges into which `tiles` output tiles with sums over `k` are to be split
// when they share a launch with products of `others` tile steps of 64 in all.
int gemm_splits(int64_t tiles, int64_t k, int64_t others);

// Whether some wait of a matrix kernel ran out since the last call on this
// device (synchronises the device).
cudaError_t gemm_take_error(int* out);

}  // namespace lst
