// Softmax cross entropy of a large vocabulary without the matrix of logits,
// and its gradients.
//
// Mathematics. l = x w^T; lse_i = log sum_v exp(l_iv); loss_i = lse_i - l_i,t;
// with p = exp(l - lse) and g = grad_scale / N the gradient with respect to
// the logits is d_iv = g (p_iv - [v = t_i]), and dx = d w, dw = d^T x.
//
// Order. Logits are formed 256 x 256 at a time on the tensor cores
// (lst_gemm.cu); a tile leaves, for each row and 128 columns (32 where few tokens
// are the columns of the tiles), the maximum M
// and the sum of exp(l - M), from which a second kernel joins lse. For the
// gradient the tile also leaves (M - l) in 16 bits of fixed point, steps of
// 2^-11: the workspace holds as many columns of those ("a piece") as fit, and
// d / g is written over them in bf16 once lse is known. That one rounding (and
// the 2^-12 of the fixed point, eight times smaller) is all that d loses;
// keeping exp(l - M) in bf16 instead and rescaling it would round twice. A
// bf16 d is what the tensor cores take next to the bf16 x and w; its error is
// that of the results' own rounding. g multiplies the fp32 results: inside d,
// -g would round alike for every token with an unlikely target, a common factor
// up to 2^-8 off on dx and dw (measured 3.3e-3 from the 64-bit gradient instead
// of 1.9e-3).
//   One piece: 2 N V H operations for the logits, 4 N V H for dx and dw.
//   More pieces: first the statistics of all of them; then each piece's logits
//   are formed again (except those of the one formed last, still there), 8 N V H in all.
// dx sums over the vocabulary: where its tiles do not fill the GPU the sum is
// split, and partial sums are added in a fixed order in fp32, which also
// carries them over the pieces.
//
// Bound by the tensor cores from about 300 tokens on; below by reading w, for which
// few tokens have a form of their own (kFewTokens).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "lst_gemm.h"
#include "lst_ops.h"

namespace lst {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxPieceBytes = int64_t(1) << 30;
// Up to these the logits are formed with the tokens as the columns of narrow tiles:
// the loss over w of 32000 x 2048 takes 28 us for 16 tokens and 29 for 64, with tiles
// of 256 x 256 36 and 31 (but 32 for 128 tokens, where two narrow tiles take 40).
constexpr int64_t kFewTokens = 64;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ int64_t target_at(const void* t, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(t)[i] : static_cast<const int32_t*>(t)[i];
}

// lse and loss of a row from the statistics of its groups of columns, a block per
// row: short chains of dependent loads, and short code.
// The target's logit is formed again as a plain fp32 dot product: the tensor
// cores' sums round towards zero, by up to 1e-5 for a logit of 10, and unlike the
// errors of the other logits this one does not average out of the loss. With
// delta = (dot product - tensor-core logit), lse moves by p delta to first order,
// so that a certain target (p = 1) keeps a loss of zero. A target at -inf (p = 0)
// has no delta: its loss is inf, its row's lse and gradient stay finite.
// No line is both read and written here: with the dot product written back over
// the target's logit, blocks of neighbouring rows took turns at their common line,
// 24 us instead of 9 for 1023 rows, 94 instead of 34 for 8192 rows of 4096.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const float2* __restrict__ stats, int64_t stat_ld, int groups, const float* __restrict__ target_logit,
                const void* __restrict__ targets, int wide, int64_t ignore, int64_t vocab,
                const uint16_t* __restrict__ x, int64_t x_ld, const uint16_t* __restrict__ w, int64_t w_ld, int hidden,
                float* __restrict__ loss, float* __restrict__ lse) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.x;
  const float ninf = __int_as_float(0xff800000);
  const int64_t t = target_at(targets, wide, r);
  const bool with_target = t != ignore && t >= 0 && t < vocab;
  float dot = 0.0f, top = ninf, sum = 0.0f;
  const float old = with_target ? target_logit[r] : 0.0f;
  if (with_target) {
    const uint16_t* a = x + r * x_ld;
    const uint16_t* b = w + t * w_ld;
    if (hidden % 8 == 0) {  // rows are on 16 bytes
#pragma unroll 1
      for (int k = 8 * threadIdx.x; k < hidden; k += 8 * kJoinThreads) {
        const uint4 u = *reinterpret_cast<const uint4*>(a + k), v = *reinterpret_cast<const uint4*>(b + k);
        const uint32_t p[4] = {u.x, u.y, u.z, u.w}, q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dot = __fmaf_rn(__uint_as_float(p[i] << 16), __uint_as_float(q[i] << 16), dot);
          dot = __fmaf_rn(__uint_as_float(p[i] & 0xffff0000u), __uint_as_float(q[i] & 0xffff0000u), dot);
        }
      }
    } else {
#pragma unroll 1
      for (int k = threadIdx.x; k < hidden; k += kJoinThreads)
        dot = __fmaf_rn(__uint_as_float(static_cast<uint32_t>(a[k]) << 16), __uint_as_float(static_cast<uint32_t>(b[k]) << 16), dot);
    }
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < groups; i += kJoinThreads) {
    const float2 s = stats[r * stat_ld + i];
    const float m = fmaxf(top, s.x), base = m == ninf ? 0.0f : m;
    sum = sum * exp2_approx((top - base) * kLog2e) + s.y * exp2_approx((s.x - base) * kLog2e);
    top = m;
  }
  __shared__ float3 part[kJoinThreads / 32];
  auto join = [&](int width) {  // over `width` lanes
    float m = top;
#pragma unroll 1
    for (int o = width / 2; o > 0; o >>= 1) {
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const float base = m == ninf ? 0.0f : m;
    sum *= exp2_approx((top - base) * kLog2e);
    top = m;
#pragma unroll 1
    for (int o = width / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  };
  join(32);
  if (lane == 0) part[warp] = make_float3(top, sum, dot);
  __syncthreads();
  if (warp == 0) {
    const float3 p = part[lane & (kJoinThreads / 32 - 1)];
    top = p.x, sum = p.y, dot = p.z;
    join(kJoinThreads / 32);
    if (lane == 0) {
      float l = (top == ninf ? 0.0f : top) + logf(sum);
      if (with_target) {
        const float delta = dot - old;
        if (fabsf(delta) <= 3.402823466e38f) l += delta * exp2_approx((old - l) * kLog2e);
      }
      lse[r] = l;
      loss[r] = with_target ? l - dot : t == ignore ? 0.0f : __int_as_float(0x7fc00000);
    }
  }
}

// The mean loss and g = grad_scale / N from all losses, in a fixed order, by one
// block: fp64 for a thread's share of the rows, fp32 for the tree above.
__device__ __forceinline__ void mean_of_losses(const float* __restrict__ loss, const void* __restrict__ targets, int wide,
                                               int64_t ignore, int rows, float grad_scale, float* __restrict__ mean,
                                               float* __restrict__ g) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double mine = 0.0;
  int count = 0;
  for (int64_t i0 = threadIdx.x; i0 < rows; i0 += 8 * 256) {
    int64_t of[8];
    float each[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t i = i0 + j * 256;
      of[j] = i < rows ? target_at(targets, wide, i) : ignore;
      each[j] = i < rows ? loss[i] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (of[j] != ignore) {
        mine += static_cast<double>(each[j]);
        ++count;
      }
  }
  float total = static_cast<float>(mine);
  __shared__ float sums[8];
  __shared__ int counts[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_down_sync(0xffffffffu, total, o);
    count += __shfl_down_sync(0xffffffffu, count, o);
  }
  if (lane == 0) {
    sums[warp] = total;
    counts[warp] = count;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 8; ++i) {
      total += sums[i];
      count += counts[i];
    }
    *mean = count ? total / static_cast<float>(count) : 0.0f;
    *g = count ? grad_scale / static_cast<float>(count) : 0.0f;
  }
}

// A row whose target takes part in the gradient.
__device__ __forceinline__ bool in_gradient(int64_t t, int64_t ignore, int64_t vocab) {
  return t != ignore && t >= 0 && t < vocab;
}

// x as the product d^T x reads it: rows without a gradient become zero, since d
// is zero there but 0 * infinity would reach dw.
struct MaskedRows {
  const uint16_t* src;
  uint16_t* dst;
  int64_t ld, dst_ld;
  int32_t rows, cols, vec;
};

// d / g over q, in place: 16 entries per thread, one row per block of columns. The
// blocks after the first `d_blocks` copy x with its rows masked, and the first of
// them forms the mean loss and g.
__global__ void __launch_bounds__(256)
    logit_grad_kernel(uint16_t* __restrict__ q, int64_t q_ld, const float2* __restrict__ stats, int64_t stat_ld,
                      int64_t first_group, int group_shift, int64_t first_column, int columns, const float* __restrict__ lse,
                      const float* __restrict__ loss, const void* __restrict__ targets, int wide,
                      int64_t ignore, int64_t vocab, int blocks_per_row, int d_blocks,
                      MaskedRows x, float grad_scale, float* __restrict__ mean, float* __restrict__ g) {
  let_next_start();
  wait_for_previous();
  if (static_cast<int>(blockIdx.x) >= d_blocks) {
    if (blockIdx.x == d_blocks) {
      mean_of_losses(loss, targets, wide, ignore, x.rows, grad_scale, mean, g);
      return;
    }
    for (int64_t r = blockIdx.x - d_blocks - 1; r < x.rows; r += gridDim.x - d_blocks - 1) {
      const bool keep = in_gradient(target_at(targets, wide, r), ignore, vocab);
      if (x.vec) {
        for (int c = threadIdx.x * 8; c < x.cols; c += 2048)
          *reinterpret_cast<uint4*>(x.dst + r * x.dst_ld + c) =
              keep ? *reinterpret_cast<const uint4*>(x.src + r * x.ld + c) : make_uint4(0, 0, 0, 0);
      } else {
        for (int c = threadIdx.x; c < x.cols; c += 256) x.dst[r * x.dst_ld + c] = keep ? x.src[r * x.ld + c] : 0;
      }
    }
    return;
  }
  const int row = blockIdx.x / blocks_per_row;
  const int col = ((blockIdx.x - row * blocks_per_row) * 256 + threadIdx.x) * 16;
  if (col >= columns) return;
  uint4* const p = reinterpret_cast<uint4*>(q + static_cast<int64_t>(row) * q_ld + col);
  const int64_t t = target_at(targets, wide, row);
  if (!in_gradient(t, ignore, vocab)) {
    p[0] = p[1] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4 x0 = p[0], x1 = p[1];
  const float l = lse[row];
  const float top = stats[row * stat_ld + first_group + (col >> group_shift)].x;
  const float base = (top - l) * kLog2e;
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  float d[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t q16 = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
    const float steps = q16 == 0xffffu ? __int_as_float(0x7f800000) : static_cast<float>(q16);
    d[i] = exp2_approx(__fmaf_rn(steps, -kLog2e / 2048.0f, base));
  }
  const int64_t at = t - first_column - col;
  if (at >= 0 && at < 16) {
    // p - 1 of the target cancels when p is near 1; p = exp(-loss)
    const float e = expm1f(-loss[row]);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i == static_cast<int>(at)) d[i] = e;
  }
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(d[2 * i], d[2 * i + 1]);
    r[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  p[0] = make_uint4(r[0], r[1], r[2], r[3]);
  p[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// dx = g times the sum of its parts, in a fixed order, rounded to bf16.
__global__ void __launch_bounds__(256)
    dx_kernel(const float* __restrict__ parts, int64_t ld, int64_t split_stride, int splits, int rows, int cols,
              __nv_bfloat16* __restrict__ dx, int64_t dx_ld, int wide_store, const float* __restrict__ gp) {
  let_next_start();
  wait_for_previous();
  const int quads = (cols + 3) / 4;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int row = static_cast<int>(i / quads);
  if (row >= rows) return;
  const int col = static_cast<int>(i - static_cast<int64_t>(row) * quads) * 4;
  const float* p = parts + static_cast<int64_t>(row) * ld + col;
  float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int s0 = 0; s0 < splits; s0 += 8) {  // eight parts in flight
    float4 b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      b[j] = s0 + j < splits ? *reinterpret_cast<const float4*>(p + (s0 + j) * split_stride) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = make_float4(a.x + b[j].x, a.y + b[j].y, a.z + b[j].z, a.w + b[j].w);
  }
  __nv_bfloat16* o = dx + static_cast<int64_t>(row) * dx_ld + col;
  const float g = *gp, v[4] = {a.x * g, a.y * g, a.z * g, a.w * g};
  if (wide_store) {
    const __nv_bfloat162 h0 = __floats2bfloat162_rn(v[0], v[1]), h1 = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(o) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
  } else {
    for (int k = 0; k < 4 && col + k < cols; ++k) o[k] = __float2bfloat16_rn(v[k]);
  }
}

// Rows at a pitch that is a multiple of 16 bytes, for operands that are not
// laid out so (a rule of the tile loads).
__global__ void __launch_bounds__(256)
    pack_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t rows, int cols, uint16_t* __restrict__ dst,
                int64_t dst_ld) {
  let_next_start();
  wait_for_previous();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += 256) dst[r * dst_ld + c] = src[r * ld + c];
}

bool tile_ready(const lst_matrix* m) {
  return reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && (m->stride * 2) % 16 == 0;
}

struct Plan {
  int64_t groups, piece, pieces, splits;
  int group_shift;  // log2 of the vocabulary entries of a group of statistics
  int64_t packed_ld, x_ld, part_ld;
  int64_t scalar_off, tlogit_off, stats_off, xm_off, xpack_off, wpack_off, part_off, q_off;
  int64_t bytes;
};

// Layout of the workspace; `bytes` < 0: for one piece, at most 1 GiB of it.
// Returns false when not even one tile of columns fits.
bool make_plan(int64_t n, int64_t h, int64_t v, bool grad, bool pack_x, bool pack_w, int64_t bytes, Plan* p) {
  p->group_shift = n <= kFewTokens ? 5 : 7;
  p->groups = ops_ceil_div(v, int64_t(1) << p->group_shift);
  p->packed_ld = ops_round_up(h, 8);
  int64_t at = 0;
  auto take = [&](int64_t size) {
    const int64_t off = at;
    at += ops_round_up(size, 256);
    return off;
  };
  p->scalar_off = take(256);
  p->tlogit_off = take(n * 4);
  p->stats_off = take(n * p->groups * 8);
  p->xpack_off = take(pack_x ? n * p->packed_ld * 2 : 0);
  p->wpack_off = take(pack_w ? v * p->packed_ld * 2 : 0);
  p->piece = p->pieces = 0;
  p->splits = 1;
  if (grad) {
    p->xm_off = take(n * p->packed_ld * 2);
    p->part_ld = ops_round_up(h, 32);
    const int64_t tiles_h = ops_ceil_div(h, kGemmTile), tiles = ops_ceil_div(n, kGemmTile) * tiles_h;
    // dx shares its launch with dw, whose sums go over the tokens (and 3 steps for a tile's ramp)
    auto split = [&](int64_t piece) {
      const int64_t columns = std::min(piece, v);
      return gemm_splits(tiles, columns, ops_ceil_div(columns, kGemmTile) * tiles_h * (ops_ceil_div(n, 64) + 3));
    };
    const int64_t whole = ops_round_up(v, kGemmTile);
    const int64_t most = std::max<int64_t>(kGemmTile, kMaxPieceBytes / (2 * n) / kGemmTile * kGemmTile);
    auto parts = [&](int64_t piece) {
      const int64_t splits = split(piece);
      return splits > 1 || piece < v ? splits * n * p->part_ld * 4 + 256 : 0;
    };
    int64_t piece = std::min(whole, most);
    if (bytes >= 0)
      while (piece > 0 && at + ops_round_up(parts(piece), 256) + n * piece * 2 > bytes)
        piece = piece > 4 * kGemmTile ? piece / 2 / kGemmTile * kGemmTile : piece - kGemmTile;
    if (piece <= 0) return false;
    p->piece = piece;
    p->pieces = ops_ceil_div(v, piece);
    p->splits = split(piece);
    p->part_off = take(parts(piece));
    p->q_off = take(n * piece * 2);
  }
  p->bytes = at;
  return bytes < 0 || at <= bytes;
}

// What the calls report: enough for one piece (at most 1 GiB of it) of this many tokens
// or of any fewer, so that a workspace sized for the largest batch serves all. What
// make_plan takes is not monotone in n:
//   statistics are per 32 entries up to kFewTokens tokens, per 128 above;
//   a piece is rounded down to tiles, so that 1 GiB is not always filled;
//   few tokens split dx more often. gemm_splits takes s > 1 ranges only where
//   blocks / (s - 1) > max(share / 2, 8), with share >= (tiles blocks + others) / 76 - 1,
//   tiles >= tiles_h n / 256 and others >= blocks tiles_h n / 256: it follows that
//   (s - 1) n < 171 * 128 / tiles_h, and s is at most 32. One piece has parts for s > 1 only.
int64_t plan_bytes(int64_t n, int64_t h, int64_t v, bool grad, bool pack_x, bool pack_w) {
  const int64_t ld = ops_round_up(h, 8), few = std::min(n, kFewTokens);
  auto size = [](int64_t bytes) { return ops_round_up(bytes, 256); };
  int64_t bytes = 256 + size(n * 4) + size(std::max(n * ops_ceil_div(v, 128), few * ops_ceil_div(v, 32)) * 8) +
                  size(pack_x ? n * ld * 2 : 0) + size(pack_w ? v * ld * 2 : 0);
  if (!grad) return bytes;
  const int64_t all = n * ops_round_up(v, kGemmTile) * 2, most = 171 * 128 / ops_ceil_div(h, kGemmTile);
  const int64_t rows = std::min(32 * n, most + (all > kMaxPieceBytes ? n : std::min(n, most)));
  const int64_t q = std::min(all, std::max(kMaxPieceBytes, n * 2 * kGemmTile));
  return bytes + size(n * ld * 2) + size(rows * ops_round_up(h, 32) * 4 + 256) + size(q);
}

// Sizes that the calls take (and whose workspace is counted in 64 bits: no device holds a
// w of more than 2^40 elements).
bool sizes_fit(int64_t n, int64_t h, int64_t v) {
  return n > 0 && h > 0 && v > 0 && n <= (int64_t(1) << 24) && v <= INT32_MAX && h <= INT32_MAX && v <= (int64_t(1) << 40) / h &&
         n <= (int64_t(1) << 40) / h;
}

// A matrix of rows; `transposed`: the product sums over its rows.
GemmOperand rows_operand(const void* ptr, int64_t rows, int64_t cols, int64_t ld, bool transposed = false) {
  return {ptr, cols, rows, ld, transposed};
}

int store_width(const lst_matrix* m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(m->data) | static_cast<uintptr_t>(m->stride * 2);
  return a % 16 == 0 ? 16 : 2;
}

lst_status check_xw(const lst_matrix* x, const lst_matrix* w, const lst_indices* targets, const char* who) {
  LST_TRY(check_matrix(x, "x", who));
  LST_TRY(check_matrix(w, "w", who));
  LST_TRY(check_indices(targets, "targets", who));
  if (x->dtype != LST_BF16 || w->dtype != LST_BF16) return fail(LST_ERR_INVALID_ARG, "%s: x and w must be bf16", who);
  if (x->rows != targets->count || x->cols != w->cols)
    return fail(LST_ERR_INVALID_ARG, "%s: x must be targets x hidden, w vocabulary x hidden", who);
  if (w->rows == 0 || w->cols == 0) return fail(LST_ERR_INVALID_ARG, "%s: empty vocabulary or hidden size", who);
  if (x->rows > (int64_t(1) << 24)) return fail(LST_ERR_INVALID_ARG, "%s: more than 2^24 targets", who);
  if (x->rows > 0 && !sizes_fit(x->rows, x->cols, w->rows))
    return fail(LST_ERR_INVALID_ARG, "%s: x or w of more than 2^40 elements", who);
  return LST_OK;
}

struct Call {
  const char* who;
  const lst_matrix *x, *w;
  const lst_indices* targets;
  int64_t ignore;
  float *loss, *lse;
  char* ws;
  cudaStream_t stream;
  Plan p;
  const void *xp, *wp;
  int64_t x_ld, w_ld;
  int wide;

  // The operands of the products, packed first where their rows are not on 16 bytes.
  cudaError_t operands() {
    xp = x->data, wp = w->data, x_ld = x->stride, w_ld = w->stride;
    auto pack = [&](const lst_matrix* m, int64_t off, const void** ptr, int64_t* ld) {
      const unsigned grid = static_cast<unsigned>(std::min<int64_t>(m->rows, 8192));
      *ptr = ws + off;
      *ld = p.packed_ld;
      return launch_chained(pack_kernel, dim3(grid), dim3(256), 0, stream, static_cast<const uint16_t*>(m->data), m->stride,
                            m->rows, static_cast<int>(m->cols), reinterpret_cast<uint16_t*>(ws + off), p.packed_ld);
    };
    cudaError_t err = cudaSuccess;
    if (!tile_ready(x)) err = pack(x, p.xpack_off, &xp, &x_ld);
    if (err == cudaSuccess && !tile_ready(w)) err = pack(w, p.wpack_off, &wp, &w_ld);
    return err;
  }

  cudaError_t logits(int64_t v0, int64_t columns, bool keep) {
    const GemmOperand tokens = rows_operand(xp, x->rows, x->cols, x_ld);
    const GemmOperand entries = rows_operand(static_cast<const uint16_t*>(wp) + v0 * w_ld, columns, w->cols, w_ld);
    const bool few = x->rows <= kFewTokens;
    GemmProblem g;
    g.a = few ? entries : tokens;
    g.b = few ? tokens : entries;
    g.m = few ? columns : x->rows;
    g.n = few ? x->rows : columns;
    g.k = x->cols;
    g.xent = {targets->data, reinterpret_cast<float2*>(ws + p.stats_off), reinterpret_cast<float*>(ws + p.tlogit_off),
              keep ? reinterpret_cast<uint16_t*>(ws + p.q_off) : nullptr, p.piece, p.groups, v0 >> p.group_shift, v0,
              targets->bits / 8};
    return launch_gemm(few ? GEMM_BF16_XENT_FEW : GEMM_BF16_XENT, &g, 1, stream);
  }

  cudaError_t sum_dx(const lst_matrix* dx) {
    const bool wide_store = dx->cols % 4 == 0 && dx->stride % 4 == 0 && reinterpret_cast<uintptr_t>(dx->data) % 8 == 0;
    return launch_chained(dx_kernel, dim3(static_cast<unsigned>(ops_ceil_div(ops_ceil_div(dx->cols, 4) * dx->rows, 256))),
                          dim3(256), 0, stream, reinterpret_cast<const float*>(ws + p.part_off), p.part_ld,
                          dx->rows * p.part_ld, static_cast<int>(p.splits), static_cast<int>(dx->rows),
                          static_cast<int>(dx->cols), static_cast<__nv_bfloat16*>(dx->data), dx->stride, wide_store,
                          reinterpret_cast<const float*>(ws + p.scalar_off));
  }

  cudaError_t join() {
    return launch_chained(join_kernel, dim3(static_cast<unsigned>(x->rows)), dim3(kJoinThreads), 0, stream,
                          reinterpret_cast<const float2*>(ws + p.stats_off), p.groups, static_cast<int>(p.groups),
                          reinterpret_cast<const float*>(ws + p.tlogit_off), targets->data, wide, ignore, w->rows,
                          static_cast<const uint16_t*>(xp), x_ld, static_cast<const uint16_t*>(wp), w_ld,
                          static_cast<int>(x->cols), loss, lse);
  }
};

}  // namespace
}  // namespace lst

using namespace lst;

extern "C" int64_t lst_xent_workspace_bytes(int64_t count, int64_t hidden, int64_t vocab, int32_t with_grad) {
  if (!sizes_fit(count, hidden, vocab)) return 0;
  const bool pack = hidden % 8 != 0;  // contiguous rows of such a length are off 16 bytes
  return plan_bytes(count, hidden, vocab, with_grad != 0, pack, pack);
}

extern "C" int64_t lst_xent_workspace_bytes_for(const lst_matrix* x, const lst_matrix* w, int32_t with_grad) {
  if (!x || !w || x->cols != w->cols || !sizes_fit(x->rows, x->cols, w->rows)) return 0;
  return plan_bytes(x->rows, x->cols, w->rows, with_grad != 0, !tile_ready(x), !tile_ready(w));
}

extern "C" lst_status lst_xent_loss(const lst_matrix* x, const lst_matrix* w, const lst_indices* targets,
                                    int64_t ignore_index, float* loss, float* lse, void* workspace,
                                    int64_t workspace_bytes, void* cuda_stream) {
  clear_error();
  const char* who = "lst_xent_loss";
  LST_TRY(check_xw(x, w, targets, who));
  if (x->rows == 0) return LST_OK;
  if (!loss || !lse) return fail(LST_ERR_INVALID_ARG, "%s: loss or lse is null", who);
  if (reinterpret_cast<uintptr_t>(loss) % 4 || reinterpret_cast<uintptr_t>(lse) % 4)
    return fail(LST_ERR_ALIGNMENT, "%s: loss or lse not 4-byte aligned", who);
  Call c{who, x, w, targets, ignore_index, loss, lse, static_cast<char*>(workspace),
         static_cast<cudaStream_t>(cuda_stream), {}, nullptr, nullptr, 0, 0, targets->bits == 64};
  make_plan(x->rows, x->cols, w->rows, false, !tile_ready(x), !tile_ready(w), -1, &c.p);
  LST_TRY(check_workspace(workspace, workspace_bytes, c.p.bytes, who));
  LST_TRY_CUDA(c.operands(), who);
  LST_TRY_CUDA(c.logits(0, w->rows, false), who);
  LST_TRY_CUDA(c.join(), who);
  return LST_OK;
}

extern "C" lst_status lst_xent_grad(const lst_matrix* x, const lst_matrix* w, const lst_indices* targets,
                                    int64_t ignore_index, float grad_scale, float* loss, float* lse, float* mean,
                                    const lst_matrix* dx, const lst_matrix* dw, int32_t accumulate_dw, void* workspace,
                                    int64_t workspace_bytes, void* cuda_stream) {
  clear_error();
  const char* who = "lst_xent_grad";
  LST_TRY(check_xw(x, w, targets, who));
  LST_TRY(check_matrix(dx, "dx", who));
  LST_TRY(check_matrix(dw, "dw", who));
  if (dx->dtype != LST_BF16 || dw->dtype != LST_BF16) return fail(LST_ERR_INVALID_ARG, "%s: dx and dw must be bf16", who);
  if (dx->rows != x->rows || dx->cols != x->cols || dw->rows != w->rows || dw->cols != w->cols)
    return fail(LST_ERR_INVALID_ARG, "%s: dx and dw must have the shapes of x and w", who);
  if (!std::isfinite(grad_scale)) return fail(LST_ERR_INVALID_ARG, "%s: grad_scale not finite", who);
  if (!mean) return fail(LST_ERR_INVALID_ARG, "%s: mean is null", who);
  if (x->rows > 0 && (!loss || !lse)) return fail(LST_ERR_INVALID_ARG, "%s: loss or lse is null", who);
  if (reinterpret_cast<uintptr_t>(loss) % 4 || reinterpret_cast<uintptr_t>(lse) % 4 ||
      reinterpret_cast<uintptr_t>(mean) % 4)
    return fail(LST_ERR_ALIGNMENT, "%s: loss, lse or mean not 4-byte aligned", who);
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  if (x->rows == 0) {
    LST_TRY_CUDA(cudaMemsetAsync(mean, 0, 4, stream), who);
    if (!accumulate_dw)
      LST_TRY_CUDA(cudaMemset2DAsync(dw->data, (size_t)dw->stride * 2, 0, (size_t)dw->cols * 2, (size_t)dw->rows, stream),
                   who);
    return LST_OK;
  }
  Call c{who, x, w, targets, ignore_index, loss, lse, static_cast<char*>(workspace), stream, {}, nullptr, nullptr,
         0, 0, targets->bits == 64};
  const bool px = !tile_ready(x), pw = !tile_ready(w);
  if (!make_plan(x->rows, x->cols, w->rows, true, px, pw, workspace_bytes < 0 ? 0 : workspace_bytes, &c.p))
    return fail(LST_ERR_INVALID_ARG,
                "%s: workspace of %lld bytes holds no piece of 256 columns (lst_xent_workspace_bytes_for: %lld for all)", who,
                (long long)workspace_bytes, (long long)plan_bytes(x->rows, x->cols, w->rows, true, px, pw));
  const Plan& p = c.p;
  LST_TRY(check_workspace(workspace, workspace_bytes, p.bytes, who));
  char* ws = c.ws;
  const int64_t n = x->rows, h = x->cols, v = w->rows;
  float* g = reinterpret_cast<float*>(ws + p.scalar_off);
  uint16_t* xm = reinterpret_cast<uint16_t*>(ws + p.xm_off);
  uint16_t* q = reinterpret_cast<uint16_t*>(ws + p.q_off);

  LST_TRY_CUDA(c.operands(), who);
  for (int64_t k = p.pieces - 1; k >= 0; --k) {
    const int64_t v0 = k * p.piece;
    LST_TRY_CUDA(c.logits(v0, std::min(p.piece, v - v0), k == 0), who);
  }
  LST_TRY_CUDA(c.join(), who);
  const bool parts = p.splits > 1 || p.pieces > 1;
  // the first piece sets every partial sum of dx: only the last can be shorter,
  // with fewer splits
  for (int64_t k = 0; k < p.pieces; ++k) {
    const int64_t v0 = k * p.piece, columns = std::min(p.piece, v - v0);
    if (k > 0) LST_TRY_CUDA(c.logits(v0, columns, true), who);
    const int blocks = static_cast<int>(ops_ceil_div(columns, 4096));
    const int64_t d_blocks = n * blocks, copies = k == 0 ? std::min<int64_t>(n, 2048) + 1 : 0;
    const MaskedRows masked = {static_cast<const uint16_t*>(c.xp), xm, c.x_ld, p.packed_ld, static_cast<int32_t>(n),
                               static_cast<int32_t>(h), h % 8 == 0};
    LST_TRY_CUDA(launch_chained(logit_grad_kernel, dim3(static_cast<unsigned>(d_blocks + copies)), dim3(256), 0, stream, q,
                                p.piece, reinterpret_cast<const float2*>(ws + p.stats_off), p.groups, v0 >> p.group_shift, p.group_shift, v0,
                                static_cast<int>(columns), lse, loss, targets->data, c.wide, ignore_index, v, blocks, static_cast<int>(d_blocks), masked,
                                grad_scale, mean, g),
                 who);
    // dw of the piece = d^T x, and dx += d w, in one launch: the tiles of the longer sums first
    GemmProblem both[2];
    GemmProblem& d = both[n > columns / p.splits ? 0 : 1];
    GemmProblem& e = both[n > columns / p.splits ? 1 : 0];
    d.a = rows_operand(q, n, columns, p.piece, true);
    d.b = rows_operand(xm, n, h, p.packed_ld, true);
    d.m = columns;
    d.n = h;
    d.k = n;
    uint16_t* dwp = static_cast<uint16_t*>(dw->data) + v0 * dw->stride;
    d.store = {dwp, accumulate_dw ? dwp : nullptr, dw->stride, 0, 1.0f, 1.0f, 0.0f, 1, store_width(dw), g};
    e.a = rows_operand(q, n, columns, p.piece);
    e.b = rows_operand(static_cast<const uint16_t*>(c.wp) + v0 * c.w_ld, columns, h, c.w_ld, true);
    e.m = n;
    e.n = h;
    e.k = columns;
    if (parts) {
      e.splits = static_cast<int>(p.splits);
      e.partial = {reinterpret_cast<float*>(ws + p.part_off), p.part_ld, n * p.part_ld, k > 0};
    } else {
      e.store = {dx->data, nullptr, dx->stride, 0, 1.0f, 0.0f, 0.0f, 1, store_width(dx), g};
    }
    LST_TRY_CUDA(launch_gemm(GEMM_BF16, both, 2, stream), who);
  }
  if (parts) LST_TRY_CUDA(c.sum_dx(dx), who);
  return LST_OK;
}
