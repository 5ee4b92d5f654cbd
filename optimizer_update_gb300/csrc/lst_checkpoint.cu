// Activations kept in 8 bits: save, restore, and the weight gradient of a linear
// layer from the checkpoint of its input. The format is described in lst_ckpt.cuh.
//
// Save and restore are one pass each, bound by memory: 2 + 1.03 bytes a bf16 value.
#include <algorithm>
#include <cmath>

#include "lst_ckpt.cuh"
#include "lst_gemm.h"

namespace lst {

namespace {

constexpr int64_t kSms = 152;
constexpr int kWarpColumns = 1024;  // of a row, per warp and turn

struct Kept {
  uint8_t* data;
  uint8_t* scales;
  int64_t stride, scale_stride;
  int32_t e4m3;
};

template <class T, bool VEC>
__global__ void __launch_bounds__(256)
    save_kernel(const T* __restrict__ x, int64_t ld, Kept out, int64_t rows, int cols, int parts) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8, tasks = rows * parts;
  for (int64_t t = blockIdx.x * 8 + (threadIdx.x >> 5); t < tasks; t += warps) {
    const int64_t row = t / parts;
    const int col = static_cast<int>(t - row * parts) * kWarpColumns;
    const Cols<VEC> c = {static_cast<uint32_t>(lane), 32u, static_cast<uint32_t>(min(cols - col, kWarpColumns))};
    Unit u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[k].fill(0.0f);
      if (c.has(k)) c.load(x + row * ld + col, k, u[k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c.save(u[k], k, out.data + row * out.stride + col, out.scales + row * out.scale_stride + col / kCkptBlock, out.e4m3);
  }
}

template <class T, bool VEC>
__global__ void __launch_bounds__(256)
    restore_kernel(Kept in, T* __restrict__ out, int64_t ld, int64_t rows, int cols, int parts) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8, tasks = rows * parts;
  for (int64_t t = blockIdx.x * 8 + (threadIdx.x >> 5); t < tasks; t += warps) {
    const int64_t row = t / parts;
    const int col = static_cast<int>(t - row * parts) * kWarpColumns;
    const Cols<VEC> c = {static_cast<uint32_t>(lane), 32u, static_cast<uint32_t>(min(cols - col, kWarpColumns))};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!c.has(k)) continue;
      Unit u;
      c.restore(in.data + row * in.stride + col, in.scales + row * in.scale_stride + col / kCkptBlock, in.e4m3, k, u);
      c.store(out + row * ld + col, k, u);
    }
  }
}

// The operands of the weight gradient's product. X: the restored rows, or with NORM those
// times rsqrt(mean of their squares + eps), as bf16 rows of whole units of 16 columns (what
// stands behind a row's last column is not read); by `threads` threads a row, 32 or 256.
// Blocks from `row_blocks` on copy the rows of dy where they are not on 16 bytes.
//
// Converting X on its way into the product instead (four warps beside the loads, codes by a
// ring of their own) kept the tensor cores waiting: a K step takes 512 cycles and 125 of
// the 128 bytes a cycle that shared memory moves; 8192 x 11008 x 4096 took 1750 us.
struct OperandArgs {
  Kept in;
  uint16_t* x;
  int64_t x_ld, rows;
  int32_t cols, threads, row_blocks;
  float eps;
  const uint16_t* dy;
  uint16_t* dy_out;
  int64_t dy_ld, dy_out_ld;
  int32_t dy_cols;
  int32_t parts;  // X as a sum of so many bf16 parts, each `rows` rows behind the one before
};
__device__ __forceinline__ void decode16(const uint4& q, uint32_t byte, bool e4m3, float2 (&v)[8]) {
  const float2 step = both(ckpt_step(byte));
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (e4m3) {
#pragma unroll
    for (int j = 0; j < 4; ++j) ckpt_decode4(w[j], true, v[2 * j], v[2 * j + 1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) ckpt_decode4(w[j], false, v[2 * j], v[2 * j + 1]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = mul2(v[j], step);
}
// Rows reach to the next 16 columns.
__device__ __forceinline__ void restore16(const uint8_t* data, const uint8_t* scales, bool e4m3, int col, float2 (&v)[8]) {
  decode16(*reinterpret_cast<const uint4*>(data + col), scales[col / kCkptBlock], e4m3, v);
}
// v rho as a sum of bf16 parts, `pitch` elements from one to the next: all but the last cut
// off behind their 8 bits, so that every part has the value's sign. Parts of a value other than
// zero are none of them zero, either (but 2^-133), so that an infinite dy times the parts is an
// infinity as the value itself gives it, not inf - inf or inf * 0.
__device__ __forceinline__ void store16(uint16_t* p, const float2 (&v)[8], float2 rho, int parts, int64_t pitch) {
  float2 x[8];
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = mul2(v[j], rho), w[j] = 0;
  for (;; p += pitch) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t cut = __byte_perm(__float_as_uint(x[j].x), __float_as_uint(x[j].y), 0x7632);
      const uint32_t part = parts > 1 ? cut : pack_bf16(x[j]), before = w[j];
      w[j] = part | (!(part & 0x7fffu) && (before & 0x7fffu) ? 1u : 0u) | (!(part & 0x7fff0000u) && (before & 0x7fff0000u) ? 0x10000u : 0u);
    }
    reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (--parts <= 0) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 hi = unpack_bf16(w[j]);
      x[j] = make_float2(copysignf(x[j].x - hi.x, x[j].x), copysignf(x[j].y - hi.y, x[j].y));
    }
  }
}
template <bool NORM>
__global__ void __launch_bounds__(256, NORM ? 2 : 5) operand_kernel(const __grid_constant__ OperandArgs a) {
  __shared__ float words[8];
  let_next_start();
  wait_for_previous();
  if (blockIdx.x >= a.row_blocks) {
    const int units = (a.dy_cols + 7) / 8;
    for (int64_t r = blockIdx.x - a.row_blocks; r < a.rows; r += gridDim.x - a.row_blocks)
      for (int u = threadIdx.x; u < units; u += 256) {
        const uint16_t* p = a.dy + r * a.dy_ld + 8 * u;
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 8 * u + i < a.dy_cols ? p[i] : 0u;
        *reinterpret_cast<uint4*>(a.dy_out + r * a.dy_out_ld + 8 * u) =
            make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
      }
    return;
  }
  const int tid = threadIdx.x & (a.threads - 1), at_once = 256 / a.threads;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * at_once; first < a.rows; first += static_cast<int64_t>(a.row_blocks) * at_once) {
    const int64_t row = first + threadIdx.x / a.threads;
    const bool mine = row < a.rows;  // whole warps; with 256 threads a row all of them
    const uint8_t *data = a.in.data + row * a.in.stride, *scales = a.in.scales + row * a.in.scale_stride;
    uint16_t* const x = a.x + row * a.x_ld;
    const int parts = NORM ? a.parts : 1;
    const int64_t pitch = a.rows * a.x_ld;
    float2 rho = both(1.0f);
    const bool once = a.cols <= 64 * a.threads;  // a thread's part of the row stays in registers
    float2 v[NORM ? 4 : 1][8];
    if (NORM) {
      float2 sums = both(0.0f);
      auto add = [&](int col, float2 (&x)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (col + 2 * j >= a.cols) x[j].x = 0.0f;  // what lies behind the row may be anything
          if (col + 2 * j + 1 >= a.cols) x[j].y = 0.0f;
          sums = fma2(x[j], x[j], sums);
        }
      };
      if (mine && once) {
        uint4 q[4];
        uint8_t s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 16 * (tid + i * a.threads);
          if (col < a.cols) q[i] = *reinterpret_cast<const uint4*>(data + col), s[i] = scales[col / kCkptBlock];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 16 * (tid + i * a.threads);
          if (col < a.cols) {
            decode16(q[i], s[i], a.in.e4m3, v[NORM ? i : 0]);
            add(col, v[NORM ? i : 0]);
          }
        }
      } else if (mine) {
        for (int col = 16 * tid; col < a.cols; col += 16 * a.threads) {
          restore16(data, scales, a.in.e4m3, col, v[0]);
          add(col, v[0]);
        }
      }
      float s = sums.x + sums.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (a.threads == 256) {
        __syncthreads();
        if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = s;
        __syncthreads();
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += words[i];
      }
      rho = both(rsqrtf(s / static_cast<float>(a.cols) + a.eps));
      if (mine && once) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 16 * (tid + i * a.threads);
          if (col < a.cols) store16(x + col, v[NORM ? i : 0], rho, parts, pitch);
        }
        continue;
      }
    }
    if (!mine) continue;
#pragma unroll 2
    for (int col = 16 * tid; col < a.cols; col += 16 * a.threads) {
      restore16(data, scales, a.in.e4m3, col, v[0]);
      store16(x + col, v[0], rho, parts, pitch);
    }
  }
}

// dw = the sum of the products' partial sums, times the weight of the column, added to dw or
// not; 4 columns a thread.
struct FinishArgs {
  const float* part;
  int64_t ld, split_stride;
  const void* weight;
  void* dw;
  int64_t dw_ld;
  int32_t splits, weight_f32, dw_f32, accumulate, cols;
  int64_t rows;
  int32_t vec;
};
__global__ void __launch_bounds__(256) wgrad_finish_kernel(const __grid_constant__ FinishArgs a) {
  let_next_start();
  wait_for_previous();
  const int quads = (a.cols + 3) / 4;
  const int64_t total = a.rows * quads;
  for (int64_t t = blockIdx.x * int64_t(256) + threadIdx.x; t < total; t += int64_t(256) * gridDim.x) {
    const int64_t row = t / quads;
    const int col = 4 * static_cast<int>(t - row * quads);
    const float* p = a.part + row * a.ld + col;  // ld is a multiple of 4
    float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int k = 0; k < a.splits; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(p + k * a.split_stride);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    float d[4] = {s.x, s.y, s.z, s.w};
    const int n = min(4, a.cols - col);
    if (a.weight)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n)
          d[j] *= a.weight_f32 ? static_cast<const float*>(a.weight)[col + j]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(a.weight)[col + j]);
    if (n == 4 && a.vec == 16 && !a.accumulate) {
      if (a.dw_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.dw) + row * a.dw_ld + col) = make_float4(d[0], d[1], d[2], d[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.dw) + row * a.dw_ld + col) =
            make_uint2(pack_bf16(make_float2(d[0], d[1])), pack_bf16(make_float2(d[2], d[3])));
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j >= n) break;
      if (a.dw_f32) {
        float* q = static_cast<float*>(a.dw) + row * a.dw_ld + col + j;
        *q = a.accumulate ? *q + d[j] : d[j];
      } else {
        __nv_bfloat16* q = static_cast<__nv_bfloat16*>(a.dw) + row * a.dw_ld + col + j;
        *q = __float2bfloat16_rn(a.accumulate ? __bfloat162float(*q) + d[j] : d[j]);
      }
    }
  }
}

Kept kept_arg(const lst_checkpoint* c) {
  return {static_cast<uint8_t*>(c->data), static_cast<uint8_t*>(c->scales), c->stride, c->scale_stride,
          c->format == LST_CHECKPOINT_E4M3};
}
bool on16(const lst_matrix* m) {
  return reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && (m->rows <= 1 || m->stride * dtype_bytes(m->dtype) % 16 == 0);
}
// Rows that tile loads take.
bool tile_rows(const lst_matrix* m) { return reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && m->stride % 8 == 0; }
unsigned warp_grid(int64_t tasks) { return static_cast<unsigned>(std::min(ops_ceil_div(tasks, 8), kSms * 8)); }

template <class T>
cudaError_t launch_save(const lst_matrix* x, const lst_checkpoint* c, bool vec, cudaStream_t stream) {
  const int64_t parts = ops_ceil_div(x->cols, kWarpColumns);
  return launch_chained(vec ? save_kernel<T, true> : save_kernel<T, false>, dim3(warp_grid(x->rows * parts)), dim3(256), 0, stream,
                        static_cast<const T*>(x->data), x->stride, kept_arg(c), x->rows, static_cast<int>(x->cols),
                        static_cast<int>(parts));
}
template <class T>
cudaError_t launch_restore(const lst_checkpoint* c, T* out, int64_t ld, bool vec, cudaStream_t stream) {
  const int64_t parts = ops_ceil_div(c->cols, kWarpColumns);
  return launch_chained(vec ? restore_kernel<T, true> : restore_kernel<T, false>, dim3(warp_grid(c->rows * parts)), dim3(256), 0,
                        stream, kept_arg(c), out, ld, c->rows, static_cast<int>(c->cols), static_cast<int>(parts));
}

lst_status check_pair(const lst_matrix* m, const char* name, const lst_checkpoint* c, const char* cname, const char* who) {
  LST_TRY(check_matrix(m, name, who));
  LST_TRY(check_checkpoint(c, cname, who));
  if (m->rows != c->rows || m->cols != c->cols)
    return fail(LST_ERR_INVALID_ARG, "%s: %s and %s must have one shape", who, name, cname);
  return LST_OK;
}

bool wgrad_sizes_fit(int64_t n, int64_t o, int64_t h) {
  // the kernels step past the last column in 32 bits, by at most 16 columns of 256 threads
  const int64_t most = int64_t(1) << 40, widest = (int64_t(1) << 31) - (1 << 14);
  return n > 0 && o > 0 && h > 0 && n <= (int64_t(1) << 24) && o <= widest && h <= widest && o <= most / n && h <= most / n &&
         o <= most / h;
}

// Normed rows go into the product as sums of bf16 parts, each with all of dy: two for a bf16
// result (2^-15 of a value is left at most, far below the result's own rounding), three for fp32 (all 24
// bits). One part would leave up to 2^-8 of every value, which no number of tokens averages out
// of the result's relative error. Values as they are kept are exact in one.
// 4096 x 256 x 2048: 26 us with two parts and 35 with three, 20 with one, whose bf16 result was
// off by 0.0024 (0.0017 is its rounding) and whose fp32 one by 0.0017, with three 4e-6 (the sums
// on the tensor cores); 8192 x 11008 x 4096: 832 and 1304 us, 452 with one.
int wgrad_parts(bool norm, const lst_matrix* dw) { return !norm ? 1 : dw->dtype == LST_F32 ? 3 : 2; }

struct WgradPlan {
  int64_t blocks, splits, part_ld, dy_ld, x_ld, dy_off, x_off, part_off, bytes;  // blocks: steps of 64 tokens of the product
};
// Sums are split where tiles of 128 columns leave half of the 76 CTA pairs idle, into ranges of
// at least 8 steps. Sizes of memory are those of any smaller count, too, with or without a norm.
int64_t wgrad_splits(int64_t blocks, int64_t o, int64_t h) {
  const int64_t tiles = ops_ceil_div(o, kGemmTile) * ops_ceil_div(h, kGemmTile / 2);
  return std::max<int64_t>(1, std::min<int64_t>(blocks / 8, 76 / tiles));
}
WgradPlan wgrad_plan(const lst_matrix* dy, const lst_checkpoint* c, const lst_matrix* dw, bool norm) {
  WgradPlan p;
  const int64_t n = dy->rows, o = dy->cols, h = c->cols, most = wgrad_parts(true, dw);
  p.blocks = wgrad_parts(norm, dw) * ops_ceil_div(n, 64);
  p.splits = wgrad_splits(p.blocks, o, h);
  p.part_ld = ops_round_up(h, 32);
  p.dy_ld = ops_round_up(o, 8);
  p.x_ld = ops_round_up(h, 16);
  int64_t at = 0;
  auto take = [&](int64_t size) {
    const int64_t off = at;
    at += ops_round_up(size, 256);
    return off;
  };
  const int64_t splits = wgrad_splits(most * ops_ceil_div(n, 64), o, h);
  p.dy_off = take(tile_rows(dy) ? 0 : n * p.dy_ld * 2);
  p.x_off = take(most * n * p.x_ld * 2);
  p.part_off = take(splits > 1 ? splits * o * p.part_ld * 4 : 0);
  p.bytes = at;
  return p;
}

}  // namespace
}  // namespace lst

using namespace lst;

extern "C" lst_status lst_checkpoint_save(const lst_matrix* x, const lst_checkpoint* out, void* cuda_stream) {
  clear_error();
  const char* who = "lst_checkpoint_save";
  LST_TRY(check_pair(x, "x", out, "out", who));
  if (x->rows == 0 || x->cols == 0) return LST_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  const bool vec = x->cols % 8 == 0 && on16(x);
  LST_TRY_CUDA(x->dtype == LST_F32 ? launch_save<float>(x, out, vec, stream) : launch_save<__nv_bfloat16>(x, out, vec, stream), who);
  return LST_OK;
}

extern "C" lst_status lst_checkpoint_restore(const lst_checkpoint* c, const lst_matrix* out, void* cuda_stream) {
  clear_error();
  const char* who = "lst_checkpoint_restore";
  LST_TRY(check_pair(out, "out", c, "c", who));
  if (out->rows == 0 || out->cols == 0) return LST_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  const bool vec = out->cols % 8 == 0 && on16(out);
  LST_TRY_CUDA(out->dtype == LST_F32
                   ? launch_restore<float>(c, static_cast<float*>(out->data), out->stride, vec, stream)
                   : launch_restore<__nv_bfloat16>(c, static_cast<__nv_bfloat16*>(out->data), out->stride, vec, stream),
               who);
  return LST_OK;
}

extern "C" int64_t lst_checkpoint_wgrad_workspace_bytes(const lst_matrix* dy, const lst_checkpoint* c, const lst_matrix* dw) {
  if (!dy || !c || !dw || dy->rows != c->rows || dw->rows != dy->cols || dw->cols != c->cols ||
      !wgrad_sizes_fit(dy->rows, dy->cols, c->cols))
    return 0;
  return wgrad_plan(dy, c, dw, false).bytes;
}

extern "C" lst_status lst_checkpoint_wgrad(const lst_matrix* dy, const lst_checkpoint* c, const lst_matrix* norm_weight,
                                           float eps, const lst_matrix* dw, int32_t accumulate, void* workspace,
                                           int64_t workspace_bytes, void* cuda_stream) {
  clear_error();
  const char* who = "lst_checkpoint_wgrad";
  LST_TRY(check_matrix(dy, "dy", who));
  LST_TRY(check_checkpoint(c, "c", who));
  LST_TRY(check_matrix(dw, "dw", who));
  if (dy->dtype != LST_BF16) return fail(LST_ERR_INVALID_ARG, "%s: dy must be bf16", who);
  if (dy->rows != c->rows || dw->rows != dy->cols || dw->cols != c->cols)
    return fail(LST_ERR_INVALID_ARG, "%s: dy must be tokens x out, c tokens x cols, dw out x cols", who);
  if (norm_weight) {
    LST_TRY(check_matrix(norm_weight, "norm_weight", who));
    if (norm_weight->rows != 1 || norm_weight->cols != c->cols)
      return fail(LST_ERR_INVALID_ARG, "%s: norm_weight must be 1 x cols", who);
    if (!(eps > 0.0f) || !std::isfinite(eps)) return fail(LST_ERR_INVALID_ARG, "%s: eps must be above zero and finite", who);
  }
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  if (dw->rows == 0 || dw->cols == 0) return LST_OK;
  if (dy->rows == 0) {
    const size_t size = dtype_bytes(dw->dtype);
    if (!accumulate)
      LST_TRY_CUDA(cudaMemset2DAsync(dw->data, static_cast<size_t>(dw->stride) * size, 0, static_cast<size_t>(dw->cols) * size,
                                     static_cast<size_t>(dw->rows), stream),
                   who);
    return LST_OK;
  }
  const int64_t n = dy->rows, o = dy->cols, h = c->cols;
  if (!wgrad_sizes_fit(n, o, h))
    return fail(LST_ERR_INVALID_ARG, "%s: more than 2^24 tokens, 2^31 - 2^14 columns or outputs, or 2^40 elements of an operand", who);
  const WgradPlan p = wgrad_plan(dy, c, dw, norm_weight != nullptr);
  const int parts = wgrad_parts(norm_weight != nullptr, dw);
  LST_TRY(check_workspace(workspace, workspace_bytes, p.bytes, who));
  char* ws = static_cast<char*>(workspace);
  const bool pack = !tile_rows(dy);
  // a warp a row where there are rows for all of them, but normed rows are to stay in registers
  const int threads = h <= 1024 || (n >= kSms * 8 && (!norm_weight || h <= 2048)) ? 32 : 256;
  const int64_t row_blocks = std::min(ops_ceil_div(n, 256 / threads), kSms * 8);
  const OperandArgs x = {kept_arg(c), reinterpret_cast<uint16_t*>(ws + p.x_off), p.x_ld, n, static_cast<int32_t>(h),
                         threads, static_cast<int32_t>(row_blocks), eps, static_cast<const uint16_t*>(dy->data),
                         reinterpret_cast<uint16_t*>(ws + p.dy_off), dy->stride, p.dy_ld, static_cast<int32_t>(o), parts};
  LST_TRY_CUDA(launch_chained(norm_weight ? operand_kernel<true> : operand_kernel<false>, dim3(static_cast<unsigned>(row_blocks + (pack ? std::min(n, kSms * 8) : 0))), dim3(256), 0, stream, x), who);
  GemmProblem g;
  if (pack)
    g.a = {x.dy_out, o, n, p.dy_ld, true};
  else
    g.a = {dy->data, o, n, dy->stride, true};
  g.b = {x.x, h, n, p.x_ld, true, parts, n * p.x_ld};
  g.m = o;
  g.n = h;
  g.k = p.blocks * 64;
  g.parts = parts;
  g.splits = static_cast<int>(p.splits);
  const bool weight_f32 = norm_weight && norm_weight->dtype == LST_F32;
  const int vec = on16(dw) && dw->stride * dtype_bytes(dw->dtype) % 16 == 0 ? 16 : 2;
  g.wgrad = {dw->data, dw->stride, norm_weight ? norm_weight->data : nullptr, dw->dtype == LST_F32, weight_f32, accumulate != 0, vec, {}};
  if (p.splits > 1) g.wgrad.partial = {reinterpret_cast<float*>(ws + p.part_off), p.part_ld, o * p.part_ld, 0};
  LST_TRY_CUDA(launch_gemm(GEMM_BF16_WGRAD, &g, 1, stream), who);
  if (p.splits == 1) return LST_OK;
  const int64_t splits = ops_ceil_div(p.blocks, ops_ceil_div(p.blocks, p.splits));
  const FinishArgs f = {g.wgrad.partial.out, p.part_ld, o * p.part_ld, g.wgrad.weight, dw->data, dw->stride, static_cast<int32_t>(splits),
                        weight_f32, dw->dtype == LST_F32, accumulate != 0, static_cast<int32_t>(h), o, vec};
  const int64_t quads = ops_ceil_div(h, 4);
  LST_TRY_CUDA(launch_chained(wgrad_finish_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(ops_ceil_div(o * quads, 256), kSms * 8))),
                              dim3(256), 0, stream, f),
               who);
  return LST_OK;
}
