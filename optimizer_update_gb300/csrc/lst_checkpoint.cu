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
constexpr int kWarpColumns = 512;  // of a row, per warp and turn

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
    Unit u[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      u[k].fill(0.0f);
      if (c.has(k)) c.load(x + row * ld + col, k, u[k]);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
      c.save(u[k], k, out.data + row * out.stride + col, out.scales + row * out.scale_stride + col / kCkptBlock, out.e4m3);
  }
}

// With `rho` (a factor per row) and `weight` (per column, or null): the norm of the row.
template <class T, bool VEC>
__global__ void __launch_bounds__(256)
    restore_kernel(Kept in, T* __restrict__ out, int64_t ld, int64_t rows, int cols, int parts, const float* __restrict__ rho) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8, tasks = rows * parts;
  for (int64_t t = blockIdx.x * 8 + (threadIdx.x >> 5); t < tasks; t += warps) {
    const int64_t row = t / parts;
    const int col = static_cast<int>(t - row * parts) * kWarpColumns;
    const Cols<VEC> c = {static_cast<uint32_t>(lane), 32u, static_cast<uint32_t>(min(cols - col, kWarpColumns))};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!c.has(k)) continue;
      Unit u;
      c.restore(in.data + row * in.stride + col, in.scales + row * in.scale_stride + col / kCkptBlock, in.e4m3, k, u);
      if (rho) {
        const float2 r = both(rho[row]);
#pragma unroll
        for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], r);
      }
      c.store(out + row * ld + col, k, u);
    }
  }
}

// rho[row] = rsqrt(mean of the restored row's squares + eps), a warp a row.
template <bool VEC>
__global__ void __launch_bounds__(256) rho_kernel(Kept in, int64_t rows, int cols, float eps, float* __restrict__ rho) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  for (int64_t row = blockIdx.x * 8 + (threadIdx.x >> 5); row < rows; row += static_cast<int64_t>(gridDim.x) * 8) {
    float2 sums = both(0.0f);
    for (int col = 0; col < cols; col += kWarpColumns) {
      const Cols<VEC> c = {static_cast<uint32_t>(lane), 32u, static_cast<uint32_t>(min(cols - col, kWarpColumns))};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!c.has(k)) continue;
        Unit u;
        c.restore(in.data + row * in.stride + col, in.scales + row * in.scale_stride + col / kCkptBlock, in.e4m3, k, u);
#pragma unroll
        for (int j = 0; j < 4; ++j) sums = fma2(u.v[j], u.v[j], sums);
      }
    }
    float s = sums.x + sums.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) rho[row] = __frsqrt_rn(s / static_cast<float>(cols) + eps);
  }
}

// Rows of dy at a pitch that is a multiple of 16 bytes.
__global__ void __launch_bounds__(256)
    pack_rows_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t rows, int cols, uint16_t* __restrict__ dst,
                     int64_t dst_ld) {
  let_next_start();
  wait_for_previous();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += 256) dst[r * dst_ld + c] = src[r * ld + c];
}

// dw = the sum of the products' partial sums, times the weight of the column, added to dw or not.
struct FinishArgs {
  const float* part;
  int64_t ld, split_stride;
  const void* weight;
  void* dw;
  int64_t dw_ld;
  int32_t splits, weight_f32, dw_f32, accumulate, cols;
  int64_t rows;
};
__global__ void __launch_bounds__(256) wgrad_finish_kernel(const __grid_constant__ FinishArgs a) {
  let_next_start();
  wait_for_previous();
  const int64_t total = a.rows * a.cols;
  for (int64_t t = blockIdx.x * int64_t(256) + threadIdx.x; t < total; t += int64_t(256) * gridDim.x) {
    const int64_t row = t / a.cols;
    const int col = static_cast<int>(t - row * a.cols);
    const float* p = a.part + row * a.ld + col;
    float s = 0.0f;
    for (int k = 0; k < a.splits; ++k) s += p[k * a.split_stride];
    if (a.weight)
      s *= a.weight_f32 ? static_cast<const float*>(a.weight)[col]
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(a.weight)[col]);
    if (a.dw_f32) {
      float* q = static_cast<float*>(a.dw) + row * a.dw_ld + col;
      *q = a.accumulate ? *q + s : s;
    } else {
      __nv_bfloat16* q = static_cast<__nv_bfloat16*>(a.dw) + row * a.dw_ld + col;
      *q = __float2bfloat16_rn(a.accumulate ? __bfloat162float(*q) + s : s);
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
unsigned warp_grid(int64_t tasks) { return static_cast<unsigned>(std::min(ops_ceil_div(tasks, 8), kSms * 8)); }

template <class T>
cudaError_t launch_save(const lst_matrix* x, const lst_checkpoint* c, bool vec, cudaStream_t stream) {
  const int64_t parts = ops_ceil_div(x->cols, kWarpColumns);
  return launch_chained(vec ? save_kernel<T, true> : save_kernel<T, false>, dim3(warp_grid(x->rows * parts)), dim3(256), 0, stream,
                        static_cast<const T*>(x->data), x->stride, kept_arg(c), x->rows, static_cast<int>(x->cols),
                        static_cast<int>(parts));
}
template <class T>
cudaError_t launch_restore(const lst_checkpoint* c, T* out, int64_t ld, bool vec, const float* rho, cudaStream_t stream) {
  const int64_t parts = ops_ceil_div(c->cols, kWarpColumns);
  return launch_chained(vec ? restore_kernel<T, true> : restore_kernel<T, false>, dim3(warp_grid(c->rows * parts)), dim3(256), 0,
                        stream, kept_arg(c), out, ld, c->rows, static_cast<int>(c->cols), static_cast<int>(parts), rho);
}

lst_status check_pair(const lst_matrix* m, const char* name, const lst_checkpoint* c, const char* cname, const char* who) {
  LST_TRY(check_matrix(m, name, who));
  LST_TRY(check_checkpoint(c, cname, who));
  if (m->rows != c->rows || m->cols != c->cols)
    return fail(LST_ERR_INVALID_ARG, "%s: %s and %s must have one shape", who, name, cname);
  return LST_OK;
}

bool wgrad_sizes_fit(int64_t n, int64_t o, int64_t h) {
  const int64_t most = int64_t(1) << 40;
  return n > 0 && o > 0 && h > 0 && n <= (int64_t(1) << 24) && o <= INT32_MAX && h <= INT32_MAX && o <= most / n && h <= most / n &&
         o <= most / h;
}

struct WgradPlan {
  int64_t splits, part_ld, dy_ld, x_ld, rho_off, dy_off, x_off, part_off, bytes;
};
WgradPlan wgrad_plan(const lst_matrix* dy, const lst_checkpoint* c, const lst_matrix* dw) {
  (void)dw;
  WgradPlan p;
  const int64_t n = dy->rows, o = dy->cols, h = c->cols;
  const int64_t blocks = ops_ceil_div(n, 64), tiles = ops_ceil_div(o, kGemmTile) * ops_ceil_div(h, kGemmTile);
  p.splits = std::max<int64_t>(1, std::min<int64_t>({32, blocks / 8, 152 / tiles}));
  p.part_ld = ops_round_up(h, 32);
  p.dy_ld = ops_round_up(o, 8);
  p.x_ld = ops_round_up(h, 8);
  int64_t at = 0;
  auto take = [&](int64_t size) {
    const int64_t off = at;
    at += ops_round_up(size, 256);
    return off;
  };
  p.rho_off = take(n * 4);
  p.dy_off = take(on16(dy) && dy->stride % 8 == 0 ? 0 : n * p.dy_ld * 2);
  p.x_off = take(n * p.x_ld * 2);
  p.part_off = take(p.splits * o * p.part_ld * 4);
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
                   ? launch_restore<float>(c, static_cast<float*>(out->data), out->stride, vec, nullptr, stream)
                   : launch_restore<__nv_bfloat16>(c, static_cast<__nv_bfloat16*>(out->data), out->stride, vec, nullptr, stream),
               who);
  return LST_OK;
}

extern "C" int64_t lst_checkpoint_wgrad_workspace_bytes(const lst_matrix* dy, const lst_checkpoint* c, const lst_matrix* dw) {
  if (!dy || !c || !dw || dy->rows != c->rows || dw->rows != dy->cols || dw->cols != c->cols ||
      !wgrad_sizes_fit(dy->rows, dy->cols, c->cols))
    return 0;
  return wgrad_plan(dy, c, dw).bytes;
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
    return fail(LST_ERR_INVALID_ARG, "%s: more than 2^24 tokens, or an operand of more than 2^40 elements", who);
  const WgradPlan p = wgrad_plan(dy, c, dw);
  LST_TRY(check_workspace(workspace, workspace_bytes, p.bytes, who));
  char* ws = static_cast<char*>(workspace);
  float* rho = norm_weight ? reinterpret_cast<float*>(ws + p.rho_off) : nullptr;
  if (rho)
    LST_TRY_CUDA(launch_chained(h % 8 == 0 ? rho_kernel<true> : rho_kernel<false>, dim3(warp_grid(n)), dim3(256), 0, stream,
                                kept_arg(c), n, static_cast<int>(h), eps, rho),
                 who);
  const void* dyp = dy->data;
  int64_t dy_ld = dy->stride;
  if (!(on16(dy) && dy->stride % 8 == 0)) {
    dyp = ws + p.dy_off;
    dy_ld = p.dy_ld;
    LST_TRY_CUDA(launch_chained(pack_rows_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(n, 8192))), dim3(256), 0, stream,
                                static_cast<const uint16_t*>(dy->data), dy->stride, n, static_cast<int>(o),
                                reinterpret_cast<uint16_t*>(ws + p.dy_off), p.dy_ld),
                 who);
  }
  __nv_bfloat16* x = reinterpret_cast<__nv_bfloat16*>(ws + p.x_off);
  LST_TRY_CUDA(launch_restore<__nv_bfloat16>(c, x, p.x_ld, h % 8 == 0, rho, stream), who);
  GemmProblem g;
  g.a = {dyp, o, n, dy_ld, true};
  g.b = {x, h, n, p.x_ld, true};
  g.m = o;
  g.n = h;
  g.k = n;
  g.splits = static_cast<int>(p.splits);
  g.partial = {reinterpret_cast<float*>(ws + p.part_off), p.part_ld, o * p.part_ld, 0};
  LST_TRY_CUDA(launch_gemm(GEMM_BF16, &g, 1, stream), who);
  const int64_t blocks = ops_ceil_div(n, 64), splits = ops_ceil_div(blocks, ops_ceil_div(blocks, p.splits));
  const FinishArgs f = {g.partial.out, p.part_ld, o * p.part_ld, norm_weight ? norm_weight->data : nullptr, dw->data, dw->stride,
                        static_cast<int32_t>(splits), norm_weight && norm_weight->dtype == LST_F32, dw->dtype == LST_F32,
                        accumulate != 0, static_cast<int32_t>(h), o};
  LST_TRY_CUDA(launch_chained(wgrad_finish_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(ops_ceil_div(o * h, 256), kSms * 8))),
                              dim3(256), 0, stream, f),
               who);
  return LST_OK;
}
