// The residual stream between two layers: norm of the block's output, gate, scales
// and sum, norm of the sum, with 8-bit checkpoints of what the backward pass reads,
// and the gradients of all that.
//
// Forward, row by row: u = y tau w_post (tau = rsqrt(mean y^2 + eps)), h = a x + b g u,
// z = h rho w_pre (rho = rsqrt(mean h^2 + eps)). A CTA holds a row in registers: it
// is read once and h, z and the checkpoints are written from there.
//
// Backward: with m = w_pre dz
//   D  = dh + rho (m - h rho^2 mean(m h)),  dx = a D,  dw_pre = sum dz h rho
//   e  = b D g w_post,  dy = tau (e - y tau^2 mean(e y))
//   A  = sum D tau y over the tokens of a gate row;  dgate = b w_post A,  dw_post = b sum g A
// so two sums per column (A and dw_pre's) give all three parameter gradients. A CTA
// takes consecutive rows and keeps the column sums in registers; they go to the
// workspace once per CTA (A once per gate row) and are added up in order by a second launch.
//
// Both are bound by memory: 8 bytes an element forward, 12 backward in bf16 (10 with
// checkpoints) against some 20 operations.
#include <algorithm>
#include <cmath>

#include "lst_ckpt.cuh"

namespace lst {

namespace {

constexpr int64_t kMaxHidden = 16384;
constexpr int64_t kSms = 152;

struct Rows {
  void* p;
  int64_t stride;  // elements
};
struct Weights {
  const void* p;
  int64_t stride;
  int32_t f32;
};
struct Kept {
  uint8_t* data;
  uint8_t* scales;
  int64_t stride, scale_stride;
  int32_t e4m3;
};
template <class T>
__device__ __forceinline__ T* row_of(const Rows& m, int64_t r) {
  return static_cast<T*>(m.p) + r * m.stride;
}
__device__ __forceinline__ const void* row_of(const Weights& w, int64_t r) {
  return static_cast<const char*>(w.p) + r * w.stride * (w.f32 ? 4 : 2);
}

// Sum of each of the M values over the CTA's threads, in every thread. `turn` alternates
// between the two halves of `words`, so that one barrier a call is enough.
template <int M>
__device__ __forceinline__ void cta_sum(float (&v)[M], float (*words)[M][32], int& turn) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
  for (int j = 0; j < M; ++j)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  if (warps == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int j = 0; j < M; ++j) words[turn][j][warp] = v[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < M; ++j) {
    v[j] = lane < warps ? words[turn][j][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
  }
  turn ^= 1;
}

struct NormArgs {
  Rows x, y, h, z;
  Weights gate, w_post, w_pre;
  Kept h8, y8;
  int64_t tokens, per_gate;  // tokens of a gate row
  int32_t hidden;
  float alpha, beta, eps;
};

template <class T, bool VEC, int K>
__global__ void __launch_bounds__(512) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float words[2][1][32];
  let_next_start();
  wait_for_previous();
  const Cols<VEC, K> c = {static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.hidden};
  const float inverse = 1.0f / static_cast<float>(a.hidden);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.tokens; row += gridDim.x) {
    float h[K][8], y[K][8], w[K][8];
    c.load(row_of<T>(a.x, row), h);
    if (a.y.p) {
      c.load(row_of<T>(a.y, row), y);
      if (a.y8.data)
        c.save(y, a.y8.data + row * a.y8.stride, a.y8.scales + row * a.y8.scale_stride, a.y8.e4m3);
      if (a.w_post.p) {
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] = __fmaf_rn(y[k][i], y[k][i], s[0]);
        cta_sum(s, words, turn);
        const float tau = __frsqrt_rn(s[0] * inverse + a.eps);
        c.load_any(a.w_post.p, a.w_post.f32, w);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[k][i] = y[k][i] * tau * w[k][i];
      }
      if (a.gate.p) {
        c.load_any(row_of(a.gate, row / a.per_gate), a.gate.f32, w);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) y[k][i] = y[k][i] * w[k][i];
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = a.alpha * h[k][i] + a.beta * y[k][i];
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = a.alpha * h[k][i];
    }
    if (a.h.p) c.store(row_of<T>(a.h, row), h);
    if (a.h8.data) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[k][i] = round_to(h[k][i], static_cast<const T*>(nullptr));
      c.save(w, a.h8.data + row * a.h8.stride, a.h8.scales + row * a.h8.scale_stride, a.h8.e4m3);
    }
    if (a.z.p) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = __fmaf_rn(h[k][i], h[k][i], s[0]);
      cta_sum(s, words, turn);
      const float rho = __frsqrt_rn(s[0] * inverse + a.eps);
      c.load_any(a.w_pre.p, a.w_pre.f32, w);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * rho * w[k][i];
      c.store(row_of<T>(a.z, row), h);
    }
  }
}

struct GradArgs {
  Rows dh, dz, h, y, dx, dy;
  Kept h8, y8;
  Weights gate, w_post, w_pre;
  void* dgate;
  int64_t dgate_stride;
  int32_t dgate_f32, accumulate;
  // sums over a CTA's rows: of dw_pre and dw_post [cta][hidden], of dgate [2 cta + (0: its first gate row)][hidden]
  float *part_pre, *part_post, *part_gate;
  int64_t tokens, per_gate;
  int32_t hidden, ctas;
  float alpha, beta, eps;
};

__device__ __forceinline__ void store_sum(void* p, int64_t at, bool f32, bool accumulate, float v) {
  if (f32) {
    float* q = static_cast<float*>(p) + at;
    *q = accumulate ? *q + v : v;
  } else {
    __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + at;
    *q = __float2bfloat16_rn(accumulate ? __bfloat162float(*q) + v : v);
  }
}

// First row of CTA c: the rows divided evenly.
__host__ __device__ __forceinline__ int64_t first_row(int64_t c, int64_t tokens, int64_t ctas) { return c * tokens / ctas; }

template <class T, bool VEC, int K>
__global__ void __launch_bounds__(512) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float words[2][2][32];
  let_next_start();
  wait_for_previous();
  const Cols<VEC, K> c = {static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), a.hidden};
  const float inverse = 1.0f / static_cast<float>(a.hidden);
  const int64_t cta = blockIdx.x;
  const int64_t begin = first_row(cta, a.tokens, a.ctas), end = first_row(cta + 1, a.tokens, a.ctas);
  const bool per_token = a.gate.p && a.per_gate == 1;
  float sum_pre[K][8] = {}, sum_a[K][8] = {}, sum_post[K][8] = {};
  int turn = 0;
  for (int64_t row = begin; row < end; ++row) {
    float d[K][8], h[K][8], w[K][8], y[K][8], g[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) d[k][i] = 0.0f, g[k][i] = 1.0f;
    if (a.dh.p) c.load(row_of<T>(a.dh, row), d);
    if (a.dz.p) {
      if (a.h8.data)
        c.restore(a.h8.data + row * a.h8.stride, a.h8.scales + row * a.h8.scale_stride, a.h8.e4m3, h);
      else
        c.load(row_of<T>(a.h, row), h);
      float m[K][8];
      c.load(row_of<T>(a.dz, row), m);
      c.load_any(a.w_pre.p, a.w_pre.f32, w);
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] = __fmaf_rn(h[k][i], h[k][i], s[0]);
          s[1] = __fmaf_rn(m[k][i] * w[k][i], h[k][i], s[1]);
        }
      cta_sum(s, words, turn);
      const float rho = __frsqrt_rn(s[0] * inverse + a.eps), back = rho * rho * (s[1] * inverse);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum_pre[k][i] = __fmaf_rn(m[k][i], h[k][i] * rho, sum_pre[k][i]);
          d[k][i] += rho * (m[k][i] * w[k][i] - h[k][i] * back);
        }
    }
    if (a.dx.p) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[k][i] = a.alpha * d[k][i];
      c.store(row_of<T>(a.dx, row), w);
    }
    if (a.gate.p) c.load_any(row_of(a.gate, row / a.per_gate), a.gate.f32, g);
    const bool has_y = a.y.p || a.y8.data;
    float tau = 1.0f;
    if (has_y) {
      if (a.y8.data)
        c.restore(a.y8.data + row * a.y8.stride, a.y8.scales + row * a.y8.scale_stride, a.y8.e4m3, y);
      else
        c.load(row_of<T>(a.y, row), y);
    }
    if (a.w_post.p) {
      c.load_any(a.w_post.p, a.w_post.f32, w);
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] = __fmaf_rn(y[k][i], y[k][i], s[0]);
          s[1] = __fmaf_rn(a.beta * d[k][i] * g[k][i] * w[k][i], y[k][i], s[1]);
        }
      cta_sum(s, words, turn);
      tau = __frsqrt_rn(s[0] * inverse + a.eps);
      const float back = tau * tau * (s[1] * inverse);
      if (a.dy.p) {
        float e[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) e[k][i] = tau * (a.beta * d[k][i] * g[k][i] * w[k][i] - y[k][i] * back);
        c.store(row_of<T>(a.dy, row), e);
      }
    } else if (a.dy.p) {
      float e[K][8];
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) e[k][i] = a.beta * d[k][i] * g[k][i];
      c.store(row_of<T>(a.dy, row), e);
    }
    if (!has_y) continue;
    if (per_token) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = d[k][i] * (y[k][i] * tau);
          sum_post[k][i] = __fmaf_rn(g[k][i], t, sum_post[k][i]);
          if (a.dgate && c.in(k, i))
            store_sum(a.dgate, row * a.dgate_stride + c.at(k, i), a.dgate_f32, a.accumulate,
                      a.beta * t * (a.w_post.p ? w[k][i] : 1.0f));
        }
      continue;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum_a[k][i] = __fmaf_rn(d[k][i], y[k][i] * tau, sum_a[k][i]);
    // the last row of a gate row, or of the CTA
    const int64_t group = a.gate.p ? row / a.per_gate : 0;
    if (row + 1 < end && (!a.gate.p || (row + 1) / a.per_gate == group)) continue;
    const bool whole = group * a.per_gate >= begin && (group + 1) * a.per_gate <= end;
    const int64_t slot = 2 * cta + (group == begin / a.per_gate ? 0 : 1);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum_post[k][i] = __fmaf_rn(g[k][i], sum_a[k][i], sum_post[k][i]);
        if (a.dgate && c.in(k, i)) {
          const float t = a.beta * sum_a[k][i] * (a.w_post.p ? w[k][i] : 1.0f);
          if (whole)
            store_sum(a.dgate, group * a.dgate_stride + c.at(k, i), a.dgate_f32, a.accumulate, t);
          else
            a.part_gate[slot * a.hidden + c.at(k, i)] = t;
        }
        sum_a[k][i] = 0.0f;
      }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c.in(k, i)) {
        if (a.part_pre) a.part_pre[cta * a.hidden + c.at(k, i)] = sum_pre[k][i];
        if (a.part_post) a.part_post[cta * a.hidden + c.at(k, i)] = a.beta * sum_post[k][i];
      }
}

// Adds up the CTAs' sums: blockIdx.y 0: dw_pre, 1: dw_post, 2 + r: gate row r, unless one
// CTA had all its rows. 32 columns a CTA, every 8th row of sums to a warp.
struct JoinArgs {
  const float *pre, *post, *gate;
  void *dw_pre, *dw_post, *dgate;
  int64_t dgate_stride, tokens, per_gate;
  int32_t pre_f32, post_f32, gate_f32, accumulate, hidden, ctas;
};
__global__ void __launch_bounds__(256) norm_join_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float words[8][33];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  const bool in = col < a.hidden;
  auto add = [&](const float* p, int64_t first, int64_t last, void* out, int64_t at, bool f32) {
    float s = 0.0f;
    if (in)
      for (int64_t c = first + warp; c < last; c += 8) s += p[c * a.hidden + col];
    words[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && in) {
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += words[i][lane];
      store_sum(out, at + col, f32, a.accumulate, s);
    }
    __syncthreads();
  };
  const int64_t which = blockIdx.y;
  if (which == 0) {
    if (a.dw_pre) add(a.pre, 0, a.ctas, a.dw_pre, 0, a.pre_f32);
    return;
  }
  if (which == 1) {
    if (a.dw_post) add(a.post, 0, a.ctas, a.dw_post, 0, a.post_f32);
    return;
  }
  // gate rows that more than one CTA worked on: CTA c's last one, where it begins in c and ends behind it
  const int64_t c0 = which - 2, begin = first_row(c0, a.tokens, a.ctas), end = first_row(c0 + 1, a.tokens, a.ctas);
  if (begin == end) return;
  const int64_t r = (end - 1) / a.per_gate;
  if (r * a.per_gate < begin || (r + 1) * a.per_gate <= end) return;
  float s = 0.0f;
  if (in && warp == 0) {
    for (int64_t c = c0; c < a.ctas && first_row(c, a.tokens, a.ctas) < (r + 1) * a.per_gate; ++c) {
      const int64_t b = first_row(c, a.tokens, a.ctas), e = first_row(c + 1, a.tokens, a.ctas);
      if (b == e) continue;
      const int64_t slot = 2 * c + (r == b / a.per_gate ? 0 : 1);
      s += a.gate[slot * a.hidden + col];
    }
    store_sum(a.dgate, r * a.dgate_stride + col, a.gate_f32, a.accumulate, s);
  }
}

// ---- host ------------------------------------------------------------------------
// Threads of a row: 8, 16 or 32 columns each.
struct Fit {
  int k, threads;
};
Fit fit(int64_t hidden) {
  const int k = hidden <= 2048 ? 1 : hidden <= 8192 ? 2 : 4;
  return {k, static_cast<int>(ops_round_up(ops_ceil_div(hidden, 8 * k), 32))};
}
int64_t grad_ctas(int64_t tokens, int64_t hidden) {
  return std::min(tokens, kSms * std::max<int64_t>(1, 512 / fit(hidden).threads));
}

bool on16(const lst_matrix* m) {
  return !m || (reinterpret_cast<uintptr_t>(m->data) % 16 == 0 && (m->rows <= 1 || m->stride * dtype_bytes(m->dtype) % 16 == 0));
}
Rows rows_arg(const lst_matrix* m) { return m ? Rows{m->data, m->stride} : Rows{nullptr, 0}; }
Weights weights_arg(const lst_matrix* m) {
  return m ? Weights{m->data, m->stride, m->dtype == LST_F32} : Weights{nullptr, 0, 0};
}
Kept kept_arg(const lst_checkpoint* c) {
  if (!c) return {nullptr, nullptr, 0, 0, 0};
  return {static_cast<uint8_t*>(c->data), static_cast<uint8_t*>(c->scales), c->stride, c->scale_stride,
          c->format == LST_CHECKPOINT_E4M3};
}

struct Shape {
  const char* who;
  int64_t tokens, hidden;
  int32_t dtype;

  // a tokens x hidden matrix of the call's type, or null
  lst_status rows(const lst_matrix* m, const char* name) const {
    if (!m) return LST_OK;
    LST_TRY(check_matrix(m, name, who));
    if (m->rows != tokens || m->cols != hidden) return fail(LST_ERR_INVALID_ARG, "%s: %s must be tokens x hidden", who, name);
    if (m->dtype != dtype) return fail(LST_ERR_INVALID_ARG, "%s: %s has another type than the other activations", who, name);
    return LST_OK;
  }
  lst_status kept(const lst_checkpoint* c, const char* name) const {
    if (!c) return LST_OK;
    LST_TRY(check_checkpoint(c, name, who));
    if (c->rows != tokens || c->cols != hidden) return fail(LST_ERR_INVALID_ARG, "%s: %s must be tokens x hidden", who, name);
    return LST_OK;
  }
  lst_status vector(const lst_matrix* m, const char* name) const {
    if (!m) return LST_OK;
    LST_TRY(check_matrix(m, name, who));
    if (m->rows != 1 || m->cols != hidden) return fail(LST_ERR_INVALID_ARG, "%s: %s must be 1 x hidden", who, name);
    return LST_OK;
  }
  lst_status gate(const lst_matrix* m, const char* name) const {
    if (!m) return LST_OK;
    LST_TRY(check_matrix(m, name, who));
    if (m->cols != hidden || m->rows < 1 || tokens % m->rows)
      return fail(LST_ERR_INVALID_ARG, "%s: %s must be rows x hidden with rows a divisor of the tokens", who, name);
    return LST_OK;
  }
  lst_status sizes(const lst_residual_params* p) const {
    if (hidden < 1 || hidden > kMaxHidden) return fail(LST_ERR_INVALID_ARG, "%s: hidden outside 1..16384", who);
    if (!p) return fail(LST_ERR_INVALID_ARG, "%s: params is null", who);
    if (!std::isfinite(p->residual_scale) || !std::isfinite(p->branch_scale))
      return fail(LST_ERR_INVALID_ARG, "%s: a scale is not finite", who);
    if (!(p->eps > 0.0f) || !std::isfinite(p->eps)) return fail(LST_ERR_INVALID_ARG, "%s: eps must be above zero and finite", who);
    return LST_OK;
  }
};

template <class Args>
using Kernel = void (*)(const Args);

template <class T>
Kernel<NormArgs> norm_of(bool vec, int k) {
  if (vec) return k == 1 ? norm_kernel<T, true, 1> : k == 2 ? norm_kernel<T, true, 2> : norm_kernel<T, true, 4>;
  return k == 1 ? norm_kernel<T, false, 1> : k == 2 ? norm_kernel<T, false, 2> : norm_kernel<T, false, 4>;
}
template <class T>
Kernel<GradArgs> norm_grad_of(bool vec, int k) {
  if (vec) return k == 1 ? norm_grad_kernel<T, true, 1> : k == 2 ? norm_grad_kernel<T, true, 2> : norm_grad_kernel<T, true, 4>;
  return k == 1 ? norm_grad_kernel<T, false, 1> : k == 2 ? norm_grad_kernel<T, false, 2> : norm_grad_kernel<T, false, 4>;
}

struct GradPlan {
  int64_t ctas, pre_off, post_off, gate_off, bytes;
};
GradPlan grad_plan(int64_t tokens, int64_t hidden, int64_t gate_rows) {
  GradPlan p;
  p.ctas = grad_ctas(tokens, hidden);
  const int64_t each = ops_round_up(p.ctas * hidden * 4, 256);
  p.pre_off = 0;
  p.post_off = each;
  p.gate_off = 2 * each;
  p.bytes = 2 * each + (gate_rows > 0 ? 2 * each : 0);
  return p;
}

cudaError_t zero_rows(const lst_matrix* m, cudaStream_t stream) {
  if (!m || m->rows == 0) return cudaSuccess;
  const size_t size = dtype_bytes(m->dtype);
  return cudaMemset2DAsync(m->data, static_cast<size_t>(m->stride) * size, 0, static_cast<size_t>(m->cols) * size,
                           static_cast<size_t>(m->rows), stream);
}

}  // namespace
}  // namespace lst

using namespace lst;

extern "C" lst_status lst_residual_norm(const lst_matrix* x, const lst_matrix* y, const lst_matrix* gate,
                                        const lst_matrix* w_post, const lst_matrix* w_pre,
                                        const lst_residual_params* params, const lst_matrix* h, const lst_matrix* z,
                                        const lst_checkpoint* h8, const lst_checkpoint* y8, void* cuda_stream) {
  clear_error();
  const char* who = "lst_residual_norm";
  LST_TRY(check_matrix(x, "x", who));
  const Shape s = {who, x->rows, x->cols, x->dtype};
  LST_TRY(s.sizes(params));
  LST_TRY(s.rows(y, "y"));
  LST_TRY(s.rows(h, "h"));
  LST_TRY(s.rows(z, "z"));
  LST_TRY(s.gate(gate, "gate"));
  LST_TRY(s.vector(w_post, "w_post"));
  LST_TRY(s.vector(w_pre, "w_pre"));
  LST_TRY(s.kept(h8, "h8"));
  LST_TRY(s.kept(y8, "y8"));
  if (!y && (gate || w_post || y8)) return fail(LST_ERR_INVALID_ARG, "%s: gate, w_post or y8 without y", who);
  if (!z != !w_pre) return fail(LST_ERR_INVALID_ARG, "%s: z and w_pre go together", who);
  if (!h && !z && !h8) return fail(LST_ERR_INVALID_ARG, "%s: none of h, z and h8", who);
  if (s.tokens == 0) return LST_OK;
  const bool vec = s.hidden % 8 == 0 && on16(x) && on16(y) && on16(h) && on16(z);
  const Fit f = fit(s.hidden);
  const NormArgs a = {rows_arg(x), rows_arg(y), rows_arg(h), rows_arg(z), weights_arg(gate), weights_arg(w_post),
                      weights_arg(w_pre), kept_arg(h8), kept_arg(y8), s.tokens, gate ? s.tokens / gate->rows : s.tokens,
                      static_cast<int32_t>(s.hidden), params->residual_scale, params->branch_scale, params->eps};
  const unsigned grid = static_cast<unsigned>(std::min(s.tokens, kSms * std::max<int64_t>(1, 1024 / f.threads)));
  const Kernel<NormArgs> kernel = s.dtype == LST_F32 ? norm_of<float>(vec, f.k) : norm_of<__nv_bfloat16>(vec, f.k);
  LST_TRY_CUDA(launch_chained(kernel, dim3(grid), dim3(static_cast<unsigned>(f.threads)), 0,
                              static_cast<cudaStream_t>(cuda_stream), a),
               who);
  return LST_OK;
}

extern "C" int64_t lst_residual_norm_grad_workspace_bytes(int64_t tokens, int64_t hidden, int64_t gate_rows) {
  if (tokens < 1 || tokens > INT32_MAX || hidden < 1 || hidden > kMaxHidden || gate_rows < 0 || gate_rows > tokens) return 0;
  return grad_plan(tokens, hidden, gate_rows).bytes;
}

extern "C" lst_status lst_residual_norm_grad(const lst_matrix* dh, const lst_matrix* dz, const lst_matrix* h,
                                             const lst_checkpoint* h8, const lst_matrix* y, const lst_checkpoint* y8,
                                             const lst_matrix* gate, const lst_matrix* w_post, const lst_matrix* w_pre,
                                             const lst_residual_params* params, const lst_matrix* dx,
                                             const lst_matrix* dy, const lst_matrix* dgate, const lst_matrix* dw_post,
                                             const lst_matrix* dw_pre, int32_t accumulate, void* workspace,
                                             int64_t workspace_bytes, void* cuda_stream) {
  clear_error();
  const char* who = "lst_residual_norm_grad";
  if (!dh && !dz) return fail(LST_ERR_INVALID_ARG, "%s: dh and dz are null", who);
  const lst_matrix* any = dh ? dh : dz;
  LST_TRY(check_matrix(any, dh ? "dh" : "dz", who));
  const Shape s = {who, any->rows, any->cols, any->dtype};
  LST_TRY(s.sizes(params));
  LST_TRY(s.rows(dz, "dz"));
  LST_TRY(s.rows(h, "h"));
  LST_TRY(s.rows(y, "y"));
  LST_TRY(s.rows(dx, "dx"));
  LST_TRY(s.rows(dy, "dy"));
  LST_TRY(s.kept(h8, "h8"));
  LST_TRY(s.kept(y8, "y8"));
  LST_TRY(s.gate(gate, "gate"));
  LST_TRY(s.vector(w_post, "w_post"));
  LST_TRY(s.vector(w_pre, "w_pre"));
  LST_TRY(s.gate(dgate, "dgate"));
  LST_TRY(s.vector(dw_post, "dw_post"));
  LST_TRY(s.vector(dw_pre, "dw_pre"));
  if ((h && h8) || (y && y8)) return fail(LST_ERR_INVALID_ARG, "%s: h or y both as a matrix and as a checkpoint", who);
  if (!dz != !w_pre) return fail(LST_ERR_INVALID_ARG, "%s: dz and w_pre go together", who);
  if (dz && !h && !h8) return fail(LST_ERR_INVALID_ARG, "%s: dz without h", who);
  if (dw_pre && !dz) return fail(LST_ERR_INVALID_ARG, "%s: dw_pre without dz", who);
  if (dw_post && !w_post) return fail(LST_ERR_INVALID_ARG, "%s: dw_post without w_post", who);
  if (dgate && (!gate || gate->rows != dgate->rows)) return fail(LST_ERR_INVALID_ARG, "%s: dgate must have the shape of gate", who);
  if ((w_post || dgate) && !y && !y8) return fail(LST_ERR_INVALID_ARG, "%s: w_post or dgate without y", who);
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  if (s.tokens == 0) {
    if (!accumulate)
      for (const lst_matrix* m : {dgate, dw_post, dw_pre}) LST_TRY_CUDA(zero_rows(m, stream), who);
    return LST_OK;
  }
  const bool need_y = w_post || dgate;  // without either, dy is a multiple of D
  const GradPlan p = grad_plan(s.tokens, s.hidden, gate ? gate->rows : 0);
  const bool sums = dw_pre || dw_post || dgate;
  LST_TRY(check_workspace(workspace, workspace_bytes, sums ? p.bytes : 0, who));
  char* ws = static_cast<char*>(workspace);
  const lst_matrix *h_in = dz ? h : nullptr, *y_in = need_y ? y : nullptr;
  const bool vec = s.hidden % 8 == 0 && on16(dh) && on16(dz) && on16(h_in) && on16(y_in) && on16(dx) && on16(dy);
  const Fit f = fit(s.hidden);
  const int64_t per_gate = gate ? s.tokens / gate->rows : s.tokens;
  GradArgs a = {};
  a.dh = rows_arg(dh), a.dz = rows_arg(dz), a.h = rows_arg(h_in), a.y = rows_arg(y_in), a.dx = rows_arg(dx), a.dy = rows_arg(dy);
  a.h8 = kept_arg(dz ? h8 : nullptr), a.y8 = kept_arg(need_y ? y8 : nullptr);
  a.gate = weights_arg(gate), a.w_post = weights_arg(w_post), a.w_pre = weights_arg(w_pre);
  if (dgate) a.dgate = dgate->data, a.dgate_stride = dgate->stride, a.dgate_f32 = dgate->dtype == LST_F32;
  a.accumulate = accumulate != 0;
  a.part_pre = dw_pre ? reinterpret_cast<float*>(ws + p.pre_off) : nullptr;
  a.part_post = dw_post ? reinterpret_cast<float*>(ws + p.post_off) : nullptr;
  a.part_gate = dgate ? reinterpret_cast<float*>(ws + p.gate_off) : nullptr;
  a.tokens = s.tokens, a.per_gate = per_gate, a.hidden = static_cast<int32_t>(s.hidden), a.ctas = static_cast<int32_t>(p.ctas);
  a.alpha = params->residual_scale, a.beta = params->branch_scale, a.eps = params->eps;
  const Kernel<GradArgs> kernel = s.dtype == LST_F32 ? norm_grad_of<float>(vec, f.k) : norm_grad_of<__nv_bfloat16>(vec, f.k);
  LST_TRY_CUDA(launch_chained(kernel, dim3(static_cast<unsigned>(p.ctas)), dim3(static_cast<unsigned>(f.threads)), 0, stream, a), who);
  if (!sums) return LST_OK;
  JoinArgs j = {a.part_pre, a.part_post, a.part_gate, dw_pre ? dw_pre->data : nullptr, dw_post ? dw_post->data : nullptr,
                a.dgate, a.dgate_stride, s.tokens, per_gate, dw_pre && dw_pre->dtype == LST_F32,
                dw_post && dw_post->dtype == LST_F32, a.dgate_f32, a.accumulate, a.hidden, a.ctas};
  const bool shared_gates = dgate && per_gate > 1;
  LST_TRY_CUDA(launch_chained(norm_join_kernel,
                              dim3(static_cast<unsigned>(ops_ceil_div(s.hidden, 32)), static_cast<unsigned>(2 + (shared_gates ? p.ctas : 0))),
                              dim3(256), 0, stream, j),
               who);
  return LST_OK;
}
