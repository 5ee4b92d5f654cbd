// The residual stream between two layers: norm of the block's output, gate, scales
// and sum, norm of the sum, with 8-bit checkpoints of what the backward pass reads,
// and the gradients of all that.
//
// Forward, row by row: u = y tau w_post (tau = rsqrt(mean y^2 + eps)), h = a x + b g u,
// z = h rho w_pre (rho = rsqrt(mean h^2 + eps)). A row is read once; h, z and the
// checkpoints are written from registers.
//
// Backward: with m = w_pre dz
//   D  = dh + rho (m - h rho^2 mean(m h)),  dx = a D,  dw_pre = sum dz h rho
//   e  = b D g w_post,  dy = tau (e - y tau^2 mean(e y))
//   A  = sum D tau y over the tokens of a gate row;  dgate = b w_post A,  dw_post = b sum g A
// so two sums per column (A and dw_pre's) give all three parameter gradients. A CTA
// takes consecutive rows (with one gate row, rows in turns) and keeps the column sums in
// registers; they go to the workspace once per CTA (A once per gate row) and are added up
// in order by a second launch. Rows above 8192 columns: lst_norm_split.cuh.
//
// Floors are memory's: 8 bytes an element forward, 12 backward in bf16 (10 with checkpoints).
// Forward runs at 5.3 TB/s (16384 x 4096 with an 8-bit copy, 114 us of 90; 5.8 without norm and
// gate of the block): issue slots are 56 % in use, and what a warp waits for is shared memory (a
// quarter of its cycles), arithmetic before it (a sixth) and the row's two barriers (another). Rows of
// 6145 to 8192 columns leave one CTA an SM, whose 13 to 16 warps stand at those barriers together
// (16384 x 8192: 243 us of 159); rows above hold 32 columns a thread, 9 to 16 warps an SM, and
// read their weights from L2 for each (4096 x 12288: 171 of 60). Backward runs at 4.8 TB/s
// (16381 x 8192 from checkpoints, 278 us and 7 for the sums): some 45 instructions an
// element and 16 warps an SM, as many as 128 registers and the rows in flight leave.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "lst_norm.cuh"
#include "lst_norm.h"

namespace lst {

namespace {

constexpr int64_t kMaxHidden = 16384;
constexpr int64_t kSms = 152;
constexpr int64_t kSharedPerSm = 228 * 1024;  // 1 KB of it the system's, per CTA
constexpr int kMaxShared = 227 * 1024;

__device__ int g_norm_error;

// ---- forward -----------------------------------------------------------------------
enum NormOperand { NORM_X, NORM_Y, NORM_GATE, NORM_OPS };
struct NormArgs {
  PipeArgs<NORM_OPS> pipe;
  Rows h, z;
  Weights gate, w_post, w_pre;
  Kept h8, y8;
  float alpha, beta, eps;
};

template <class T, bool VEC, int K>
__global__ void __maxnreg__(K == 4 ? 128 : 80) norm_kernel(const __grid_constant__ NormArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  let_next_start();
  Pipe<NORM_OPS> p(a.pipe, smem);
  wait_for_previous();
  p.start(VEC && a.pipe.pad);
  const int group = threadIdx.x / a.pipe.group, tid = threadIdx.x - group * a.pipe.group, warp = tid >> 5, warps = a.pipe.group >> 5;
  Cols<VEC> c = {static_cast<uint32_t>(tid), static_cast<uint32_t>(a.pipe.group), static_cast<uint32_t>(a.pipe.hidden)};
  const float inverse = 1.0f / static_cast<float>(a.pipe.hidden);
  const bool has_y = a.pipe.in[NORM_Y].p != nullptr, per_token = a.pipe.in[NORM_GATE].p != nullptr;
  const bool has_post = a.w_post.p != nullptr, has_h = a.h.p != nullptr, has_z = a.z.p != nullptr;
  float* const words = p.words() + group * 16;
  // w_pre and beta * gate * w_post as fp32 in shared memory (registers would allow half as many
  // warps); K = 4 reads them again for every row
  constexpr bool kHold = K <= 2;
  const int columns = VEC ? 8 * K * a.pipe.group : a.pipe.hidden;
  float* const held_pre = reinterpret_cast<float*>(smem + kPipeHeader + a.pipe.stages * p.stage_bytes);
  float* const held_gw = held_pre + columns;
  auto load_pre = [&](int k, Unit& u) {
    u.fill(0.0f);
    if (has_z && c.has(k)) c.load_any(a.w_pre.p, a.w_pre.f32, k, u);
  };
  auto load_gw = [&](int k, Unit& u) {
    Unit g;
    u.fill(c.has(k) ? a.beta : 0.0f);
    if (has_post && c.has(k)) {
      c.load_any(a.w_post.p, a.w_post.f32, k, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], g.v[j]);
    }
    if (a.gate.p && !per_token && c.has(k)) {
      c.load_any(row_of(a.gate, p.row / a.pipe.per_segment), a.gate.f32, k, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], g.v[j]);
    }
  };
  int turn = 0;
  auto sum = [&](float2 s) { return group_sum(s.x + s.y, words, turn, warps, warp, 1 + group, a.pipe.group); };
  do {
    if (kHold) {
      // each thread the columns that it reads itself, or one group for all
      if (a.pipe.groups > 1) asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
      if (group == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Unit u;
          load_pre(k, u);
          c.store(held_pre, k, u);
          load_gw(k, u);
          c.store(held_gw, k, u);
        }
      }
      if (a.pipe.groups > 1) asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
    }
    int rows;
    do {
      rows = p.rows();
      if (!VEC) asm volatile("" : "+r"(c.threads));  // columns' offsets are formed again: held, they would spill
      p.wait();
      const bool mine = group < rows;
      const int64_t row = static_cast<uint32_t>(p.row) + group;
      Unit h[K];
      if (mine) {
        const uint8_t* const staged = p.staged(group);
        const T* const x = reinterpret_cast<const T*>(p.at(NORM_X, group, staged, VEC));
        if (has_y) {
          const T* const y = reinterpret_cast<const T*>(p.at(NORM_Y, group, staged, VEC));
          float2 s = both(0.0f);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            c.load(y, k, h[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) s = fma2(h[k].v[j], h[k].v[j], s);
          }
          if (a.y8.data) {
#pragma unroll
            for (int k = 0; k < K; ++k)
              c.save(h[k], k, a.y8.data + row * a.y8.stride, a.y8.scales + row * a.y8.scale_stride, a.y8.e4m3);
          }
          const float2 tau = both(has_post ? rsqrtf(sum(s) * inverse + a.eps) : 1.0f);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            Unit u;
            if (kHold)
              c.load(held_gw, k, u);
            else
              load_gw(k, u);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[k].v[j] = mul2(mul2(h[k].v[j], tau), u.v[j]);
            if (per_token) {
              if (a.gate.f32)
                c.load(reinterpret_cast<const float*>(p.at(NORM_GATE, group, staged, VEC)), k, u);
              else
                c.load(reinterpret_cast<const __nv_bfloat16*>(p.at(NORM_GATE, group, staged, VEC)), k, u);
#pragma unroll
              for (int j = 0; j < 4; ++j) h[k].v[j] = mul2(h[k].v[j], u.v[j]);
            }
            c.load(x, k, u);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[k].v[j] = fma2(u.v[j], both(a.alpha), h[k].v[j]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            c.load(x, k, h[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[k].v[j] = mul2(h[k].v[j], both(a.alpha));
          }
        }
      }
      p.release();
      p.refill(false);
      if (mine) {
        float2 s = both(0.0f);
        T* const to = row_of<T>(a.h, row);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (has_h && c.has(k)) c.store(to, k, h[k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) s = fma2(h[k].v[j], h[k].v[j], s);
        }
        if (a.h8.data) {
#pragma unroll
          for (int k = 0; k < K; ++k) {
            Unit r;
#pragma unroll
            for (int j = 0; j < 4; ++j) r.v[j] = round_to(h[k].v[j], static_cast<const T*>(nullptr));
            c.save(r, k, a.h8.data + row * a.h8.stride, a.h8.scales + row * a.h8.scale_stride, a.h8.e4m3);
          }
        }
        if (has_z) {
          const float2 rho = both(rsqrtf(sum(s) * inverse + a.eps));
          T* const out = row_of<T>(a.z, row);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            Unit u;
            if (kHold)
              c.load(held_pre, k, u);
            else
              load_pre(k, u);
#pragma unroll
            for (int j = 0; j < 4; ++j) h[k].v[j] = mul2(mul2(h[k].v[j], rho), u.v[j]);
            if (c.has(k)) c.store(out, k, h[k]);
          }
        }
      }
    } while (p.next(rows));
  } while (p.next_segment());
  p.finish(&g_norm_error);
}

// Adds up the CTAs' sums, 128 columns a CTA: blockIdx.y 0: dw_pre, 1: dw_post (with one gate row
// or none, the sums are A: dw_post from it times the gate, dgate times w_post); from 2 on the
// gate rows that more than one CTA worked on, by their number or (where there are more
// gate rows than CTAs) as the last gate row of CTA blockIdx.y - 2.
struct JoinArgs {
  const float *pre, *post, *gate;
  void *dw_pre, *dw_post, *dgate;
  int64_t dgate_stride, tokens, per_gate;
  int32_t pre_f32, post_f32, gate_f32, accumulate, hidden, ld, ctas, by_row, single;
  Weights gate_row, w_post;  // factors of A
};
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float4 words[kJoinWarps][32];
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 128 + 4 * lane;
  const float* part = blockIdx.y == 0 ? a.pre : a.post;
  void* out = blockIdx.y == 0 ? a.dw_pre : a.dw_post;
  bool f32 = blockIdx.y == 0 ? a.pre_f32 : a.post_f32;
  const bool both_of_a = blockIdx.y == 1 && a.single;
  if (blockIdx.y < 2 && !out && !(both_of_a && a.dgate)) return;
  int64_t at = 0, r = -1, first = 0, last = a.ctas;
  if (blockIdx.y >= 2) {
    part = a.gate, out = a.dgate, f32 = a.gate_f32;
    auto owner = [&](int64_t row) {  // the CTA whose rows include `row`
      int64_t c = row * a.ctas / a.tokens;
      while (first_row(c + 1, a.tokens, a.ctas) <= row) ++c;
      return c;
    };
    if (a.by_row) {
      r = blockIdx.y - 2;
      first = owner(r * a.per_gate);
    } else {
      first = blockIdx.y - 2;
      const int64_t begin = first_row(first, a.tokens, a.ctas), end = first_row(first + 1, a.tokens, a.ctas);
      r = (end - 1) / a.per_gate;
      if (begin == end || r * a.per_gate < begin) return;
    }
    last = owner((r + 1) * a.per_gate - 1) + 1;
    if (last == first + 1) return;  // its CTA has written it
    at = r * a.dgate_stride;
  }
  float4 s = make_float4(0, 0, 0, 0);
  if (col < a.ld) {
    // a gate row that more CTAs share begins in the first one (its first gate row, or its last) and is the first of the others
    const int64_t step = r < 0 ? 1 : 2;
    const int64_t odd = r >= 0 && r != first_row(first, a.tokens, a.ctas) / a.per_gate;
    const float* p = part + col;
#pragma unroll 8
    for (int64_t c = first + warp; c < last; c += kJoinWarps) {
      const float4 v = *reinterpret_cast<const float4*>(p + (step * c + (c == first ? odd : 0)) * a.ld);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
  }
  words[warp][lane] = s;
  __syncthreads();
  const int mine = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x >= 128 || mine >= a.hidden) return;
  float v = 0.0f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) v += reinterpret_cast<const float*>(words[i])[threadIdx.x];
  if (both_of_a && a.dgate) store_sum(a.dgate, mine, a.gate_f32, a.accumulate, a.w_post.p ? v * weight_at(a.w_post, 0, mine) : v);
  if (both_of_a && a.gate_row.p) v *= weight_at(a.gate_row, 0, mine);
  if (out) store_sum(out, at + mine, f32, a.accumulate, v);
}

// ---- host ------------------------------------------------------------------------
// 16 columns a thread (32 of rows above 8192), and short rows several at a time, so that a CTA
// has about 256 threads, 512 where a row needs them. An SM holds up to 512 threads of the backward
// kernel and 768 of the forward one, as many as their registers allow (forward with 512: 157 us
// for 16384 x 4096 with a checkpoint and its restore, with 1024 of 64 registers 184, so 155), in
// whole CTAs: forward 416 to 512 from 6145 to 8192 columns, 288 to 512 above.
struct Fit {
  int k, group, groups, per_sm;
  int threads() const { return group * groups; }
};
Fit fit(int64_t hidden, int threads_per_sm, int k) {
  Fit f;
  f.k = k;
  f.group = static_cast<int>(ops_round_up(ops_ceil_div(hidden, 8 * f.k), 32));
  f.groups = std::max(1, 256 / f.group);
  f.per_sm = std::max(1, (f.k == 4 ? 512 : threads_per_sm) / f.threads());
  return f;
}
Fit norm_fit(int64_t hidden) { return fit(hidden, 768, hidden <= 8192 ? 2 : 4); }
// Backward, rows that are not whole units take 8 columns a thread where 512 threads are enough: code
// that goes value by value is long, and half of it with twice the warps runs faster (1023 x 4095 in
// fp32 with a gate per token: 74 us with 16 columns a thread, 49 with 8).
Fit grad_fit(int64_t hidden, bool vec) { return fit(hidden, 512, !vec && hidden <= 4096 ? 1 : 2); }
int64_t ctas_of(const Fit& f, int64_t tokens) { return std::min(ops_ceil_div(tokens, f.groups), kSms * f.per_sm); }

// Operands in the order of their slots in a staged row.
template <int OPS>
struct Operands {
  PipeArgs<OPS> pipe = {};
  int64_t columns;  // of a staged row: all that its threads hold where it is read unit by unit
  int scales_only;  // nothing but scales lies off 16 bytes
  Operands(const Fit& f, bool vec, int64_t hidden) : columns(vec ? int64_t(8) * f.k * f.group : hidden) {}
  void range(int op, const void* data, int64_t stride, int64_t bytes, int64_t place) {
    pipe.in[op] = {static_cast<const uint8_t*>(data), stride, static_cast<int32_t>(bytes), pipe.row_bytes};
    pipe.row_bytes += static_cast<int32_t>(ops_round_up(place + 15, 16));
  }
  void matrix(int op, const lst_matrix* m) {
    if (m) range(op, m->data, m->stride * dtype_bytes(m->dtype), m->cols * dtype_bytes(m->dtype), columns * dtype_bytes(m->dtype));
  }
  // values and scales; returns 1 for integers, 2 for e4m3, 0 for no checkpoint
  int32_t kept(int op, const lst_checkpoint* c) {
    if (!c) return 0;
    range(op, c->data, c->stride, ops_round_up(c->cols, 16), ops_round_up(columns, 16));  // rows reach to there
    range(op + 1, c->scales, c->scale_stride, ops_ceil_div(c->cols, kCkptBlock), ops_ceil_div(columns, kCkptBlock));
    return c->format == LST_CHECKPOINT_E4M3 ? 2 : 1;
  }
  // `sums`: floats per column that each of several groups leaves in shared memory; `held`: that
  // the CTA keeps there. Where not even one stage fits, rows are taken fewer at a time, then
  // fewer CTAs to an SM. Returns the shared memory of a CTA.
  size_t plan(const Fit& f, int64_t tokens, int64_t hidden, int64_t per_segment, int sums, int held) {
    pipe.pad = columns > hidden;
    pipe.simple = scales_only = 1;
    for (int op = 0; op < OPS; ++op) {
      const Range& r = pipe.in[op];
      if (!r.p) continue;
      pipe.row_total += r.bytes;
      pipe.margin = std::max(pipe.margin, static_cast<int32_t>(ops_ceil_div(15, std::max<int64_t>(1, r.stride))));
      if (reinterpret_cast<uintptr_t>(r.p) % 16 || (tokens > 1 && r.stride % 16) || r.bytes % 16)
        pipe.simple = 0, scales_only &= OPS == GRAD_OPS && (op == GRAD_H_SCALES || op == GRAD_Y_SCALES);
    }
    pipe.tokens = static_cast<int32_t>(tokens), pipe.per_segment = static_cast<int32_t>(per_segment);
    pipe.hidden = static_cast<int32_t>(hidden);
    pipe.group = f.group, pipe.ctas = static_cast<int32_t>(ctas_of(f, tokens));
    int groups = f.groups, per_sm = f.per_sm;
    for (;;) {
      const int64_t stage = static_cast<int64_t>(pipe.row_bytes) * groups;
      const int64_t extra = ((groups > 1 ? groups * sums : 0) + held) * columns * 4;
      const int64_t room = std::min<int64_t>(kSharedPerSm / per_sm - 1024, kMaxShared) - kPipeHeader - extra;
      pipe.groups = groups;
      pipe.stages = room < stage ? 0 : static_cast<int32_t>(std::min<int64_t>(kMaxStages, room / stage));
      if (pipe.stages > 0 || (groups == 1 && per_sm == 1)) {
        pipe.ctas = static_cast<int32_t>(std::min<int64_t>(pipe.ctas, kSms * per_sm));  // all at once
        if (per_segment == tokens) pipe.step = pipe.ctas * groups;
        return static_cast<size_t>(kPipeHeader + pipe.stages * stage + extra);
      }
      if (groups > 1)
        groups /= 2;
      else
        --per_sm;
    }
  }
  unsigned threads() const { return static_cast<unsigned>(pipe.group * pipe.groups); }
};

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

template <class T, bool VEC>
NormKernel<NormArgs> norm_of(int k) {
  return k == 2 ? norm_kernel<T, VEC, 2> : norm_kernel<T, VEC, 4>;
}

// Elements of a row of sums in the workspace.
int64_t sum_row(int64_t hidden) { return ops_round_up(hidden, 4); }

// Rows above 8192 columns go backward in two launches (lst_norm_split.cuh), by tiles of columns
// and chunks of rows.
constexpr int64_t kWide = 8192;
int64_t split_chunks(int64_t tokens, int64_t hidden, bool vec) { return std::min(tokens, split_ctas(vec) * kSms / ops_ceil_div(hidden, kSplitTile)); }

struct GradPlan {
  int64_t ctas, pre_off, post_off, gate_off, stats_off, bytes;
};
GradPlan grad_plan(int64_t tokens, int64_t hidden, int64_t gate_rows) {
  GradPlan p;
  p.ctas = hidden > kWide ? split_chunks(tokens, hidden, false)
                          : std::max(ctas_of(grad_fit(hidden, false), tokens), ctas_of(grad_fit(hidden, true), tokens));
  const int64_t each = ops_round_up(p.ctas * sum_row(hidden) * 4, 256);
  p.pre_off = 0;
  p.post_off = each;
  p.gate_off = 2 * each;
  p.stats_off = 2 * each + (gate_rows > 0 ? 2 * each : 0);
  p.bytes = p.stats_off + (hidden > kWide ? ops_round_up(tokens * 16, 256) : 0);
  return p;
}

cudaError_t zero_rows(const lst_matrix* m, cudaStream_t stream) {
  if (!m || m->rows == 0) return cudaSuccess;
  const size_t size = dtype_bytes(m->dtype);
  return cudaMemset2DAsync(m->data, static_cast<size_t>(m->stride) * size, 0, static_cast<size_t>(m->cols) * size,
                           static_cast<size_t>(m->rows), stream);
}

}  // namespace

cudaError_t norm_take_error(int* out) {
  int err[3] = {};
  cudaError_t st = cudaMemcpyFromSymbol(&err[0], g_norm_error, sizeof(int));
  if (st == cudaSuccess && err[0]) {
    const int zero = 0;
    st = cudaMemcpyToSymbol(g_norm_error, &zero, sizeof(int));
  }
  if (st == cudaSuccess) st = norm_grad_bf16_take_error(&err[1]);
  if (st == cudaSuccess) st = norm_grad_f32_take_error(&err[2]);
  *out = err[0] | err[1] | err[2];
  return st;
}

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
  const bool token = gate && gate->rows == s.tokens && s.tokens > 1;
  const bool vec = s.hidden % 8 == 0 && on16(x) && on16(y) && on16(h) && on16(z) && (!token || on16(gate));
  const Fit f = norm_fit(s.hidden);
  Operands<NORM_OPS> o(f, vec, s.hidden);
  o.matrix(NORM_X, x);
  o.matrix(NORM_Y, y);
  if (token) o.matrix(NORM_GATE, gate);
  const size_t smem = o.plan(f, s.tokens, s.hidden, gate && !token ? s.tokens / gate->rows : s.tokens, 0, f.k == 2 ? 2 : 0);
  const NormArgs a = {o.pipe, rows_arg(h), rows_arg(z), weights_arg(gate), weights_arg(w_post), weights_arg(w_pre), kept_arg(h8),
                      kept_arg(y8), params->residual_scale, params->branch_scale, params->eps};
  const NormKernel<NormArgs> kernel = s.dtype == LST_F32 ? (vec ? norm_of<float, true>(f.k) : norm_of<float, false>(f.k))
                                  : vec              ? norm_of<__nv_bfloat16, true>(f.k)
                                                     : norm_of<__nv_bfloat16, false>(f.k);
  LST_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared), who);
  LST_TRY_CUDA(launch_chained(kernel, dim3(static_cast<unsigned>(o.pipe.ctas)), dim3(o.threads()), smem,
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
  const bool sums = dw_pre || dw_post || dgate, wide = s.hidden > kWide;
  LST_TRY(check_workspace(workspace, workspace_bytes, sums || wide ? p.bytes : 0, who));
  char* ws = static_cast<char*>(workspace);
  const lst_matrix *h_in = dz ? h : nullptr, *y_in = need_y ? y : nullptr;
  const int64_t per_gate = gate ? s.tokens / gate->rows : s.tokens;
  const bool token = per_gate == 1 && s.tokens > 1;
  const bool vec = s.hidden % 8 == 0 && on16(dh) && on16(dz) && on16(h_in) && on16(y_in) && on16(dx) && on16(dy) && (!token || on16(gate));
  const Fit f = grad_fit(s.hidden, vec);
  Operands<GRAD_OPS> o(f, vec, s.hidden);
  GradArgs a = {};
  o.matrix(GRAD_DH, dh), o.matrix(GRAD_DZ, dz), o.matrix(GRAD_H, h_in), o.matrix(GRAD_Y, y_in);
  a.h_kept = o.kept(GRAD_H, dz ? h8 : nullptr);
  a.y_kept = o.kept(GRAD_Y, need_y ? y8 : nullptr);
  if (token) o.matrix(GRAD_GATE, gate);
  size_t smem = 0;
  if (wide) {
    o.pipe.tokens = static_cast<int32_t>(s.tokens), o.pipe.hidden = static_cast<int32_t>(s.hidden);
    o.pipe.ctas = static_cast<int32_t>(split_chunks(s.tokens, s.hidden, vec));
  } else {
    smem = o.plan(f, s.tokens, s.hidden, token ? s.tokens : per_gate, 2, 2);
  }
  a.pipe = o.pipe;
  a.dx = rows_arg(dx), a.dy = rows_arg(dy);
  a.gate = weights_arg(gate), a.w_post = weights_arg(w_post), a.w_pre = weights_arg(w_pre);
  if (dgate) a.dgate = dgate->data, a.dgate_stride = dgate->stride, a.dgate_f32 = dgate->dtype == LST_F32;
  a.per_gate = static_cast<int32_t>(per_gate), a.accumulate = accumulate != 0;
  a.part_pre = dw_pre ? reinterpret_cast<float*>(ws + p.pre_off) : nullptr;
  const bool single = token || per_gate == s.tokens;  // one gate row, none, or one per token (whose dgate is complete)
  a.part_post = dw_post || (dgate && single && !token) ? reinterpret_cast<float*>(ws + p.post_off) : nullptr;
  a.part_gate = dgate ? reinterpret_cast<float*>(ws + p.gate_off) : nullptr;
  a.alpha = params->residual_scale, a.beta = params->branch_scale, a.eps = params->eps;
  if (wide) {
    const SplitKernels kernels = s.dtype == LST_F32 ? norm_split_f32(vec) : norm_split_bf16(vec);
    a.stats = reinterpret_cast<float4*>(ws + p.stats_off), a.token = token, a.single = single;
    if (dz || w_post)
      LST_TRY_CUDA(launch_chained(kernels.stats, dim3(static_cast<unsigned>(std::min(s.tokens, 4 * kSms))), dim3(256), 0, stream, a), who);
    const dim3 grid(static_cast<unsigned>(ops_ceil_div(s.hidden, kSplitTile)), static_cast<unsigned>(o.pipe.ctas));
    LST_TRY_CUDA(launch_chained(kernels.apply, grid, dim3(kSplitTile / 8), 0, stream, a), who);
  } else {
    const bool whole = vec && o.scales_only && dz && !token && (!need_y || a.h_kept == a.y_kept);
    const int block = !need_y ? 0 : w_post && dh && dx && dy ? 2 : 1, form = whole ? 1 + a.h_kept + 3 * block : 0;
    const NormKernel<GradArgs> kernel = s.dtype == LST_F32 ? norm_grad_f32(vec, f.k, form, o.pipe.groups == 1) : norm_grad_bf16(vec, f.k, form, o.pipe.groups == 1);
    LST_TRY_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared), who);
    LST_TRY_CUDA(launch_chained(kernel, dim3(static_cast<unsigned>(o.pipe.ctas)), dim3(o.threads()), smem, stream, a), who);
  }
  if (!sums) return LST_OK;
  const int64_t gate_rows = dgate && !single ? gate->rows : 0;
  const JoinArgs j = {a.part_pre, a.part_post, a.part_gate, dw_pre ? dw_pre->data : nullptr, dw_post ? dw_post->data : nullptr,
                      token ? nullptr : a.dgate, a.dgate_stride, s.tokens, per_gate, dw_pre && dw_pre->dtype == LST_F32,
                      dw_post && dw_post->dtype == LST_F32, a.dgate_f32, a.accumulate, static_cast<int32_t>(s.hidden),
                      static_cast<int32_t>(sum_row(s.hidden)), o.pipe.ctas, gate_rows <= o.pipe.ctas, single && !token,
                      token ? Weights{} : a.gate, a.w_post};
  LST_TRY_CUDA(launch_chained(norm_join_kernel,
                              dim3(static_cast<unsigned>(ops_ceil_div(s.hidden, 128)), static_cast<unsigned>(2 + std::min<int64_t>(gate_rows, o.pipe.ctas))),
                              dim3(32 * kJoinWarps), 0, stream, j),
               who);
  return LST_OK;
}
