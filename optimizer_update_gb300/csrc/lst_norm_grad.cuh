// The backward kernel of the residual norm; the mathematics is at the top of lst_norm.cu.
#pragma once

#include "lst_norm.cuh"

namespace lst {

namespace {

__device__ int g_norm_grad_error;

// The sums of a gate row, or of all of the CTA's rows, to the workspace (or to dgate where
// the CTA has all of a gate row's tokens). With one gate row, or none, that is A as it is,
// from which the join forms dw_post and dgate.
template <bool VEC, int K, bool ONE, class P>
__device__ __forceinline__ void flush_sums(const GradArgs& a, const P& p, const Cols<VEC>& c, int group, float* group_sums, int columns,
                                           bool token, bool has_y, bool has_post, bool first_flush, const Unit (&sum_a)[K],
                                           const Unit (&sum_pre)[K]) {
  const int hidden = a.pipe.hidden, ld = (hidden + 3) & ~3;
  const int64_t cta = blockIdx.x;
  const bool last = p.row >= p.end;
  const int64_t gate_row = (p.segment - 1) / a.per_gate;
  const bool whole = gate_row * a.per_gate >= p.begin && (gate_row + 1) * a.per_gate <= p.end;
  float* const gate_sums = a.part_gate + (2 * cta + (gate_row == p.begin / a.per_gate ? 0 : 1)) * ld;
  float *const post = a.part_post + cta * ld, *const pre = a.part_pre + cta * ld;
  const bool several = !a.pipe.step, gated = several && !token && a.gate.p, gates = several && !token && has_y && a.dgate;
  const bool posts = has_y && a.part_post, pres = last && a.part_pre;
  if (ONE || a.pipe.groups == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!c.has(k)) continue;
      Unit u, w;
      if (posts) {
        u = sum_a[k];
        if (gated) {
          c.load_any(row_of(a.gate, gate_row), a.gate.f32, k, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], w.v[j]);
        }
        if (!first_flush) {
          c.load_any(post, true, k, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) u.v[j] = add2(u.v[j], w.v[j]);
        }
        c.store(post, k, u);
      }
      if (gates) {
        u = sum_a[k];
        if (has_post) {
          c.load_any(a.w_post.p, a.w_post.f32, k, w);
#pragma unroll
          for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], w.v[j]);
        }
        if (whole)
          store_sums(a.dgate, gate_row * a.dgate_stride, a.dgate_f32, a.accumulate, c, k, u);
        else
          c.store(gate_sums, k, u);
      }
      if (pres) c.store(pre, k, sum_pre[k]);
    }
  } else {
    // the groups' sums, added up in order
    float* const mine = group_sums + group * 2 * columns;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!c.has(k)) continue;
      for_each(c, k, sum_a[k], [&](uint32_t col, float v) { mine[col] = v; });
      for_each(c, k, sum_pre[k], [&](uint32_t col, float v) { mine[columns + col] = v; });
    }
    asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
    for (int col = threadIdx.x; col < hidden; col += blockDim.x) {
      float sa = 0.0f, sp = 0.0f;
      for (int r = 0; r < a.pipe.groups; ++r) sa += group_sums[r * 2 * columns + col], sp += group_sums[(r * 2 + 1) * columns + col];
      if (posts) {
        const float v = gated ? weight_at(a.gate, gate_row, col) * sa : sa;
        post[col] = first_flush ? v : post[col] + v;
      }
      if (gates) {
        const float v = has_post ? weight_at(a.w_post, 0, col) * sa : sa;
        if (whole)
          store_sum(a.dgate, gate_row * a.dgate_stride + col, a.dgate_f32, a.accumulate, v);
        else
          gate_sums[col] = v;
      }
      if (pres) pre[col] = sp;
    }
    asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
  }
}

// With q = g w_post y, the six sums h^2, m h, y^2, dh q, m q and h q of a row give both
// norms' statistics at once, for D is linear in dh, m and h:
//   sum e y = b (sum dh q + rho (sum m q - rho^2 mean(m h) sum h q)),
// so a row needs one barrier instead of two. Its roundings are those of D's own terms.
// This kernel takes whatever the call has, up to 8192 columns.
template <class T, bool VEC, int K>
__global__ void __maxnreg__(128) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  let_next_start();
  Pipe<GRAD_OPS> p(a.pipe, smem);
  wait_for_previous();
  p.start(VEC && a.pipe.pad);
  const int group = threadIdx.x / a.pipe.group, tid = threadIdx.x - group * a.pipe.group, warp = tid >> 5, warps = a.pipe.group >> 5;
  Cols<VEC> c = {static_cast<uint32_t>(tid), static_cast<uint32_t>(a.pipe.group), static_cast<uint32_t>(a.pipe.hidden)};
  const int hidden = a.pipe.hidden;
  const float inverse = 1.0f / static_cast<float>(hidden);
  const bool has_dh = a.pipe.in[GRAD_DH].p != nullptr, has_z = a.pipe.in[GRAD_DZ].p != nullptr;
  const bool has_post = a.w_post.p != nullptr, has_y = a.pipe.in[GRAD_Y].p != nullptr;
  const bool has_dx = a.dx.p != nullptr, has_dy = a.dy.p != nullptr;
  const int h_kept = a.h_kept, y_kept = a.y_kept;
  const bool token = a.pipe.in[GRAD_GATE].p != nullptr;  // a gate per token
  float* const words = p.words() + group * warps * 8;
  int turn = 0;
  // weights as fp32 in shared memory, where registers would spill; on the vector path units
  // behind the row are zeros there: only stores pass over them
  const int columns = VEC ? 8 * K * a.pipe.group : hidden;
  float* const group_sums = reinterpret_cast<float*>(smem + kPipeHeader + a.pipe.stages * p.stage_bytes);
  float* const held_pre = group_sums + (a.pipe.groups > 1 ? a.pipe.groups * 2 * columns : 0);
  float* const held_gw = held_pre + columns;
  Unit sum_pre[K], sum_a[K];
  // w_pre and gate * w_post of unit k (a gate per token comes with the row)
  auto load_pre = [&](int k, Half& u, int i0) {
    if (has_z) c.load_any(a.w_pre.p, a.w_pre.f32, k, u, i0);
  };
  auto load_gw = [&](int row, int k, Half& u, int i0) {
    u.fill(1.0f);
    if (has_post) c.load_any(a.w_post.p, a.w_post.f32, k, u, i0);
    if (!token && a.gate.p) {
      Half g;
      c.load_any(row_of(a.gate, row / a.per_gate), a.gate.f32, k, g, i0);
#pragma unroll
      for (int j = 0; j < 2; ++j) u.v[j] = mul2(u.v[j], g.v[j]);
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) sum_pre[k].fill(0.0f), sum_a[k].fill(0.0f);
  bool first_flush = true;
  do {
    // each thread the columns that it reads itself, or one group for all
    if (a.pipe.groups > 1) asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
    if (group == 0) {
#pragma unroll
      for (int q = 0; q < 2 * K; ++q) {
        const int k = q >> 1, i0 = 4 * (q & 1);
        Half u;
        u.fill(0.0f);
        if (has_z && c.has(k)) load_pre(k, u, i0);
        c.store(held_pre, k, u, i0);
        u.fill(0.0f);
        if (c.has(k)) load_gw(p.row, k, u, i0);
        c.store(held_gw, k, u, i0);
      }
    }
    if (a.pipe.groups > 1) asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
    int rows;
    do {
      rows = p.rows();
      if (!VEC) asm volatile("" : "+r"(c.threads));  // columns' offsets are formed again: held, they would spill
      p.wait();
      if (group < rows) {
        const int64_t row = static_cast<uint32_t>(p.row) + group;
        const uint8_t* const staged = p.staged(group);
        T *const dx_row = row_of<T>(a.dx, row), *const dy_row = row_of<T>(a.dy, row);
        const T* const dh_row = reinterpret_cast<const T*>(p.at(GRAD_DH, group, staged, VEC));
        const T* const dz_row = reinterpret_cast<const T*>(p.at(GRAD_DZ, group, staged, VEC));
        auto either = [&](int op, int kept, int k, int i0, Half& u) {
          if (kept == 0)
            c.load(reinterpret_cast<const T*>(p.at(op, group, staged, VEC)), k, u, i0);
          else
            c.restore(p.at(op, group, staged, true), p.at(op + 1, group, staged, false), kept == 2, k, u, i0);
        };
        auto gate_unit = [&](int k, int i0, Half& u) {
          if (a.gate.f32)
            c.load(reinterpret_cast<const float*>(p.at(GRAD_GATE, group, staged, VEC)), k, u, i0);
          else
            c.load(reinterpret_cast<const __nv_bfloat16*>(p.at(GRAD_GATE, group, staged, VEC)), k, u, i0);
        };
        Half m, h, y, g;
        float s[8] = {};
        if (has_z || has_post) {
          float2 s2[6];
#pragma unroll
          for (int j = 0; j < 6; ++j) s2[j] = both(0.0f);
#pragma unroll
          for (int q = 0; q < 2 * K; ++q) {
            const int k = q >> 1, i0 = 4 * (q & 1);
            if (!VEC) asm volatile("" ::: "memory");  // what is loaded of more columns at once would spill
            Half w, d;
            if (has_z) {
              c.load(held_pre, k, w, i0);
              c.load(dz_row, k, m, i0);
              either(GRAD_H, h_kept, k, i0, h);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                m.v[j] = mul2(m.v[j], w.v[j]);
                s2[0] = fma2(h.v[j], h.v[j], s2[0]);
                s2[1] = fma2(m.v[j], h.v[j], s2[1]);
              }
            }
            if (has_post) {
              either(GRAD_Y, y_kept, k, i0, y);
              c.load(held_gw, k, w, i0);
              if (token) gate_unit(k, i0, g);
              if (has_dh) c.load(dh_row, k, d, i0);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float2 gy = mul2(w.v[j], y.v[j]);
                if (token) gy = mul2(gy, g.v[j]);
                s2[2] = fma2(y.v[j], y.v[j], s2[2]);
                if (has_dh) s2[3] = fma2(d.v[j], gy, s2[3]);
                if (has_z) {
                  s2[4] = fma2(m.v[j], gy, s2[4]);
                  s2[5] = fma2(h.v[j], gy, s2[5]);
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 6; ++j) s[j] = s2[j].x + s2[j].y;
          group_sum8<6>(s, words, turn, warps, warp, 1 + group, a.pipe.group);
        }
        p.refill(false);
        const RowFactors f = row_factors(s, inverse, a.eps, a.beta, has_z, has_post);
        const float2 rho2 = both(f.rho), of_h = both(-f.rho * f.back), alpha = both(a.alpha), tau_beta = both(f.tau * a.beta), of_y = both(-f.tau * f.back_y);
#pragma unroll
        for (int q = 0; q < 2 * K; ++q) {
          const int k = q >> 1, i0 = 4 * (q & 1), j0 = i0 / 2;
          const bool there = c.has(k);
          if (!VEC) asm volatile("" ::: "memory");
          Half w, d, out;
          if (has_dh)
            c.load(dh_row, k, d, i0);
          else
            d.fill(0.0f);
          if (has_z) {
            c.load(held_pre, k, w, i0);
            c.load(dz_row, k, m, i0);
            either(GRAD_H, h_kept, k, i0, h);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float2 t = mul2(m.v[j], rho2);
              sum_pre[k].v[j0 + j] = fma2(t, h.v[j], sum_pre[k].v[j0 + j]);
              d.v[j] = fma2(h.v[j], of_h, fma2(t, w.v[j], d.v[j]));
            }
          }
          if (has_dx) {
#pragma unroll
            for (int j = 0; j < 2; ++j) out.v[j] = mul2(d.v[j], alpha);
            if (there) c.store(dx_row, k, out, i0);
          }
          if (has_y) either(GRAD_Y, y_kept, k, i0, y);
          c.load(held_gw, k, w, i0);
          if (token) gate_unit(k, i0, g);
#pragma unroll
          for (int j = 0; j < 2; ++j) d.v[j] = mul2(d.v[j], tau_beta);
          if (has_dy) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              out.v[j] = mul2(d.v[j], w.v[j]);
              if (token) out.v[j] = mul2(out.v[j], g.v[j]);
              if (has_post) out.v[j] = fma2(y.v[j], of_y, out.v[j]);
            }
            if (there) c.store(dy_row, k, out, i0);
          }
          if (has_y) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if (token) {
                const float2 v = mul2(d.v[j], y.v[j]);
                sum_a[k].v[j0 + j] = fma2(g.v[j], v, sum_a[k].v[j0 + j]);
                out.v[j] = mul2(v, w.v[j]);
              } else {
                sum_a[k].v[j0 + j] = fma2(d.v[j], y.v[j], sum_a[k].v[j0 + j]);
              }
            }
            if (token && a.dgate && there) store_sums(a.dgate, row * a.dgate_stride, a.dgate_f32, a.accumulate, c, k, out, i0);
          }
        }
      }
      p.release();
    } while (p.next(rows));
    flush_sums<VEC, K, false>(a, p, c, group, group_sums, columns, token, has_y, has_post, first_flush, sum_a, sum_pre);
#pragma unroll
    for (int k = 0; k < K; ++k) sum_a[k].fill(0.0f);
    first_flush = false;
  } while (p.next_segment());
  p.finish(&g_norm_grad_error);
}

// Four values as they lie, and two of them as fp32.
__device__ __forceinline__ uint2 load_raw(const __nv_bfloat16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ float4 load_raw(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float2 pair(const uint2& r, int i) { return unpack_bf16(i ? r.y : r.x); }
__device__ __forceinline__ float2 pair(const float4& r, int i) { return i ? make_float2(r.z, r.w) : make_float2(r.x, r.y); }

// The same for rows of up to 8192 columns with everything but scales on 16 bytes, with dz,
// no gate per token, and h and y alike: KEPT 0 matrices, 1 integers, 2 e4m3. BLOCK 0: y is
// not read; 1: it is (for a norm behind the block, or the gate's gradient); 2: there is that norm,
// and dh, dx and dy (asking whether costs 16384 x 8192 54 us of 393). h and y stay in registers from the
// row's sums to its results, dh and dz are read from shared memory again: held too, they
// would spill, and with all of the shared memory in use local memory lies in L2. (The
// general kernel, which asks in every unit what there is: 633 us for 16381 x 8192 from
// checkpoints, this one 283.)
// Rows of scales off 16 bytes come with the 16-byte pieces around them: 8192 x 2056 from
// checkpoints 66 us, with the general kernel 136.
// ONE: a row at a time (rows above 2048), whose addresses are then the same in all threads.
template <class T, int KEPT, int BLOCK, bool ONE>
__global__ void __maxnreg__(128) norm_grad_rows_kernel(const __grid_constant__ GradArgs a) {
  constexpr int K = 2;
  extern __shared__ __align__(16) uint8_t smem[];
  let_next_start();
  Pipe<GRAD_OPS, false> p(a.pipe, smem);
  wait_for_previous();
  p.start(a.pipe.pad);
  const int group = ONE ? 0 : threadIdx.x / a.pipe.group, tid = threadIdx.x - group * a.pipe.group, warp = tid >> 5, warps = a.pipe.group >> 5;
  const Cols<true> c = {static_cast<uint32_t>(tid), static_cast<uint32_t>(a.pipe.group), static_cast<uint32_t>(a.pipe.hidden)};
  const float inverse = 1.0f / static_cast<float>(a.pipe.hidden);
  float* const words = p.words() + group * warps * 8;
  int turn = 0;
  const bool has_dh = BLOCK == 2 || a.pipe.in[GRAD_DH].p, has_dx = BLOCK == 2 || a.dx.p, has_dy = BLOCK == 2 || a.dy.p;
  const bool has_post = BLOCK == 2 || (BLOCK == 1 && a.w_post.p);
  const int columns = 8 * K * a.pipe.group;
  float* const group_sums = reinterpret_cast<float*>(smem + kPipeHeader + a.pipe.stages * p.stage_bytes);
  float* const held_pre = group_sums + (ONE ? 0 : a.pipe.groups * 2 * columns);
  float* const held_gw = held_pre + columns;
  Unit sum_pre[K], sum_a[K];
  bool there[K];
#pragma unroll
  for (int k = 0; k < K; ++k) sum_pre[k].fill(0.0f), sum_a[k].fill(0.0f), there[k] = c.has(k);
  bool first_flush = true;
  do {
    // each thread the columns that it reads itself, or one group for all
    if (!ONE) asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
    if (ONE || group == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Unit u, g;
        u.fill(0.0f);
        if (there[k]) c.load_any(a.w_pre.p, a.w_pre.f32, k, u);
        c.store(held_pre, k, u);
        u.fill(there[k] ? 1.0f : 0.0f);
        if (has_post && there[k]) c.load_any(a.w_post.p, a.w_post.f32, k, u);
        if (a.gate.p && there[k]) {
          c.load_any(row_of(a.gate, p.row / a.per_gate), a.gate.f32, k, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], g.v[j]);
        }
        c.store(held_gw, k, u);
      }
    }
    if (!ONE) asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
    int rows;
    do {
      rows = ONE ? 1 : p.rows();
      const bool mine = ONE || group < rows;
      Unit h[K], y[K];
      float s[8] = {};
      p.wait();
      const uint8_t* const staged = p.staged(group);
      const uint8_t *const dz_row = staged + a.pipe.in[GRAD_DZ].slot, *const dh_row = staged + a.pipe.in[GRAD_DH].slot;
      if (mine) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (KEPT == 0) {
            c.load(reinterpret_cast<const T*>(staged + a.pipe.in[GRAD_H].slot), k, h[k]);
            if (BLOCK) c.load(reinterpret_cast<const T*>(staged + a.pipe.in[GRAD_Y].slot), k, y[k]);
          } else {
            c.restore(staged + a.pipe.in[GRAD_H].slot, p.at(GRAD_H_SCALES, group, staged, false), KEPT == 2, k, h[k]);
            if (BLOCK) c.restore(staged + a.pipe.in[GRAD_Y].slot, p.at(GRAD_Y_SCALES, group, staged, false), KEPT == 2, k, y[k]);
          }
        }
      }
      if (mine) {
        float2 t[6];
#pragma unroll
        for (int j = 0; j < 6; ++j) t[j] = both(0.0f);
        // four columns at a time: what is loaded for more would spill
#pragma unroll
        for (int i = 0; i < 2 * K; ++i) {
          const int k = i >> 1, j0 = 2 * (i & 1), u = (tid + k * c.threads) * 8 + 2 * j0;
          asm volatile("" ::: "memory");
          const auto z = load_raw(reinterpret_cast<const T*>(dz_row + sizeof(T) * u));
          const float4 w = *reinterpret_cast<const float4*>(held_pre + u);
          const float2 m0 = mul2(pair(z, 0), make_float2(w.x, w.y)), m1 = mul2(pair(z, 1), make_float2(w.z, w.w));
          const float2 h0 = h[k].v[j0], h1 = h[k].v[j0 + 1];
          t[0] = fma2(h0, h0, t[0]), t[1] = fma2(m0, h0, t[1]);
          t[0] = fma2(h1, h1, t[0]), t[1] = fma2(m1, h1, t[1]);
          if (BLOCK) {
            const auto d = has_dh ? load_raw(reinterpret_cast<const T*>(dh_row + sizeof(T) * u)) : decltype(z){};
            const float4 g = *reinterpret_cast<const float4*>(held_gw + u);
            const float2 y0 = y[k].v[j0], y1 = y[k].v[j0 + 1];
            const float2 q0 = mul2(make_float2(g.x, g.y), y0), q1 = mul2(make_float2(g.z, g.w), y1);
            t[2] = fma2(y0, y0, t[2]), t[3] = fma2(pair(d, 0), q0, t[3]), t[4] = fma2(m0, q0, t[4]), t[5] = fma2(h0, q0, t[5]);
            t[2] = fma2(y1, y1, t[2]), t[3] = fma2(pair(d, 1), q1, t[3]), t[4] = fma2(m1, q1, t[4]), t[5] = fma2(h1, q1, t[5]);
          }
        }
#pragma unroll
        for (int j = 0; j < 6; ++j) s[j] = t[j].x + t[j].y;
        group_sum8<BLOCK ? 6 : 2>(s, words, turn, warps, warp, 1 + group, a.pipe.group);
      }
      if (a.pipe.stages > 1) p.refill(false);
      asm volatile("" ::: "memory");  // what follows is read again
      if (mine) {
        const int64_t row = static_cast<uint32_t>(p.row) + group;
        const RowFactors f = row_factors(s, inverse, a.eps, a.beta, true, has_post);
        const float2 rho2 = both(f.rho), of_h = both(-f.rho * f.back), alpha = both(a.alpha), tau_beta = both(f.tau * a.beta), of_y = both(-f.tau * f.back_y);
        T *const dx_out = row_of<T>(a.dx, row), *const dy_out = row_of<T>(a.dy, row);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Unit dx, dy;
#pragma unroll
          for (int j0 = 0; j0 < 4; j0 += 2) {
            const int u = (tid + k * c.threads) * 8 + 2 * j0;
            asm volatile("" ::: "memory");
            const auto z = load_raw(reinterpret_cast<const T*>(dz_row + sizeof(T) * u));
            const auto d = has_dh ? load_raw(reinterpret_cast<const T*>(dh_row + sizeof(T) * u)) : decltype(z){};
            const float4 w = *reinterpret_cast<const float4*>(held_pre + u), g = *reinterpret_cast<const float4*>(held_gw + u);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int j = j0 + i;
              const float2 t = mul2(pair(z, i), rho2);
              sum_pre[k].v[j] = fma2(t, h[k].v[j], sum_pre[k].v[j]);
              const float2 D = fma2(h[k].v[j], of_h, fma2(t, i ? make_float2(w.z, w.w) : make_float2(w.x, w.y), pair(d, i)));
              dx.v[j] = mul2(D, alpha);
              const float2 e = mul2(D, tau_beta);
              dy.v[j] = mul2(e, i ? make_float2(g.z, g.w) : make_float2(g.x, g.y));
              if (BLOCK) {
                if (has_post) dy.v[j] = fma2(y[k].v[j], of_y, dy.v[j]);
                sum_a[k].v[j] = fma2(e, y[k].v[j], sum_a[k].v[j]);
              }
            }
          }
          if (there[k]) {
            if (has_dx) c.store(dx_out, k, dx);
            if (has_dy) c.store(dy_out, k, dy);
          }
        }
      }
      p.release();
    } while (p.next(rows));
    flush_sums<true, K, ONE>(a, p, c, group, group_sums, columns, false, BLOCK > 0, has_post, first_flush, sum_a, sum_pre);
#pragma unroll
    for (int k = 0; k < K; ++k) sum_a[k].fill(0.0f);
    first_flush = false;
  } while (p.next_segment());
  p.finish(&g_norm_grad_error);
}

cudaError_t take_norm_error(int* out) {
  cudaError_t err = cudaMemcpyFromSymbol(out, g_norm_grad_error, sizeof(int));
  if (err != cudaSuccess || *out == 0) return err;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_norm_grad_error, &zero, sizeof(int));
}

}  // namespace

}  // namespace lst
