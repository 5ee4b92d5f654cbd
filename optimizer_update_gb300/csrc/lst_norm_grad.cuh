// The backward kernel of the residual norm; the mathematics is at the top of lst_norm.cu.
#pragma once

#include "lst_norm.cuh"

namespace lst {

namespace {

__device__ int g_norm_grad_error;

// A unit of a row of parameter gradients that starts at element `at`.
template <bool VEC>
__device__ __forceinline__ void store_sums(void* p, int64_t at, bool f32, bool accumulate, const Cols<VEC>& c, int k, const Unit& u) {
  if (VEC && !accumulate && (reinterpret_cast<uintptr_t>(p) + at * (f32 ? 4 : 2)) % 16 == 0) {
    if (f32)
      c.store(static_cast<float*>(p) + at, k, u);
    else
      c.store(static_cast<__nv_bfloat16*>(p) + at, k, u);
  } else {
    for_each(c, k, u, [&](uint32_t col, float v) { store_sum(p, at + col, f32, accumulate, v); });
  }
}

// With q = g w_post y, the six sums h^2, m h, y^2, dh q, m q and h q of a row give both
// norms' statistics at once, for D is linear in dh, m and h:
//   sum e y = b (sum dh q + rho (sum m q - rho^2 mean(m h) sum h q)),
// so a row needs one barrier instead of two. Its roundings are those of D's own terms.
// FORM: what is there, where the kernel is made for it (the checks
// of every operand in every unit were a third of the instructions): 0 whatever the call
// has; all of dh, dz, dx and dy, and 1 h and y as matrices, 2 as integers, 3 as e4m3; 4 to 6
// the same without y (no norm after the block); 1 to 6 without a gate per token.
template <class T, bool VEC, int K, bool STAGED, int FORM>
__global__ void __maxnreg__(128) norm_grad_kernel(const __grid_constant__ GradArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  let_next_start();
  Pipe<GRAD_OPS, STAGED> p(a.pipe, smem);
  wait_for_previous();
  p.start(VEC && a.pipe.pad);
  const int group = threadIdx.x / a.pipe.group, tid = threadIdx.x - group * a.pipe.group, warp = tid >> 5, warps = a.pipe.group >> 5;
  const int64_t cta = blockIdx.x;
  Cols<VEC> c = {static_cast<uint32_t>(tid), static_cast<uint32_t>(a.pipe.group), static_cast<uint32_t>(a.pipe.hidden)};
  const int hidden = a.pipe.hidden;
  const float inverse = 1.0f / static_cast<float>(hidden);
  const bool has_dh = FORM ? true : a.pipe.in[GRAD_DH].p != nullptr, has_z = FORM ? true : a.pipe.in[GRAD_DZ].p != nullptr;
  const bool has_post = FORM ? FORM <= 3 : a.w_post.p != nullptr, has_y = FORM ? FORM <= 3 : a.pipe.in[GRAD_Y].p != nullptr;
  const bool has_dx = FORM ? true : a.dx.p != nullptr, has_dy = FORM ? true : a.dy.p != nullptr;
  const int h_kept = FORM ? (FORM - 1) % 3 : a.h_kept, y_kept = FORM ? (FORM - 1) % 3 : a.y_kept;
  const bool token = FORM ? false : a.pipe.in[GRAD_GATE].p != nullptr;  // a gate per token
  float* const words = p.words() + group * warps * 8;
  int turn = 0;
  // weights as fp32 in shared memory, where registers would spill; K = 4 reads them again for every row
  constexpr bool kHold = K <= 2;
  constexpr bool kPadded = VEC && STAGED;  // units behind the row are zeros there: only stores pass over them
  const int columns = kPadded ? 8 * K * a.pipe.group : hidden;
  float* const group_sums = reinterpret_cast<float*>(smem + kPipeHeader + a.pipe.stages * p.stage_bytes);
  float* const held_pre = group_sums + (a.pipe.groups > 1 ? a.pipe.groups * 2 * columns : 0);
  float* const held_gw = held_pre + columns;
  Unit sum_pre[K], sum_a[K];
  // w_pre and gate * w_post of unit k (a gate per token comes with the row)
  auto load_pre = [&](int k, Unit& u) {
    if (has_z) c.load_any(a.w_pre.p, a.w_pre.f32, k, u);
  };
  auto load_gw = [&](int row, int k, Unit& u) {
    u.fill(1.0f);
    if (has_post) c.load_any(a.w_post.p, a.w_post.f32, k, u);
    if (!token && a.gate.p) {
      Unit g;
      c.load_any(row_of(a.gate, row / a.per_gate), a.gate.f32, k, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) u.v[j] = mul2(u.v[j], g.v[j]);
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) sum_pre[k].fill(0.0f), sum_a[k].fill(0.0f);
  bool first_flush = true;
  do {
    if (kHold) {
      // each thread the columns that it reads itself, or one group for all
      if (a.pipe.groups > 1) asm volatile("bar.sync 15, %0;" ::"r"(blockDim.x) : "memory");
      if (group == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          Unit u;
          u.fill(0.0f);
          if (has_z && c.has(k)) load_pre(k, u);
          c.store(held_pre, k, u);
          u.fill(0.0f);
          if (c.has(k)) load_gw(p.row, k, u);
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
      if (group < rows) {
        const int64_t row = p.row + group;
        auto pre_unit = [&](int k, Unit& u) {
          if (kHold)
            c.load(held_pre, k, u);
          else
            load_pre(k, u);
        };
        auto gw_unit = [&](int k, Unit& u) {
          if (kHold)
            c.load(held_gw, k, u);
          else
            load_gw(p.row + group, k, u);
        };
        const uint8_t* const staged = p.staged(group);
        T *const dx_row = row_of<T>(a.dx, row), *const dy_row = row_of<T>(a.dy, row);
        const T* const dh_row = reinterpret_cast<const T*>(p.at(GRAD_DH, group, staged, VEC));
        const T* const dz_row = reinterpret_cast<const T*>(p.at(GRAD_DZ, group, staged, VEC));
        auto either = [&](int op, int kept, int k, Unit& u) {
          if (kept == 0)
            c.load(reinterpret_cast<const T*>(p.at(op, group, staged, VEC)), k, u);
          else
            c.restore(p.at(op, group, staged, true), p.at(op + 1, group, staged, false), kept == 2, k, u);
        };
        auto gate_unit = [&](int k, Unit& u) {
          if (a.gate.f32)
            c.load(reinterpret_cast<const float*>(p.at(GRAD_GATE, group, staged, VEC)), k, u);
          else
            c.load(reinterpret_cast<const __nv_bfloat16*>(p.at(GRAD_GATE, group, staged, VEC)), k, u);
        };
        Unit m, h, y, g;
        float s[8] = {};
        if (has_z || has_post) {
          float2 s2[6];
#pragma unroll
          for (int j = 0; j < 6; ++j) s2[j] = both(0.0f);
#pragma unroll
          for (int k = 0; k < K; ++k) {
            if (!kPadded && !c.has(k)) continue;
            Unit w, d;
            if (has_z) {
              pre_unit(k, w);
              c.load(dz_row, k, m);
              either(GRAD_H, h_kept, k, h);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                m.v[j] = mul2(m.v[j], w.v[j]);
                s2[0] = fma2(h.v[j], h.v[j], s2[0]);
                s2[1] = fma2(m.v[j], h.v[j], s2[1]);
              }
            }
            if (has_post) {
              either(GRAD_Y, y_kept, k, y);
              gw_unit(k, w);
              if (token) gate_unit(k, g);
              if (has_dh) c.load(dh_row, k, d);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float2 q = mul2(w.v[j], y.v[j]);
                if (token) q = mul2(q, g.v[j]);
                s2[2] = fma2(y.v[j], y.v[j], s2[2]);
                if (has_dh) s2[3] = fma2(d.v[j], q, s2[3]);
                if (has_z) {
                  s2[4] = fma2(m.v[j], q, s2[4]);
                  s2[5] = fma2(h.v[j], q, s2[5]);
                }
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 6; ++j) s[j] = s2[j].x + s2[j].y;
          group_sum8<6>(s, words, turn, warps, warp, 1 + group, a.pipe.group);
        }
        p.refill(false);
        const float rho = has_z ? rsqrtf(s[0] * inverse + a.eps) : 0.0f, back = rho * rho * (s[1] * inverse);
        const float tau = has_post ? rsqrtf(s[2] * inverse + a.eps) : 1.0f;
        const float back_y = has_post ? tau * tau * (a.beta * (s[3] + rho * (s[4] - back * s[5])) * inverse) : 0.0f;
        const float2 rho2 = both(rho), of_h = both(-rho * back), alpha = both(a.alpha), tau_beta = both(tau * a.beta), of_y = both(-tau * back_y);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const bool there = c.has(k);
          if (!kPadded && !there) continue;
          Unit w, d, out;
          if (has_dh)
            c.load(dh_row, k, d);
          else
            d.fill(0.0f);
          if (has_z) {
            pre_unit(k, w);
            c.load(dz_row, k, m);
            either(GRAD_H, h_kept, k, h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 t = mul2(m.v[j], rho2);
              sum_pre[k].v[j] = fma2(t, h.v[j], sum_pre[k].v[j]);
              d.v[j] = fma2(h.v[j], of_h, fma2(t, w.v[j], d.v[j]));
            }
          }
          if (has_dx) {
#pragma unroll
            for (int j = 0; j < 4; ++j) out.v[j] = mul2(d.v[j], alpha);
            if (there) c.store(dx_row, k, out);
          }
          if (has_y) either(GRAD_Y, y_kept, k, y);
          gw_unit(k, w);
          if (token) gate_unit(k, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) d.v[j] = mul2(d.v[j], tau_beta);
          if (has_dy) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              out.v[j] = mul2(d.v[j], w.v[j]);
              if (token) out.v[j] = mul2(out.v[j], g.v[j]);
              if (has_post) out.v[j] = fma2(y.v[j], of_y, out.v[j]);
            }
            if (there) c.store(dy_row, k, out);
          }
          if (has_y) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (token) {
                const float2 v = mul2(d.v[j], y.v[j]);
                sum_a[k].v[j] = fma2(g.v[j], v, sum_a[k].v[j]);
                out.v[j] = mul2(v, w.v[j]);
              } else {
                sum_a[k].v[j] = fma2(d.v[j], y.v[j], sum_a[k].v[j]);
              }
            }
            if (token && a.dgate && there) store_sums(a.dgate, row * a.dgate_stride, a.dgate_f32, a.accumulate, c, k, out);
          }
        }
      }
      p.release();
    } while (p.next(rows));
    // the sums of a gate row, or of all of the CTA's rows
    const bool last = p.row >= p.end;
    const int64_t gate_row = (p.segment - 1) / a.per_gate;
    const bool whole = gate_row * a.per_gate >= p.begin && (gate_row + 1) * a.per_gate <= p.end;
    float* const gate_sums = a.part_gate + (2 * cta + (gate_row == p.begin / a.per_gate ? 0 : 1)) * hidden;
    float *const post = a.part_post + cta * hidden, *const pre = a.part_pre + cta * hidden;
    const bool gated = !token && a.gate.p, gates = !token && has_y && a.dgate, posts = has_y && a.part_post, pres = last && a.part_pre;
    if (a.pipe.groups == 1) {
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
