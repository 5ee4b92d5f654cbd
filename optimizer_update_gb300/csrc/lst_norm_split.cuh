// The backward pass of the residual norm for rows above 8192 columns, whose sums and values fit
// neither in a CTA's registers nor beside each other in its shared memory: every row's
// statistics, then the gradients by tiles of columns. Inputs are read twice, but neither launch
// holds a row, and the second has no barrier. The mathematics is at the top of lst_norm.cu.
// 4096 x 12288 in bf16: 115 us for the statistics and 195 for the gradients (rows read where they
// are by one kernel that keeps their sums: 636), of 90 that the bytes take once. What bounds both is
// latency: 512 threads an SM with 8 columns each in flight in the second.
#pragma once

#include "lst_norm.cuh"

namespace lst {

namespace {

// What a thread reads of a row, from column `col0` on; with `kept` a checkpoint.
template <class T, bool VEC, int P>
__device__ __forceinline__ void load_operand(const GradArgs& a, int op, int kept, int64_t row, int col0, const Cols<VEC>& c, int k, Part<P>& u, int i0 = 0) {
  const uint8_t* p = a.pipe.in[op].p + row * a.pipe.in[op].stride;
  if (kept == 0)
    c.load(reinterpret_cast<const T*>(p) + col0, k, u, i0);
  else
    c.restore(p + col0, a.pipe.in[op + 1].p + row * a.pipe.in[op + 1].stride + col0 / kCkptBlock, kept == 2, k, u, i0);
}
template <bool VEC, int P>
__device__ __forceinline__ void load_weight(const Weights& w, int64_t row, int col0, const Cols<VEC>& c, int k, Part<P>& u, int i0 = 0) {
  c.load_any(static_cast<const char*>(row_of(w, row)) + static_cast<int64_t>(col0) * (w.f32 ? 4 : 2), w.f32, k, u, i0);
}

// rho, the factor of h in D, tau b and the factor of y in dy, of every row, a CTA a row. The
// sums are those of norm_grad_kernel.
template <class T, bool VEC>
__global__ void __launch_bounds__(256, 4) norm_stats_kernel(const __grid_constant__ GradArgs a) {
  __shared__ float words[256];
  // 16 bytes a load and operand at once, as much as the 64 registers of four CTAs an SM hold (bf16: but 68 bytes)
  constexpr int P = VEC && sizeof(T) == 2 ? 4 : 2, kUnroll = P == 4 ? 1 : 2;
  let_next_start();
  wait_for_previous();
  const Cols<VEC> c = {threadIdx.x, 256u, static_cast<uint32_t>(a.pipe.hidden)};
  const float inverse = 1.0f / static_cast<float>(a.pipe.hidden);
  const bool has_dh = a.pipe.in[GRAD_DH].p != nullptr, has_z = a.pipe.in[GRAD_DZ].p != nullptr, has_post = a.w_post.p != nullptr;
  const int units = (a.pipe.hidden + 8 * 256 - 1) / (8 * 256);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.pipe.tokens; row += gridDim.x) {
    float2 s2[6];
#pragma unroll
    for (int j = 0; j < 6; ++j) s2[j] = both(0.0f);
#pragma unroll kUnroll
    for (int q = 0; q < (4 / P) * units; ++q) {
      const int k = P == 4 ? q : q >> 1, i0 = P == 4 ? 0 : 4 * (q & 1);
      if (!c.has(k)) continue;
      Part<P> m, h, y, w, g, d;
      if (has_z) {
        load_weight(a.w_pre, 0, 0, c, k, w, i0);
        load_operand<T>(a, GRAD_DZ, 0, row, 0, c, k, m, i0);
        load_operand<T>(a, GRAD_H, a.h_kept, row, 0, c, k, h, i0);
      }
      if (has_post) {
        load_operand<T>(a, GRAD_Y, a.y_kept, row, 0, c, k, y, i0);
        load_weight(a.w_post, 0, 0, c, k, g, i0);
        if (has_dh) load_operand<T>(a, GRAD_DH, 0, row, 0, c, k, d, i0);
        if (a.gate.p) {
          Part<P> of_gate;
          load_weight(a.gate, row / a.per_gate, 0, c, k, of_gate, i0);
#pragma unroll
          for (int j = 0; j < P; ++j) g.v[j] = mul2(g.v[j], of_gate.v[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (has_z) {
          m.v[j] = mul2(m.v[j], w.v[j]);
          s2[0] = fma2(h.v[j], h.v[j], s2[0]);
          s2[1] = fma2(m.v[j], h.v[j], s2[1]);
        }
        if (has_post) {
          const float2 gy = mul2(g.v[j], y.v[j]);
          s2[2] = fma2(y.v[j], y.v[j], s2[2]);
          if (has_dh) s2[3] = fma2(d.v[j], gy, s2[3]);
          if (has_z) {
            s2[4] = fma2(m.v[j], gy, s2[4]);
            s2[5] = fma2(h.v[j], gy, s2[5]);
          }
        }
      }
    }
    float s[8] = {};
#pragma unroll
    for (int j = 0; j < 6; ++j) s[j] = s2[j].x + s2[j].y;
    group_sum8<6>(s, words, turn, 8, threadIdx.x >> 5, 1, 256);
    if (threadIdx.x == 0) {
      const RowFactors f = row_factors(s, inverse, a.eps, a.beta, has_z, has_post);
      a.stats[row] = make_float4(f.rho, -f.rho * f.back, f.tau * a.beta, -f.tau * f.back_y);
    }
  }
}

// Tile blockIdx.x of the columns, rows first_row(blockIdx.y) on.
template <class T, bool VEC>
__global__ void __launch_bounds__(kSplitTile / 8, split_ctas(VEC)) norm_apply_kernel(const __grid_constant__ GradArgs a) {
  // Pairs of columns at a time: whole units, of which 140 bytes a thread spill, or in single values halves of
  // them, with twice the threads an SM on 64 registers and 544 bytes that spill.
  constexpr int P = VEC ? 4 : 2;
  let_next_start();
  wait_for_previous();
  const int hidden = a.pipe.hidden, ld = (hidden + 3) & ~3, col0 = blockIdx.x * kSplitTile;
  const Cols<VEC> c = {threadIdx.x, kSplitTile / 8, static_cast<uint32_t>(min(hidden - col0, kSplitTile))};
  const bool there = c.has(0), has_dh = a.pipe.in[GRAD_DH].p != nullptr, has_z = a.pipe.in[GRAD_DZ].p != nullptr;
  const bool has_y = a.pipe.in[GRAD_Y].p != nullptr, has_post = a.w_post.p != nullptr, token = a.token != 0, stats = has_z || has_post;
  const int64_t chunk = blockIdx.y, begin = first_row(chunk, a.pipe.tokens, a.pipe.ctas), end = first_row(chunk + 1, a.pipe.tokens, a.pipe.ctas);
  Unit pre, gw, sum_a, sum_pre, post;
  sum_a.fill(0.0f), sum_pre.fill(0.0f), post.fill(0.0f), pre.fill(0.0f);
  if (has_z && there) load_weight(a.w_pre, 0, col0, c, 0, pre);
  int64_t row = begin;
  while (row < end) {
    const int64_t gate_row = row / a.per_gate, segment = token ? end : min(end, (gate_row + 1) * a.per_gate);
    gw.fill(1.0f);
    if (has_post && there) load_weight(a.w_post, 0, col0, c, 0, gw);
    if (!token && a.gate.p && there) {
      Unit g;
      load_weight(a.gate, gate_row, col0, c, 0, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) gw.v[j] = mul2(gw.v[j], g.v[j]);
    }
    sum_a.fill(0.0f);
    if (there) {
#pragma unroll 1
      for (int64_t r = row; r < segment; ++r) {
        const float4 st = stats ? a.stats[r] : make_float4(0.0f, 0.0f, a.beta, 0.0f);
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 2 * P) {
          Part<P> d, z, h, y, g, out;
          d.fill(0.0f);
          if (has_dh) load_operand<T>(a, GRAD_DH, 0, r, col0, c, 0, d, i0);
          if (has_z) {
            load_operand<T>(a, GRAD_DZ, 0, r, col0, c, 0, z, i0);
            load_operand<T>(a, GRAD_H, a.h_kept, r, col0, c, 0, h, i0);
          }
          if (has_y) load_operand<T>(a, GRAD_Y, a.y_kept, r, col0, c, 0, y, i0);
          if (token) load_weight(a.gate, r, col0, c, 0, g, i0);
          if (has_z) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              const float2 t = mul2(z.v[j], both(st.x));
              sum_pre.v[i0 / 2 + j] = fma2(t, h.v[j], sum_pre.v[i0 / 2 + j]);
              d.v[j] = fma2(h.v[j], both(st.y), fma2(t, pre.v[i0 / 2 + j], d.v[j]));
            }
          }
          if (a.dx.p) {
#pragma unroll
            for (int j = 0; j < P; ++j) out.v[j] = mul2(d.v[j], both(a.alpha));
            c.store(row_of<T>(a.dx, r) + col0, 0, out, i0);
          }
#pragma unroll
          for (int j = 0; j < P; ++j) d.v[j] = mul2(d.v[j], both(st.z));
          if (a.dy.p) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              out.v[j] = mul2(d.v[j], gw.v[i0 / 2 + j]);
              if (token) out.v[j] = mul2(out.v[j], g.v[j]);
              if (has_post) out.v[j] = fma2(y.v[j], both(st.w), out.v[j]);
            }
            c.store(row_of<T>(a.dy, r) + col0, 0, out, i0);
          }
          if (has_y) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
              const float2 v = mul2(d.v[j], y.v[j]);
              sum_a.v[i0 / 2 + j] = token ? fma2(g.v[j], v, sum_a.v[i0 / 2 + j]) : add2(v, sum_a.v[i0 / 2 + j]);
              out.v[j] = mul2(v, gw.v[i0 / 2 + j]);
            }
            if (token && a.dgate) store_sums(a.dgate, r * a.dgate_stride + col0, a.dgate_f32, a.accumulate, c, 0, out, i0);
          }
        }
      }
    }
    if (!a.single && has_y && there) {
      Unit u;
      load_weight(a.gate, gate_row, col0, c, 0, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) post.v[j] = fma2(sum_a.v[j], u.v[j], post.v[j]);
      if (a.dgate) {
        if (has_post) {
          load_weight(a.w_post, 0, col0, c, 0, u);
#pragma unroll
          for (int j = 0; j < 4; ++j) sum_a.v[j] = mul2(sum_a.v[j], u.v[j]);
        }
        if (gate_row * a.per_gate >= begin && (gate_row + 1) * a.per_gate <= end)
          store_sums(a.dgate, gate_row * a.dgate_stride + col0, a.dgate_f32, a.accumulate, c, 0, sum_a);
        else
          c.store(a.part_gate + (2 * chunk + (gate_row == begin / a.per_gate ? 0 : 1)) * ld + col0, 0, sum_a);
      }
    }
    row = segment;
  }
  if (!there) return;
  if (has_y && a.part_post) c.store(a.part_post + chunk * ld + col0, 0, a.single ? sum_a : post);
  if (a.part_pre) c.store(a.part_pre + chunk * ld + col0, 0, sum_pre);
}

}  // namespace

}  // namespace lst
