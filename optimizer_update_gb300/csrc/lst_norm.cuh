// What the residual-norm kernels share (lst_norm.cu, lst_norm_grad.cuh): arguments, the
// pipe that brings rows to shared memory, sums over a row.
#pragma once

#include "lst_ckpt.cuh"
#include "lst_tc.cuh"

namespace lst {

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
__device__ __forceinline__ float weight_at(const Weights& w, int64_t r, int64_t col) {
  const void* p = row_of(w, r);
  return w.f32 ? static_cast<const float*>(p)[col] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[col]);
}

// f(column, value) for the columns of a unit, or of a half of it
template <bool VEC, int P, class F>
__device__ __forceinline__ void for_each(const Cols<VEC>& c, int k, const Part<P>& u, F f, int i0 = 0) {
  c.template each<P>(k, i0, [&](int i, uint32_t e, bool inside) {
    if (inside) f(e, u.at(i));
  });
}

// ---- rows through shared memory ----------------------------------------------------
// A CTA takes consecutive rows, `groups` at a time (a turn), each by a group of `group`
// threads. What a row reads are ranges of bytes (a checkpoint's values and scales are
// two); they come to shared memory by bulk copies some turns ahead of their use, which
// holds more bytes in flight than registers can.
struct Range {
  const uint8_t* p;  // row 0, or null
  int64_t stride;    // bytes
  int32_t bytes, slot;  // of a row; where it lies in a staged row
};
template <int OPS>
struct PipeArgs {
  Range in[OPS];
  int32_t tokens, per_segment;  // no turn holds rows of two segments (gate rows)
  int32_t hidden, ctas, group, groups, row_bytes, stages, pad;
  int32_t simple, row_total;  // all ranges on 16 bytes, and their bytes in a row
  int32_t margin;             // rows that span 15 bytes in every range
  int32_t step;               // from a turn's first row to the next one's where CTAs take turns of rows (one segment only), or 0
};

// First row of CTA c: the rows divided evenly.
__host__ __device__ __forceinline__ int64_t first_row(int64_t c, int64_t tokens, int64_t ctas) { return c * tokens / ctas; }

// Bulk copies go from and to 16-byte boundaries; up to 15 bytes at either end of a range
// are copied by lanes. A range keeps its offset from such a boundary.
struct Piece {
  const uint8_t* src;
  uint32_t dst;
  int head, mid, tail;
};
__device__ __forceinline__ Piece piece_of(const Range& r, int64_t row, uint32_t slot) {
  Piece p = {nullptr, 0, 0, 0, 0};
  if (!r.p) return p;
  p.src = r.p + row * r.stride;
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p.src) & 15);
  p.dst = slot + r.slot + off;
  p.head = min(r.bytes, (16 - off) & 15);
  p.tail = (r.bytes - p.head) & 15;
  p.mid = r.bytes - p.head - p.tail;
  return p;
}

constexpr int kMaxStages = 4;
constexpr int kPipeHeader = 64 + 2 * 16 * 8 * 4;  // barriers; two turns of 16 warps' sums

// The rows from `ahead` on where some range is not on 16 bytes, `margin` rows from the first
// and the last of all, so that the 16-byte pieces around a range's ends lie within the
// matrix (what else they hold goes to a place's slack and is not used).
template <int OPS>
__device__ __forceinline__ void fill_rounded(const PipeArgs<OPS>& a, int ahead, int n, uint32_t to, uint32_t bar) {
  const int lane = threadIdx.x & 31;
  const bool mine = lane < OPS && a.in[lane].p;
  const Range& r = a.in[mine ? lane : 0];
  int bytes = 0;
  for (int i = 0; i < n && mine; ++i) {
    const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(r.p)) + static_cast<uint32_t>(ahead + i) * static_cast<uint32_t>(r.stride);
    bytes += ((low & 15) + r.bytes + 15) & ~15;
  }
  bytes = __reduce_add_sync(0xffffffffu, bytes);
  tc::fence_async_proxy_cta();  // lanes' bytes of the stage's last use, which may have been fill_ragged's, before these copies
  if (lane == 0) tc::mbar_expect_tx(bar, bytes);
  __syncwarp();
  for (int i = 0; i < n && mine; ++i) {
    const uint8_t* src = r.p + (ahead + i) * r.stride;
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
    tc::bulk_load(to + i * a.row_bytes + r.slot, src - off, (off + r.bytes + 15) & ~15, bar);
  }
  if (lane == 0) tc::mbar_arrive(bar);
}
// The same for any rows, byte by byte at a range's ends.
template <int OPS>
__device__ __forceinline__ void fill_ragged(const PipeArgs<OPS>& a, int ahead, int n, uint32_t to, uint32_t bar) {
  const int lane = threadIdx.x & 31, pieces = n * OPS;
  int bytes = 0;
  bool edges = false;
  for (int i = lane; i < pieces; i += 32) {
    const Piece p = piece_of(a.in[i % OPS], ahead + i / OPS, to + (i / OPS) * a.row_bytes);
    bytes += p.mid;
    edges |= p.head + p.tail > 0;
  }
  bytes = __reduce_add_sync(0xffffffffu, bytes);
  edges = __any_sync(0xffffffffu, edges);
  tc::fence_async_proxy_cta();  // lanes' bytes of the stage's last use before this one's copies, whether or not it has such bytes itself
  if (lane == 0) tc::mbar_expect_tx(bar, bytes);
  __syncwarp();
  for (int i = lane; i < pieces; i += 32) {
    const Piece p = piece_of(a.in[i % OPS], ahead + i / OPS, to + (i / OPS) * a.row_bytes);
    if (p.mid > 0) tc::bulk_load(p.dst + p.head, p.src + p.head, p.mid, bar);
  }
  if (edges) {
    for (int r = 0; r < n; ++r) {
      uint32_t v[OPS], at[OPS];
#pragma unroll
      for (int j = 0; j < OPS; ++j) {
        const Piece p = piece_of(a.in[j], ahead + r, to + r * a.row_bytes);
        const int k = lane & 15, from = lane < 16 ? k : p.head + p.mid + k;
        at[j] = k < (lane < 16 ? p.head : p.tail) ? p.dst + from : 0u;
        if (at[j]) v[j] = p.src[from];
      }
#pragma unroll
      for (int j = 0; j < OPS; ++j)
        if (at[j]) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at[j]), "r"(v[j]) : "memory");
    }
  }
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
}

// The same where only scales (operands 3 and 5 of the backward pass) are not on 16 bytes, in
// few registers: their rows beside the first and the last of all go byte by byte.
template <int OPS>
__device__ __forceinline__ void fill_scales(const PipeArgs<OPS>& a, int ahead, int n, uint32_t to, uint32_t bar) {
  const int lane = threadIdx.x & 31;
  const bool mine = lane < OPS && a.in[lane].p, scales = lane == 3 || lane == 5;
  const Range& r = a.in[mine ? lane : 0];
  auto inside = [&](int row) { return !scales || (row >= a.margin && row < a.tokens - a.margin); };
  auto low_bits = [&](const Range& x, int row) {
    return (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x.p)) + static_cast<uint32_t>(row) * static_cast<uint32_t>(x.stride)) & 15;
  };
  int bytes = 0;
#pragma unroll 1
  for (int i = 0; i < n && mine; ++i)
    if (inside(ahead + i)) bytes += (low_bits(r, ahead + i) + r.bytes + 15) & ~15;
  bytes = __reduce_add_sync(0xffffffffu, bytes);
  tc::fence_async_proxy_cta();  // lanes' bytes of the stage's last use before this one's copies
  if (lane == 0) tc::mbar_expect_tx(bar, bytes);
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < n && mine; ++i) {
    if (!inside(ahead + i)) continue;
    const int off = low_bits(r, ahead + i);
    tc::bulk_load(to + i * a.row_bytes + r.slot, r.p + static_cast<int64_t>(ahead + i) * r.stride - off, (off + r.bytes + 15) & ~15, bar);
  }
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    if (ahead + i >= a.margin && ahead + i < a.tokens - a.margin) continue;
#pragma unroll 1
    for (int op = 3; op <= 5; op += 2) {
      const Range& x = a.in[op];
      if (!x.p) continue;
      const uint8_t* src = x.p + static_cast<int64_t>(ahead + i) * x.stride;
      const uint32_t dst = to + i * a.row_bytes + x.slot + low_bits(x, ahead + i);
#pragma unroll 1
      for (int b = lane; b < x.bytes; b += 32) asm volatile("st.shared.u8 [%0], %1;" ::"r"(dst + b), "r"(static_cast<uint32_t>(src[b])) : "memory");
    }
  }
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(bar);
}

// With RAGGED false all ranges but scales are on 16 bytes.
template <int OPS, bool RAGGED = true>
struct Pipe {
  const PipeArgs<OPS>& a;
  uint8_t* smem;
  uint32_t full, empty;
  int begin, end, row, segment;   // rows of this CTA, of this turn, and where its segment ends
  int ahead, ahead_segment;       // the next turn to be filled
  int stage_bytes, stage, into;
  const uint8_t* current;  // the stage of this turn
  uint32_t phase;
  bool ok;

  __device__ __forceinline__ Pipe(const PipeArgs<OPS>& args, uint8_t* shared) : a(args), smem(shared) {
    full = tc::smem_addr(smem), empty = full + 8 * kMaxStages;
    stage_bytes = a.row_bytes * a.groups;
    stage = into = 0, phase = 0, ok = true;
    current = smem + kPipeHeader;
    for (int i = threadIdx.x; i < 256; i += blockDim.x) words()[i] = 0.0f;
    if (threadIdx.x == 0) {
      for (int i = 0; i < a.stages; ++i) {
        tc::mbar_init(full + 8 * i, 2);
        tc::mbar_init(empty + 8 * i, blockDim.x >> 5);
      }
      tc::mbar_init_fence();
    }
    __syncthreads();
    begin = row = ahead = a.step ? static_cast<int>(blockIdx.x) * a.groups : static_cast<int>(first_row(blockIdx.x, a.tokens, a.ctas));
    end = a.step ? a.tokens : static_cast<int>(first_row(blockIdx.x + 1, a.tokens, a.ctas));
    segment = ahead_segment = segment_end(begin);
  }
  __device__ __forceinline__ int segment_end(int r) const {
    return static_cast<int>(min(static_cast<int64_t>(end), (r / a.per_segment + int64_t(1)) * a.per_segment));
  }
  __device__ __forceinline__ int rows() const { return min(a.groups, segment - row); }
  // Warp 0 fills stage `into` with the next turn's rows. `full` takes two arrivals: the
  // first with the bytes of the bulk copies, the second when the lanes' bytes are there.
  __device__ __forceinline__ void fill() {
    const int lane = threadIdx.x & 31, n = min(a.groups, ahead_segment - ahead);
    const uint32_t to = tc::smem_addr(smem + kPipeHeader) + into * stage_bytes, bar = full + 8 * into;
    if (a.simple) {
      // whole rows by bulk copies, a lane an operand: all other warps wait for this one
      if (lane == 0) tc::mbar_expect_tx(bar, n * a.row_total);
      __syncwarp();
      if (lane < OPS && a.in[lane].p) {
        const Range& r = a.in[lane];
        const uint8_t* src = r.p + ahead * r.stride;
        for (int i = 0; i < n; ++i) tc::bulk_load(to + i * a.row_bytes + r.slot, src + i * r.stride, r.bytes, bar);
      }
      if (lane == 0) tc::mbar_arrive(bar);
    } else if (!RAGGED) {
      fill_scales<OPS>(a, ahead, n, to, bar);
    } else if (ahead >= a.margin && ahead + n <= a.tokens - a.margin) {
      fill_rounded<OPS>(a, ahead, n, to, bar);
    } else {
      fill_ragged<OPS>(a, ahead, n, to, bar);
    }
    ahead = static_cast<int>(min(static_cast<int64_t>(ahead) + (a.step ? a.step : n), int64_t(INT32_MAX)));
    if (ahead == ahead_segment && ahead < end) ahead_segment = segment_end(ahead);
    if (++into == a.stages) into = 0;
  }
  // With `pad`, ranges are shorter than their places in a stage, where zeros stand behind them.
  __device__ __forceinline__ void start(bool pad) {
    if (pad) {
      uint4* const p = reinterpret_cast<uint4*>(smem + kPipeHeader);
      for (int i = threadIdx.x; i < a.stages * stage_bytes / 16; i += blockDim.x) p[i] = make_uint4(0, 0, 0, 0);
      tc::fence_async_proxy_cta();
      __syncthreads();
    }
    if (threadIdx.x < 32)
      for (int i = 0; i < a.stages && ahead < end; ++i) fill();
  }
  // Warp 0, while a turn is under way: the stage of the turn before is filled again (a
  // warp for that alone would cost the others an eighth of their registers). A lone
  // stage is filled again at its turn's end.
  __device__ __forceinline__ void refill(bool lone) {
    if (threadIdx.x >= 32 || ahead >= end || lone != (a.stages == 1) || (!lone && row == begin)) return;
    const uint32_t parity = lone || stage > 0 ? phase : phase ^ 1;
    ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(empty + 8 * into, parity));
    if (ok) fill();
  }
  __device__ __forceinline__ void wait() {
    ok = ok && tc::mbar_wait(full + 8 * stage, phase);
  }
  // The staged row of group `g` in this turn, and operand `op` of it; `aligned`: its rows are on 16 bytes.
  __device__ __forceinline__ const uint8_t* staged(int g) const {
    return current + g * a.row_bytes;
  }
  __device__ __forceinline__ const uint8_t* at(int op, int g, const uint8_t* staged_row, bool aligned) const {
    if (aligned) return staged_row + a.in[op].slot;
    const uint32_t low = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(a.in[op].p)) +
                         static_cast<uint32_t>(row + g) * static_cast<uint32_t>(a.in[op].stride);
    return staged_row + a.in[op].slot + (low & 15);
  }
  // This warp has read the turn's rows.
  __device__ __forceinline__ void release() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(empty + 8 * stage);
  }
  // The next turn; false behind the last of a segment.
  __device__ __forceinline__ bool next(int n) {
    refill(true);
    current += stage_bytes;
    if (++stage == a.stages) stage = 0, phase ^= 1, current = smem + kPipeHeader;
    row = static_cast<int>(min(static_cast<int64_t>(row) + (a.step ? a.step : n), int64_t(INT32_MAX)));
    return row < segment;
  }
  // The next segment; false behind the last.
  __device__ __forceinline__ bool next_segment() {
    if (row >= end) return false;
    segment = segment_end(row);
    return true;
  }
  // A wait ran out (all later ones are passed over): copies in flight get time to land before the CTA ends.
  __device__ __forceinline__ void finish(int* error) {
    if (!ok) {
      atomicExch(error, 1);
      for (int i = 0; i < 1000; ++i) __nanosleep(1000);
    }
  }
  __device__ __forceinline__ float* words() const { return reinterpret_cast<float*>(smem + 64); }
};

// Sum of v over the threads of a row's group, in each of them: `words` holds 16 values of a
// group, zeros behind its warps'. Calls take alternate halves of them (`turn`), so that one
// barrier is enough; every thread adds up the warps' sums itself, which takes less time
// than four exchanges.
__device__ __forceinline__ float group_sum(float v, float* words, int& turn, int warps, int warp, int bar, int threads) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (warps == 1) return v;
  words += turn * 128;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) words[warp] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
  const float4* const q = reinterpret_cast<const float4*>(words);
  const float4 a = q[0], b = q[1];
  v = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
  if (warps > 8) {
    const float4 c = q[2], d = q[3];
    v += ((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w));
  }
  return v;
}
// The same for 8 values: lanes exchange halves, quarters and eighths of them (9 shuffles
// instead of 40). The first `kWanted` are given back.
template <int kWanted>
__device__ __forceinline__ void group_sum8(float (&v)[8], float* words, int& turn, int warps, int warp, int bar, int threads) {
  const int lane = threadIdx.x & 31;
  float u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float mine = lane & 16 ? v[j + 4] : v[j], other = lane & 16 ? v[j] : v[j + 4];
    u[j] = mine + __shfl_xor_sync(0xffffffffu, other, 16);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float mine = lane & 8 ? u[j + 2] : u[j], other = lane & 8 ? u[j] : u[j + 2];
    u[j] = mine + __shfl_xor_sync(0xffffffffu, other, 8);
  }
  float s = (lane & 4 ? u[1] : u[0]) + __shfl_xor_sync(0xffffffffu, lane & 4 ? u[0] : u[1], 4);
  s += __shfl_xor_sync(0xffffffffu, s, 2);
  s += __shfl_xor_sync(0xffffffffu, s, 1);  // value lane / 4
  if (warps > 1) {
    words += turn * 128;
    turn ^= 1;
    if ((lane & 3) == 0) words[warp * 8 + (lane >> 2)] = s;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(threads) : "memory");
    float t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int w = (lane & 3) + 4 * j;
      t[j] = w < warps ? words[w * 8 + (lane >> 2)] : 0.0f;
    }
    s = (t[0] + t[1]) + (t[2] + t[3]);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
  }
#pragma unroll
  for (int j = 0; j < kWanted; ++j) v[j] = __shfl_sync(0xffffffffu, s, 4 * j);
}

// ---- backward ----------------------------------------------------------------------
enum GradOperand { GRAD_DH, GRAD_DZ, GRAD_H, GRAD_H_SCALES, GRAD_Y, GRAD_Y_SCALES, GRAD_GATE, GRAD_OPS };
struct GradArgs {
  PipeArgs<GRAD_OPS> pipe;
  Rows dx, dy;
  Weights gate, w_post, w_pre;
  void* dgate;
  int64_t dgate_stride;
  int32_t per_gate;
  int32_t dgate_f32, accumulate, h_kept, y_kept;  // kept: 0 a matrix; 1 integers, 2 e4m3
  // sums over a CTA's rows: of dw_pre and dw_post [cta][hidden], of dgate [2 cta + (0: its first gate row)][hidden]
  float *part_pre, *part_post, *part_gate;
  float alpha, beta, eps;
  // lst_norm_split.cuh: rho and the factors of every row; a gate per token; one gate row or none (or one per token)
  float4* stats;
  int32_t token, single;
};

// What the six sums of a row (the top of norm_grad_kernel) give.
struct RowFactors {
  float rho, back, tau, back_y;
};
__device__ __forceinline__ RowFactors row_factors(const float (&s)[8], float inverse, float eps, float beta, bool has_z, bool has_post) {
  RowFactors f;
  f.rho = has_z ? rsqrtf(s[0] * inverse + eps) : 0.0f, f.back = f.rho * f.rho * (s[1] * inverse);
  f.tau = has_post ? rsqrtf(s[2] * inverse + eps) : 1.0f;
  // where a sum of squares has overflowed its norm's gradient is zero, and sum h q, which may have
  // overflowed with it, has no part in it
  const float of_h = f.back == 0.0f || f.tau == 0.0f ? 0.0f : f.back * s[5];
  f.back_y = has_post ? f.tau * f.tau * (beta * (s[3] + f.rho * (s[4] - of_h)) * inverse) : 0.0f;
  return f;
}

// One value of a parameter gradient.
__device__ __forceinline__ void store_sum(void* p, int64_t at, bool f32, bool accumulate, float v) {
  if (f32) {
    float* q = static_cast<float*>(p) + at;
    *q = accumulate ? *q + v : v;
  } else {
    __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + at;
    *q = __float2bfloat16_rn(accumulate ? __bfloat162float(*q) + v : v);
  }
}

// A unit of a row of parameter gradients that starts at element `at`.
template <bool VEC, int P>
__device__ __forceinline__ void store_sums(void* p, int64_t at, bool f32, bool accumulate, const Cols<VEC>& c, int k, const Part<P>& u, int i0 = 0) {
  if (VEC && !accumulate && (reinterpret_cast<uintptr_t>(p) + at * (f32 ? 4 : 2)) % 16 == 0) {
    if (f32)
      c.store(static_cast<float*>(p) + at, k, u, i0);
    else
      c.store(static_cast<__nv_bfloat16*>(p) + at, k, u, i0);
  } else {
    for_each(c, k, u, [&](uint32_t col, float v) { store_sum(p, at + col, f32, accumulate, v); }, i0);
  }
}

template <class Args>
using NormKernel = void (*)(const Args);
// The backward kernel for activations of a type (lst_norm_grad_bf16.cu, lst_norm_grad_f32.cu),
// 8 k columns a thread, and the word that its waits set when one runs out. `form`: 0 the general
// kernel, 1 + KEPT + 3 BLOCK that for whole units; `one`: its ONE.
NormKernel<GradArgs> norm_grad_bf16(bool vec, int k, int form, bool one);
NormKernel<GradArgs> norm_grad_f32(bool vec, int k, int form, bool one);
// The two for rows above 8192 columns (lst_norm_split.cuh): columns of a CTA of the second one,
// 8 a thread, and CTAs of an SM.
constexpr int kSplitTile = 1024;
constexpr int split_ctas(bool vec) { return vec ? 4 : 8; }
struct SplitKernels {
  NormKernel<GradArgs> stats, apply;
};
SplitKernels norm_split_bf16(bool vec);
SplitKernels norm_split_f32(bool vec);
cudaError_t norm_grad_bf16_take_error(int* out);
cudaError_t norm_grad_f32_take_error(int* out);

}  // namespace lst
