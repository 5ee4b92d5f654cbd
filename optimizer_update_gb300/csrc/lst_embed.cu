// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[i] = scale * table[t_i]. One read of the rows, one write; bound
// by memory bandwidth, and by launch latency for a few tokens.
//
// Gradient: grad[t] = scale * sum_{i : t_i = t} dout[i]. Adding rows with
// atomics would make the sum's order, and so its last bits, differ from run to
// run, and would read and write fp32 sums of a large gradient; instead
//   1. one cluster of 8 CTAs sorts (token, position) pairs, stable, by radix
//      passes in shared memory, and marks the tokens seen in a bit per token;
//   2. every 32 consecutive sorted positions and 1024 columns go to a CTA that
//      adds up runs of equal tokens in registers and writes the gradient of
//      every run that ends inside; the parts of runs that cross into another
//      CTA's positions go to the workspace. Other CTAs of the same launch
//      zero the rows of tokens that were not seen;
//   3. the crossing runs are added up, part by part in order.
// Each dout row is read once and each gradient row written once.
#include <cuda_bf16.h>

#include "lst_ops.h"

namespace lst {

namespace {

// ---- typed vectors of 8 elements ------------------------------------------------
// `left` elements are inside the row (8 or more on the vector path, which
// needs 16-byte aligned rows and a column count that is a multiple of 8).
template <bool VEC>
__device__ __forceinline__ void load8(const float* p, int left, float (&v)[8]) {
  if (VEC) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int left, float (&v)[8]) {
  if (VEC) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? __bfloat162float(p[i]) : 0.0f;
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* p, int left, const float (&v)[8]) {
  if (VEC) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4*>(p + 4), make_float4(v[4], v[5], v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = v[i];
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int left, const float (&v)[8]) {
  if (VEC) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = __float2bfloat16_rn(v[i]);
  }
}

__device__ __forceinline__ int64_t token_at(const void* t, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(t)[i] : static_cast<const int32_t*>(t)[i];
}

// ---- lookup -----------------------------------------------------------------------
template <class TI, class TO, bool VEC>
__global__ void __launch_bounds__(256)
    embed_kernel(const TI* __restrict__ table, int64_t table_ld, const void* __restrict__ tokens, int wide,
                 TO* __restrict__ out, int64_t out_ld, int hidden, int64_t vocab, uint32_t units_per_row,
                 uint32_t rows_per_launch, int64_t row_base, float scale) {
  let_next_start();
  wait_for_previous();
  const uint64_t unit = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x;
  const uint32_t r = static_cast<uint32_t>(unit / units_per_row);
  if (r >= rows_per_launch) return;
  const int col = static_cast<int>(unit - static_cast<uint64_t>(r) * units_per_row) * 8;
  const int64_t row = row_base + r;
  const int64_t t = token_at(tokens, wide, row);
  float v[8];
  if (t >= 0 && t < vocab) {
    load8<VEC>(table + t * table_ld + col, hidden - col, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], scale);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __int_as_float(0x7fc00000);
  }
  store8<VEC>(out + row * out_ld + col, hidden - col, v);
}

// ---- stable sort of (token, position) ---------------------------------------------
constexpr int kSortCtas = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote_u32(const uint32_t* p, uint32_t rank) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), v;
  asm volatile("{\n\t.reg .u32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\tld.shared::cluster.u32 %0, [r];\n\t}"
               : "=r"(v)
               : "r"(a), "r"(rank)
               : "memory");
  return v;
}

// Least-significant-digit radix sort. Every warp of the cluster owns one range
// of positions, so that (warp, order within the warp) is the input order and
// each pass is stable: count digits per warp, place the warps' counts one after
// the other (over the cluster by distributed shared memory), scatter. Tokens
// outside the vocabulary get the key `vocab` and sort last.
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1)
    sort_kernel(const void* __restrict__ tokens, int wide, int n, int vocab, int passes, int digit_bits, uint2* buf0,
                uint2* buf1, uint32_t* seen) {
  let_next_start();
  wait_for_previous();
  extern __shared__ uint32_t sm[];
  const int bins = 1 << digit_bits;
  uint32_t* const count = sm;                        // [warp][bin]
  uint32_t* const total = sm + kSortWarps * bins;    // [bin], this CTA
  uint32_t* const start = total + bins;              // [bin], first place of this CTA's digit
  __shared__ uint32_t warp_sum[kSortWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t cta = blockIdx.x;
  const uint32_t below = (1u << lane) - 1;
  const int per_warp = ((n + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) + 31) & ~31;
  const int64_t first = static_cast<int64_t>(cta * kSortWarps + warp) * per_warp;
  const int64_t last = first + per_warp < n ? first + per_warp : n;

  for (int64_t i = static_cast<int64_t>(cta) * kSortThreads + tid; i < (static_cast<int64_t>(vocab) + 31) / 32;
       i += kSortCtas * kSortThreads)
    seen[i] = 0;
  cluster_barrier();

  for (int pass = 0; pass < passes; ++pass) {
    const uint2* const src = (pass & 1) ? buf0 : buf1;  // unused in pass 0
    uint2* const dst = (pass & 1) ? buf1 : buf0;
    const int shift = pass * digit_bits;
    for (int i = tid; i < kSortWarps * bins; i += kSortThreads) count[i] = 0;
    __syncthreads();
    uint32_t* const mine = count + warp * bins;
    for (int64_t i0 = first; i0 < last; i0 += 32) {
      const bool in = i0 + lane < last;
      uint32_t digit = bins;
      if (in) {
        uint32_t key;
        if (pass == 0) {
          const int64_t t = token_at(tokens, wide, i0 + lane);
          const bool valid = t >= 0 && t < vocab;
          key = valid ? static_cast<uint32_t>(t) : static_cast<uint32_t>(vocab);
          if (valid) atomicOr(seen + (key >> 5), 1u << (key & 31));
        } else {
          key = src[i0 + lane].x;
        }
        digit = (key >> shift) & (bins - 1);
      }
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in && (same & below) == 0) mine[digit] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    for (int d = tid; d < bins; d += kSortThreads) {
      uint32_t sum = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = count[w * bins + d];
        count[w * bins + d] = sum;
        sum += c;
      }
      total[d] = sum;
    }
    cluster_barrier();
    // bins <= kSortThreads: one digit per thread
    uint32_t all = 0, lower = 0;
    if (tid < bins) {
      for (uint32_t c = 0; c < kSortCtas; ++c) {
        const uint32_t x = remote_u32(total + tid, c);
        all += x;
        lower += c < cta ? x : 0;
      }
    }
    uint32_t scan = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += x;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    if (tid < bins) start[tid] = before + scan - all + lower;
    __syncthreads();
    for (int64_t i0 = first; i0 < last; i0 += 32) {
      const bool in = i0 + lane < last;
      uint32_t digit = bins;
      uint2 item = make_uint2(0, 0);
      if (in) {
        if (pass == 0) {
          const int64_t t = token_at(tokens, wide, i0 + lane);
          item = make_uint2(t >= 0 && t < vocab ? static_cast<uint32_t>(t) : static_cast<uint32_t>(vocab),
                            static_cast<uint32_t>(i0 + lane));
        } else {
          item = src[i0 + lane];
        }
        digit = (item.x >> shift) & (bins - 1);
      }
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in) dst[start[digit] + mine[digit] + __popc(same & below)] = item;
      __syncwarp();
      if (in && (same & below) == 0) mine[digit] += __popc(same);
      __syncwarp();
    }
    cluster_barrier();  // items placed; totals read by all
  }
}

// ---- runs of equal tokens -----------------------------------------------------------
constexpr int kRun = 32;             // sorted positions of a CTA
constexpr int kSumThreads = 128;     // x 8 columns
constexpr int kSumCols = kSumThreads * 8;
constexpr int kZeroRows = 16;

template <class TG>
struct Grad {
  TG* data;
  int64_t ld;
  float scale;
  int accumulate;
};

template <class TG, bool VEC>
__device__ __forceinline__ void write_row(const Grad<TG>& g, int64_t row, int col, int left, float (&acc)[8]) {
  TG* p = g.data + row * g.ld + col;
  float v[8];
  if (g.accumulate) {
    load8<VEC>(p, left, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(acc[i], g.scale, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(acc[i], g.scale);
  }
  store8<VEC>(p, left, v);
}

template <class TD, class TG, bool VEC>
__global__ void __launch_bounds__(kSumThreads)
    sum_kernel(const TD* __restrict__ dout, int64_t dout_ld, const uint2* __restrict__ sorted, int n, int vocab,
               int hidden, int slices, int sum_blocks, const uint32_t* __restrict__ seen, float* __restrict__ parts,
               int64_t parts_ld, Grad<TG> g) {
  let_next_start();
  wait_for_previous();
  if (static_cast<int>(blockIdx.x) >= sum_blocks) {
    const int64_t r0 = static_cast<int64_t>(blockIdx.x - sum_blocks) * kZeroRows;
    float zero[8] = {};
    for (int64_t r = r0; r < r0 + kZeroRows && r < vocab; ++r) {
      if ((seen[r >> 5] >> (r & 31)) & 1) continue;
      for (int col = threadIdx.x * 8; col < hidden; col += kSumCols) store8<VEC>(g.data + r * g.ld + col, hidden - col, zero);
    }
    return;
  }
  const int chunk = blockIdx.x / slices;
  const int col = (blockIdx.x - chunk * slices) * kSumCols + threadIdx.x * 8;
  __shared__ uint32_t key[kRun + 2], pos[kRun];
  const int64_t e0 = static_cast<int64_t>(chunk) * kRun;
  const int len = n - e0 < kRun ? static_cast<int>(n - e0) : kRun;
  constexpr uint32_t kNone = 0xffffffffu;
  if (threadIdx.x < kRun + 2) {
    const int64_t e = e0 + threadIdx.x - 1;
    const uint2 it = e >= 0 && e < n ? sorted[e] : make_uint2(kNone, 0);
    key[threadIdx.x] = it.x;
    if (threadIdx.x >= 1 && threadIdx.x <= kRun) pos[threadIdx.x - 1] = it.y;
  }
  __syncthreads();
  if (col >= hidden) return;
  const int left = hidden - col;
  float acc[8] = {};
  bool head = key[0] == key[1];
  constexpr int kBatch = 4;  // rows in flight per thread
  for (int j0 = 0; j0 < len; j0 += kBatch) {
    float v[kBatch][8];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (j0 + j < len) load8<VEC>(dout + static_cast<int64_t>(pos[j0 + j]) * dout_ld + col, left, v[j]);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int e = j0 + j;
      if (e >= len) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], v[j][i]);
      const uint32_t k = key[e + 1];
      const bool more = key[e + 2] == k;       // the run goes on
      if (more && e + 1 < len) continue;
      if (k < static_cast<uint32_t>(vocab)) {
        if (head || more) {
          float* p = parts + (static_cast<int64_t>(chunk) * 2 + (head ? 0 : 1)) * parts_ld + col;
          *reinterpret_cast<float4*>(p) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          *reinterpret_cast<float4*>(p + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        } else {
          write_row<TG, VEC>(g, k, col, left, acc);
        }
      }
      head = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    }
  }
}

// A run that leaves the CTA it began in: its first part, then the parts of the
// following CTAs in order.
template <class TG, bool VEC>
__global__ void __launch_bounds__(kSumThreads)
    join_kernel(const uint2* __restrict__ sorted, int n, int vocab, int hidden, int slices,
                const float* __restrict__ parts, int64_t parts_ld, Grad<TG> g) {
  let_next_start();
  wait_for_previous();
  const int chunk = blockIdx.x / slices;
  const int64_t e0 = static_cast<int64_t>(chunk) * kRun, e1 = e0 + kRun;
  if (e1 >= n) return;
  const uint32_t k = sorted[e1 - 1].x;
  if (k >= static_cast<uint32_t>(vocab) || sorted[e1].x != k) return;
  if (e0 > 0 && sorted[e0 - 1].x == k) return;  // began earlier (sorted: the whole chunk is this run)
  const int col = (blockIdx.x - chunk * slices) * kSumCols + threadIdx.x * 8;
  if (col >= hidden) return;
  float acc[8];
  load8<true>(parts + (static_cast<int64_t>(chunk) * 2 + 1) * parts_ld + col, 8, acc);
  for (int64_t c = chunk + 1;; ++c) {
    float v[8];
    load8<true>(parts + c * 2 * parts_ld + col, 8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], v[i]);
    const int64_t next = (c + 1) * kRun;
    if (next >= n || sorted[next].x != k) break;
  }
  write_row<TG, VEC>(g, k, col, hidden - col, acc);
}

bool vec_rows(const lst_matrix* m) {
  const int e = dtype_bytes(m->dtype);
  return m->cols % 8 == 0 && (m->stride * e) % 16 == 0 && reinterpret_cast<uintptr_t>(m->data) % 16 == 0;
}

template <class TI, class TO>
cudaError_t launch_embed(const lst_matrix* table, const lst_indices* tokens, const lst_matrix* out, float scale,
                         cudaStream_t stream) {
  const bool vec = vec_rows(table) && vec_rows(out);
  const int64_t units = ops_ceil_div(out->cols, 8);
  const int64_t rows_max = ((int64_t(1) << 31) - 1) / units * 128;
  for (int64_t r0 = 0; r0 < out->rows; r0 += rows_max) {
    const int64_t rows = out->rows - r0 < rows_max ? out->rows - r0 : rows_max;
    const unsigned grid = static_cast<unsigned>(ops_ceil_div(rows * units, 256));
    auto k = vec ? embed_kernel<TI, TO, true> : embed_kernel<TI, TO, false>;
    const cudaError_t err = launch_chained(k, dim3(grid), dim3(256), 0, stream, static_cast<const TI*>(table->data), table->stride, tokens->data, tokens->bits == 64,
                                static_cast<TO*>(out->data), out->stride, static_cast<int>(out->cols), table->rows,
                                static_cast<uint32_t>(units), static_cast<uint32_t>(rows), r0, scale);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

struct GradPlan {
  int passes, digit_bits;
  int64_t chunks, parts_ld;
  int64_t buf_off[2], seen_off, parts_off, bytes;
};

GradPlan grad_plan(int64_t n, int64_t hidden, int64_t vocab) {
  GradPlan p;
  int bits = 1;
  while ((int64_t(1) << bits) <= vocab) ++bits;  // keys 0..vocab
  p.passes = bits <= 10 ? 1 : bits <= 20 ? 2 : 3;
  p.digit_bits = static_cast<int>(ops_ceil_div(bits, p.passes));
  p.chunks = ops_ceil_div(n, kRun);
  p.parts_ld = ops_round_up(hidden, 8);
  int64_t at = 0;
  for (int i = 0; i < 2; ++i) {
    p.buf_off[i] = at;
    at += ops_round_up(n * 8, 256);
  }
  p.seen_off = at;
  at += ops_round_up((vocab + 31) / 32 * 4, 256);
  p.parts_off = at;
  at += ops_round_up(p.chunks * 2 * p.parts_ld * 4, 256);
  p.bytes = at;
  return p;
}

template <class TD, class TG>
cudaError_t launch_grad(const lst_matrix* dout, const lst_matrix* grad, const GradPlan& p, float scale, int accumulate,
                        char* ws, cudaStream_t stream) {
  const bool vec = vec_rows(dout) && vec_rows(grad);
  const int n = static_cast<int>(dout->rows), hidden = static_cast<int>(dout->cols);
  const int vocab = static_cast<int>(grad->rows);
  const uint2* sorted = reinterpret_cast<const uint2*>(ws + p.buf_off[(p.passes - 1) & 1]);
  const uint32_t* seen = reinterpret_cast<const uint32_t*>(ws + p.seen_off);
  float* parts = reinterpret_cast<float*>(ws + p.parts_off);
  const int64_t slices = ops_ceil_div(hidden, kSumCols);
  const int64_t sum_blocks = p.chunks * slices;
  const int64_t zero_blocks = accumulate ? 0 : ops_ceil_div(vocab, kZeroRows);
  if (sum_blocks + zero_blocks > INT32_MAX) return cudaErrorInvalidValue;
  const Grad<TG> g = {static_cast<TG*>(grad->data), grad->stride, scale, accumulate};
  if (sum_blocks + zero_blocks > 0) {
    auto k = vec ? sum_kernel<TD, TG, true> : sum_kernel<TD, TG, false>;
    const cudaError_t err = launch_chained(k, dim3(static_cast<unsigned>(sum_blocks + zero_blocks)), dim3(kSumThreads), 0, stream, 
        static_cast<const TD*>(dout->data), dout->stride, sorted, n, vocab, hidden, static_cast<int>(slices),
        static_cast<int>(sum_blocks), seen, parts, p.parts_ld, g);
    if (err != cudaSuccess) return err;
  }
  if (p.chunks > 1) {
    auto k = vec ? join_kernel<TG, true> : join_kernel<TG, false>;
    return launch_chained(k, dim3(static_cast<unsigned>(sum_blocks)), dim3(kSumThreads), 0, stream, sorted, n, vocab, hidden, static_cast<int>(slices),
                                                                     parts, p.parts_ld, g);
  }
  return cudaSuccess;
}

}  // namespace
}  // namespace lst

using namespace lst;

extern "C" lst_status lst_embed(const lst_matrix* table, const lst_indices* tokens, const lst_matrix* out, float scale,
                                void* cuda_stream) {
  clear_error();
  const char* who = "lst_embed";
  LST_TRY(check_matrix(table, "table", who));
  LST_TRY(check_indices(tokens, "tokens", who));
  LST_TRY(check_matrix(out, "out", who));
  if (out->rows != tokens->count || out->cols != table->cols)
    return fail(LST_ERR_INVALID_ARG, "%s: out must be tokens x hidden", who);
  if (out->rows == 0 || out->cols == 0) return LST_OK;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const int kind = (table->dtype == LST_F32 ? 2 : 0) + (out->dtype == LST_F32 ? 1 : 0);
  cudaError_t err;
  switch (kind) {
    case 0: err = launch_embed<__nv_bfloat16, __nv_bfloat16>(table, tokens, out, scale, s); break;
    case 1: err = launch_embed<__nv_bfloat16, float>(table, tokens, out, scale, s); break;
    case 2: err = launch_embed<float, __nv_bfloat16>(table, tokens, out, scale, s); break;
    default: err = launch_embed<float, float>(table, tokens, out, scale, s); break;
  }
  if (err != cudaSuccess) return cuda_fail(err, who);
  return LST_OK;
}

extern "C" int64_t lst_embed_grad_workspace_bytes(int64_t count, int64_t hidden, int64_t vocab) {
  if (count < 0 || hidden < 0 || vocab < 0 || count > (int64_t(1) << 30) || vocab > (int64_t(1) << 30)) return 0;
  return grad_plan(count, hidden, vocab).bytes;
}

extern "C" lst_status lst_embed_grad(const lst_matrix* dout, const lst_indices* tokens, const lst_matrix* grad,
                                     float scale, int32_t accumulate, void* workspace, int64_t workspace_bytes,
                                     void* cuda_stream) {
  clear_error();
  const char* who = "lst_embed_grad";
  LST_TRY(check_matrix(dout, "dout", who));
  LST_TRY(check_indices(tokens, "tokens", who));
  LST_TRY(check_matrix(grad, "grad", who));
  if (dout->rows != tokens->count || dout->cols != grad->cols)
    return fail(LST_ERR_INVALID_ARG, "%s: dout must be tokens x hidden", who);
  if (grad->rows > (int64_t(1) << 30)) return fail(LST_ERR_INVALID_ARG, "%s: vocabulary above 2^30", who);
  if (grad->rows == 0 || grad->cols == 0) return LST_OK;
  const GradPlan p = grad_plan(dout->rows, dout->cols, grad->rows);
  LST_TRY(check_workspace(workspace, workspace_bytes, p.bytes, who));
  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  const int bins = 1 << p.digit_bits;
  const int smem = (kSortWarps + 2) * bins * 4;
  // the largest case (10-bit digits) needs 139,264 bytes; a function attribute
  // is per device, so it is set on every call (host only, under a microsecond)
  LST_TRY_CUDA(cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem), who);
  LST_TRY_CUDA(launch_chained(sort_kernel, dim3(kSortCtas), dim3(kSortThreads), smem, s, tokens->data, tokens->bits == 64, static_cast<int>(dout->rows),
                                                    static_cast<int>(grad->rows), p.passes, p.digit_bits,
                                                    reinterpret_cast<uint2*>(ws + p.buf_off[0]),
                                                    reinterpret_cast<uint2*>(ws + p.buf_off[1]),
                                                    reinterpret_cast<uint32_t*>(ws + p.seen_off)), who);
  const int kind = (dout->dtype == LST_F32 ? 2 : 0) + (grad->dtype == LST_F32 ? 1 : 0);
  cudaError_t err;
  switch (kind) {
    case 0: err = launch_grad<__nv_bfloat16, __nv_bfloat16>(dout, grad, p, scale, accumulate != 0, ws, s); break;
    case 1: err = launch_grad<__nv_bfloat16, float>(dout, grad, p, scale, accumulate != 0, ws, s); break;
    case 2: err = launch_grad<float, __nv_bfloat16>(dout, grad, p, scale, accumulate != 0, ws, s); break;
    default: err = launch_grad<float, float>(dout, grad, p, scale, accumulate != 0, ws, s); break;
  }
  if (err != cudaSuccess) return cuda_fail(err, who);
  return LST_OK;
}
