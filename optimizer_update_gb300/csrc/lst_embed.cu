// Embedding lookup with scaling, and its gradient by sorted tokens.
//
// Lookup: out[i] = scale * table[t_i]. One read of the rows, one write; bound
// by memory bandwidth, and by launch latency for a few tokens.
//
// Gradient: grad[t] = scale * sum_{i : t_i = t} dout[i]. Adding rows with
// atomics would make the sum's order, and so its last bits, differ from run to
// run, and would read and write fp32 sums of a large gradient; instead
//   1. one cluster of 8 or 16 CTAs sorts (token, position) pairs, stable, by radix
//      passes in shared memory, while the launch's other CTAs zero the gradient
//      (the rows that step 2 writes too, which costs less than waiting for the
//      sort to know them);
//   2. every 32 (or 8) consecutive sorted positions and 1024 columns go to a CTA that
//      adds up runs of equal tokens in registers and writes the gradient of
//      every run that ends inside; the parts of runs that cross into another
//      CTA's positions go to the workspace;
//   3. the crossing runs are added up, part by part in order.
// Each dout row is read once.
#include <cuda_bf16.h>

#include <algorithm>

#include "lst_ops.h"

namespace lst {

namespace {

// ---- 8 elements of a row per thread ------------------------------------------------
// A group of THREADS threads covers 8 THREADS columns. On the vector path (rows on
// 16 bytes, a column count that is a multiple of 8) a thread has 8 consecutive
// ones, otherwise every THREADS-th, so that a warp's accesses stay consecutive.
// `p` is the row at the group's first column, `left` the columns from there on.
template <bool VEC, int THREADS>
__device__ __forceinline__ void load8(const float* p, int thread, int left, float (&v)[8]) {
  if (VEC) {
    const float4* q = reinterpret_cast<const float4*>(p) + 2 * thread;
    if (thread * 8 < left) {
      const float4 a = q[0], b = q[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (thread + i * THREADS < left) v[i] = p[thread + i * THREADS];
  }
}
template <bool VEC, int THREADS>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int thread, int left, float (&v)[8]) {
  if (VEC) {
    if (thread * 8 < left) {
      const uint4 a = reinterpret_cast<const uint4*>(p)[thread];
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (thread + i * THREADS < left) v[i] = __bfloat162float(p[thread + i * THREADS]);
  }
}
template <bool VEC, int THREADS>
__device__ __forceinline__ void store8(float* p, int thread, int left, const float (&v)[8]) {
  if (VEC) {
    float4* q = reinterpret_cast<float4*>(p) + 2 * thread;
    if (thread * 8 < left) {
      __stcs(q, make_float4(v[0], v[1], v[2], v[3]));
      __stcs(q + 1, make_float4(v[4], v[5], v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (thread + i * THREADS < left) p[thread + i * THREADS] = v[i];
  }
}
template <bool VEC, int THREADS>
__device__ __forceinline__ void store8(__nv_bfloat16* p, int thread, int left, const float (&v)[8]) {
  if (VEC) {
    if (thread * 8 < left) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      __stcs(reinterpret_cast<uint4*>(p) + thread, make_uint4(w[0], w[1], w[2], w[3]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (thread + i * THREADS < left) p[thread + i * THREADS] = __float2bfloat16_rn(v[i]);
  }
}

__device__ __forceinline__ int64_t token_at(const void* t, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(t)[i] : static_cast<const int32_t*>(t)[i];
}

// ---- lookup -----------------------------------------------------------------------
// A warp takes 256 columns of a row at a time, and two such pieces at once; the
// CTAs of a launch walk the output from start to end. (A persistent grid whose
// warps took pieces a grid apart wrote all over the output at once: 281 us for
// 65536 x 4096 bf16, against 144. Four pieces at once: 198.)
constexpr int kPieces = 2;

template <class TI, class TO, bool VEC>
__global__ void __launch_bounds__(256)
    embed_kernel(const TI* __restrict__ table, int64_t table_ld, const void* __restrict__ tokens, int wide,
                 TO* __restrict__ out, int64_t out_ld, int hidden, int64_t vocab, uint32_t pieces_per_row, int64_t pieces,
                 float scale) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * 8 * kPieces + (threadIdx.x >> 5);
  float v[kPieces][8];
  int64_t row[kPieces];
  int col[kPieces];
  bool inside[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const int64_t p = p0 + k * 8;
    inside[k] = false;
    if (p < pieces) {
      // 32-bit division where it suffices
      row[k] = p <= 0xffffffffll ? static_cast<int64_t>(static_cast<uint32_t>(p) / pieces_per_row) : p / pieces_per_row;
      col[k] = static_cast<int>(p - row[k] * pieces_per_row) * 256;
      const int64_t t = token_at(tokens, wide, row[k]);
      inside[k] = t >= 0 && t < vocab;
      if (inside[k]) load8<VEC, 32>(table + t * table_ld + col[k], lane, hidden - col[k], v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    if (p0 + k * 8 >= pieces) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = inside[k] ? __fmul_rn(v[k][i], scale) : __int_as_float(0x7fc00000);
    store8<VEC, 32>(out + row[k] * out_ld + col[k], lane, hidden - col[k], v[k]);
  }
}

// ---- stable sort of (token, position) ---------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortAhead = 8;  // loads in flight per thread
constexpr int kSortMaxBits = 10;  // of a digit: one bin per thread
constexpr int sort_smem(int digit_bits) { return (kSortWarps + 2) * (1 << digit_bits) * 4; }

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
template <int kSortCtas>
__global__ void __cluster_dims__(kSortCtas, 1, 1) __launch_bounds__(kSortThreads, 1)
    sort_kernel(const void* __restrict__ tokens, int wide, int n, int vocab, int passes, int digit_bits, uint2* buf0,
                uint2* buf1, char* zero, int64_t zero_pitch, int64_t zero_row, int zero_vec) {
  let_next_start();
  wait_for_previous();
  if (blockIdx.x >= kSortCtas) {
    const int64_t first = static_cast<int64_t>(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x;
    const int64_t step = static_cast<int64_t>(gridDim.x - kSortCtas) * kSortThreads;
    if (zero_vec) {  // one range of whole 16-byte words
#pragma unroll 8
      for (int64_t i = first; i < zero_row / 16; i += step) reinterpret_cast<uint4*>(zero)[i] = make_uint4(0, 0, 0, 0);
    } else {  // rows of 2-byte units, a warp at a time
      const int lane = threadIdx.x & 31;
      for (int64_t r = first >> 5; r < vocab; r += step >> 5)
        for (int64_t c = lane; c < zero_row / 2; c += 32) reinterpret_cast<uint16_t*>(zero + r * zero_pitch)[c] = 0;
    }
    return;
  }
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

  for (int pass = 0; pass < passes; ++pass) {
    const uint2* const src = (pass & 1) ? buf0 : buf1;  // unused in pass 0
    uint2* const dst = (pass & 1) ? buf1 : buf0;
    const int shift = pass * digit_bits;
    for (int i = tid; i < kSortWarps * bins; i += kSortThreads) count[i] = 0;
    __syncthreads();
    uint32_t* const mine = count + warp * bins;
    auto item_at = [&](int64_t i) {
      if (pass > 0) return src[i];
      const int64_t t = token_at(tokens, wide, i);
      return make_uint2(t >= 0 && t < vocab ? static_cast<uint32_t>(t) : static_cast<uint32_t>(vocab),
                        static_cast<uint32_t>(i));
    };
    for (int64_t i0 = first; i0 < last; i0 += 32 * kSortAhead) {
      uint32_t key[kSortAhead];
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j)
        if (i0 + 32 * j + lane < last) key[j] = item_at(i0 + 32 * j + lane).x;
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j) {
        if (i0 + 32 * j >= last) break;
        const bool in = i0 + 32 * j + lane < last;
        const uint32_t digit = in ? (key[j] >> shift) & (bins - 1) : bins;
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        if (in && (same & below) == 0) mine[digit] += __popc(same);
        __syncwarp();
      }
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
    for (int64_t i0 = first; i0 < last; i0 += 32 * kSortAhead) {
      uint2 item[kSortAhead];
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j)
        if (i0 + 32 * j + lane < last) item[j] = item_at(i0 + 32 * j + lane);
#pragma unroll
      for (int j = 0; j < kSortAhead; ++j) {
        if (i0 + 32 * j >= last) break;
        const bool in = i0 + 32 * j + lane < last;
        const uint32_t digit = in ? (item[j].x >> shift) & (bins - 1) : bins;
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        if (in) dst[start[digit] + mine[digit] + __popc(same & below)] = item[j];
        __syncwarp();
        if (in && (same & below) == 0) mine[digit] += __popc(same);
        __syncwarp();
      }
    }
    cluster_barrier();  // items placed; totals read by all
  }
}

// ---- runs of equal tokens -----------------------------------------------------------
constexpr int kMaxRun = 32;          // sorted positions of a CTA, at most
constexpr int kSumThreads = 128;     // x 8 columns
constexpr int kSumCols = kSumThreads * 8;

template <class TG>
struct Grad {
  TG* data;
  int64_t ld;
  float scale;
  int accumulate;
};

// Row `row` from column `col` on: the thread's 8 sums, scaled.
template <class TG, bool VEC>
__device__ __forceinline__ void write_row(const Grad<TG>& g, int64_t row, int col, int left, const float (&acc)[8]) {
  TG* p = g.data + row * g.ld + col;
  float v[8] = {};
  if (g.accumulate) {
    load8<VEC, kSumThreads>(p, threadIdx.x, left, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(acc[i], g.scale, v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(acc[i], g.scale);
  }
  store8<VEC, kSumThreads>(p, threadIdx.x, left, v);
}

template <class TD, class TG, bool VEC>
__global__ void __launch_bounds__(kSumThreads)
    sum_kernel(const TD* __restrict__ dout, int64_t dout_ld, const uint2* __restrict__ sorted, int n, int vocab,
               int hidden, int slices, int run, float* __restrict__ parts, int64_t parts_ld, Grad<TG> g) {
  let_next_start();
  wait_for_previous();
  const int chunk = blockIdx.x / slices;
  const int col = (blockIdx.x - chunk * slices) * kSumCols, left = hidden - col;
  __shared__ uint32_t key[kMaxRun + 2], pos[kMaxRun];
  const int64_t e0 = static_cast<int64_t>(chunk) * run;
  const int len = n - e0 < run ? static_cast<int>(n - e0) : run;
  constexpr uint32_t kNone = 0xffffffffu;
  if (static_cast<int>(threadIdx.x) < run + 2) {
    const int64_t e = e0 + threadIdx.x - 1;
    const uint2 it = e >= 0 && e < n ? sorted[e] : make_uint2(kNone, 0);
    key[threadIdx.x] = it.x;
    if (threadIdx.x >= 1 && static_cast<int>(threadIdx.x) <= run) pos[threadIdx.x - 1] = it.y;
  }
  __syncthreads();
  float acc[8] = {};
  bool head = key[0] == key[1];
  // Rows in flight per thread. More cost registers, and so resident CTAs. 65521 rows,
  // added to 32000: 4096 bf16 in vectors 186 us by two, 196 by one, 206 by four, 255 by
  // eight; 4096 fp32 in vectors 275 by four, 276 by two, 280 by one; 4095 without
  // vectors, bf16 (written) 219 by one, 269 by two, 317 by four, fp32 308, 311, 316.
  constexpr int kBatch = !VEC ? 1 : sizeof(TD) == 2 ? 2 : 4;
  for (int j0 = 0; j0 < len; j0 += kBatch) {
    float v[kBatch][8] = {};
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (j0 + j < len)
        load8<VEC, kSumThreads>(dout + static_cast<int64_t>(pos[j0 + j]) * dout_ld + col, threadIdx.x, left, v[j]);
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
          store8<VEC, kSumThreads>(p, threadIdx.x, left, acc);
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
// following CTAs in order. Bound by latency where one token is frequent: all parts of
// its run are one CTA's per 1024 columns (65521 tokens of 4096 bf16 columns, added:
// 217 us uniform, 598 with one token on half of them, 879 with one on all).
template <class TG, bool VEC>
__global__ void __launch_bounds__(kSumThreads)
    join_kernel(const uint2* __restrict__ sorted, int n, int vocab, int hidden, int slices, int run, int chunks,
                const float* __restrict__ parts, int64_t parts_ld, Grad<TG> g) {
  let_next_start();
  wait_for_previous();
  const int chunk = blockIdx.x / slices;
  const int64_t e0 = static_cast<int64_t>(chunk) * run, e1 = e0 + run;
  if (e1 >= n) return;
  const uint32_t k = sorted[e1 - 1].x, after = sorted[e1].x, before = e0 > 0 ? sorted[e0 - 1].x : 0xffffffffu;
  // no run that crosses here, or one that began earlier (sorted: all of this CTA's positions are it)
  if (k >= static_cast<uint32_t>(vocab) || after != k || before == k) return;
  const int col = (blockIdx.x - chunk * slices) * kSumCols, left = hidden - col;
  float acc[8] = {};
  load8<VEC, kSumThreads>(parts + (static_cast<int64_t>(chunk) * 2 + 1) * parts_ld + col, threadIdx.x, left, acc);
  constexpr int kBatch = 4;  // parts in flight; those past the run's end are not used
  for (int64_t c0 = chunk + 1;; c0 += kBatch) {
    float v[kBatch][8] = {};
    bool part[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      part[j] = c0 + j < chunks && sorted[(c0 + j) * run].x == k;
      if (c0 + j < chunks) load8<VEC, kSumThreads>(parts + (c0 + j) * 2 * parts_ld + col, threadIdx.x, left, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (part[j]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], v[j][i]);
      }
    if (!part[kBatch - 1]) break;
  }
  write_row<TG, VEC>(g, k, col, left, acc);
}

bool vec_rows(const lst_matrix* m) {
  const int e = dtype_bytes(m->dtype);
  return m->cols % 8 == 0 && (m->stride * e) % 16 == 0 && reinterpret_cast<uintptr_t>(m->data) % 16 == 0;
}

template <class TI, class TO>
cudaError_t launch_embed(const lst_matrix* table, const lst_indices* tokens, const lst_matrix* out, float scale,
                         cudaStream_t stream) {
  const bool vec = vec_rows(table) && vec_rows(out);
  const int64_t per_row = ops_ceil_div(out->cols, 256), pieces = out->rows * per_row;
  const int64_t per_block = 8 * kPieces;
  // 2^30 rows of 2^23 pieces at most; a launch covers what its grid can count
  const int64_t most = (int64_t(1) << 30) / per_row * per_row;
  const int64_t at_once = std::max<int64_t>(per_row, std::min(pieces, most * per_block));
  const int64_t rows_at_once = at_once / per_row;
  for (int64_t r = 0; r < out->rows; r += rows_at_once) {
    const int64_t rows = std::min(rows_at_once, out->rows - r), now = rows * per_row;
    const cudaError_t err = launch_chained(
        vec ? embed_kernel<TI, TO, true> : embed_kernel<TI, TO, false>,
        dim3(static_cast<unsigned>(ops_ceil_div(now, per_block))), dim3(256), 0, stream,
        static_cast<const TI*>(table->data), table->stride,
        static_cast<const char*>(tokens->data) + r * (tokens->bits / 8), tokens->bits == 64,
        static_cast<TO*>(out->data) + r * out->stride, out->stride, static_cast<int>(out->cols), table->rows,
        static_cast<uint32_t>(per_row), now, scale);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// The sort takes 16 CTAs instead of 8 where it is the longer part of its launch: from
// 16384 tokens on (whole gradients of 65521 tokens, 256 columns, added: 72 us against
// 85; of 16384 29.8 and 31.4; of 4096 22 and 21), unless more is to be zeroed than it
// leaves time for (65521 tokens, 32000 rows of 2 KB: 119 and 132 us; of 8 KB: 231 and
// 226, since fewer CTAs in clusters of 16 are resident).
bool wide_sort(int64_t n, int64_t zeroed_bytes) { return n >= 16384 && zeroed_bytes <= 2000 * n; }

struct GradPlan {
  int passes, digit_bits, run;
  int64_t chunks, parts_ld;
  int64_t buf_off[2], parts_off, bytes;
};

// 32 positions to a CTA, or 8 where that leaves the GPU short of CTAs: a short
// call's time is the latency of a CTA's rows one batch after the other.
constexpr int64_t kManyCtas = 152 * 16;

GradPlan grad_plan(int64_t n, int64_t hidden, int64_t vocab) {
  GradPlan p;
  int bits = 1;
  while ((int64_t(1) << bits) <= vocab) ++bits;  // keys 0..vocab
  p.passes = static_cast<int>(ops_ceil_div(bits, kSortMaxBits));  // 4 for 2^30 entries, 31 bits
  p.digit_bits = static_cast<int>(ops_ceil_div(bits, p.passes));
  p.run = ops_ceil_div(n, kMaxRun) * ops_ceil_div(hidden, kSumCols) >= kManyCtas ? kMaxRun : 8;
  p.chunks = ops_ceil_div(n, p.run);
  p.parts_ld = ops_round_up(hidden, 8);
  int64_t at = 0;
  for (int i = 0; i < 2; ++i) {
    p.buf_off[i] = at;
    at += ops_round_up(n * 8, 256);
  }
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
  float* parts = reinterpret_cast<float*>(ws + p.parts_off);
  const int64_t slices = ops_ceil_div(hidden, kSumCols);
  const int64_t sum_blocks = p.chunks * slices;
  if (sum_blocks == 0) return cudaSuccess;
  if (sum_blocks > INT32_MAX) return cudaErrorInvalidValue;
  const Grad<TG> g = {static_cast<TG*>(grad->data), grad->stride, scale, accumulate};
  const cudaError_t err = launch_chained(
      vec ? sum_kernel<TD, TG, true> : sum_kernel<TD, TG, false>, dim3(static_cast<unsigned>(sum_blocks)),
      dim3(kSumThreads), 0, stream, static_cast<const TD*>(dout->data), dout->stride, sorted, n, vocab, hidden,
      static_cast<int>(slices), p.run, parts, p.parts_ld, g);
  if (err != cudaSuccess || p.chunks == 1) return err;
  return launch_chained(vec ? join_kernel<TG, true> : join_kernel<TG, false>, dim3(static_cast<unsigned>(sum_blocks)),
                        dim3(kSumThreads), 0, stream, sorted, n, vocab, hidden, static_cast<int>(slices), p.run,
                        static_cast<int>(p.chunks), parts, p.parts_ld, g);
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
  if (count < 0 || hidden < 0 || vocab < 0 || count > (int64_t(1) << 30) || vocab > (int64_t(1) << 30) || hidden > INT32_MAX)
    return 0;
  const GradPlan p = grad_plan(count, hidden, vocab);
  if (p.run != kMaxRun) return p.bytes;
  // fewer tokens in runs of 8 leave more parts: the most that do
  const int64_t most = (kManyCtas - 1) / ops_ceil_div(hidden, kSumCols) * kMaxRun;
  return std::max(p.bytes, grad_plan(most, hidden, vocab).bytes);
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
  const int smem = sort_smem(p.digit_bits);
  const int64_t row = grad->cols * dtype_bytes(grad->dtype), pitch = grad->stride * dtype_bytes(grad->dtype);
  const bool flat = row == pitch && reinterpret_cast<uintptr_t>(grad->data) % 16 == 0 && row * grad->rows % 16 == 0;
  auto sort = [&](auto kernel, unsigned grid) {
    return launch_chained(kernel, dim3(grid), dim3(kSortThreads), smem, s, tokens->data, tokens->bits == 64,
                          static_cast<int>(dout->rows), static_cast<int>(grad->rows), p.passes, p.digit_bits,
                          reinterpret_cast<uint2*>(ws + p.buf_off[0]), reinterpret_cast<uint2*>(ws + p.buf_off[1]),
                          static_cast<char*>(grad->data), pitch, flat ? row * grad->rows : row, flat ? 1 : 0);
  };
  // The clusters after the first zero the gradient: two CTAs per SM (one where digits
  // of 10 bits take 139,264 bytes a CTA). The function's limit is set to the largest
  // size on every call, host only and under a microsecond: it is state of the device
  // that all threads share, and a limit of this call's own size would fail the
  // launch of another thread's larger one.
  constexpr int kLimit = sort_smem(kSortMaxBits);
  if (wide_sort(dout->rows, accumulate ? 0 : row * grad->rows)) {
    LST_TRY_CUDA(cudaFuncSetAttribute(sort_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLimit), who);
    LST_TRY_CUDA(cudaFuncSetAttribute(sort_kernel<16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), who);
    LST_TRY_CUDA(sort(sort_kernel<16>, accumulate ? 16 : 2 * 152), who);
  } else {
    LST_TRY_CUDA(cudaFuncSetAttribute(sort_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kLimit), who);
    LST_TRY_CUDA(sort(sort_kernel<8>, accumulate ? 8 : 2 * 152), who);
  }
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
