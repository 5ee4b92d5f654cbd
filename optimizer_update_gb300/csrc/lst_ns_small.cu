// Newton-Schulz orthogonalisation of small matrices in one kernel: at most 128
// on the short side, 4096 on the long one.
//
// The tiled path (lst_muon.cu, lst_gemm.cu) takes 11 dependent launches, about
// 90 us however small the matrix; this kernel 15 us for 16 x 16, 27 for 64 x 300, 46
// for 128 x 1000 and 80 for 128 x 4096. Here a cluster of 1 to 8 CTAs keeps the whole
// matrix and the iteration on chip. With X (m x n, m <= 128 <= n, a tall matrix
// transposed on its way in and out) each CTA holds a slice of up to 512 columns
// of X in shared memory, in fp16, and its own copies of the m x m matrices:
//   A = X X^T     partial over the slice on the tensor cores, partial sums added
//                 over the cluster in rank order through distributed shared
//                 memory: each CTA adds up 128 / C rows and sends them to all;
//   Q, Q A, ...   128 x 128 x 128 products, every CTA for itself (0.3 us of MMA);
//   X <- S X      the slice's columns, in place.
// One layout serves all operands: 64 columns x 128 rows in 128-byte swizzled rows
// are a K-major operand of A = X X^T (columns summed) and an MN-major operand of
// S X (rows summed).
// Steps run as 2 + 1 + 2 + ... (lst_muon.cu): here a product costs about 0.7 us
// and a Gram matrix with its exchange about 4.
// Bound by latency: MMA, tensor memory to registers to shared memory and a
// barrier, about 11 products, 3 exchanges and 3 applications one after another.
#include "lst_ns.h"

#include <algorithm>
#include <mutex>

#include "lst_device.cuh"
#include "lst_ops.h"
#include "lst_tc.cuh"

namespace lst {

namespace {

constexpr int kM = 128;                       // rows held, zero beyond m
constexpr int kChunk = kM * 128;              // bytes of 64 columns
constexpr int kMaxChunks = 8;                 // of X per CTA
constexpr int kMatrix = 2 * kChunk;           // bytes of an m x m matrix
constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kSmallSmem = kMaxChunks * kChunk + 3 * kMatrix + 1024 + 256;

__device__ int g_ns_small_error;

struct SmallTable {
  NsSmallItem it[kNsSmallItems];
};

// Byte of element (row, column of a 64-column chunk) in a swizzled chunk.
__device__ __forceinline__ uint32_t chunk_at(int row, int col) {
  return row * 128 + ((((col >> 3) ^ (row & 7)) << 4) | ((col & 7) << 1));
}
// Byte of a float4 of the exchange buffer (128 x 128 fp32).
__device__ __forceinline__ uint32_t part_at(int row, int quad) { return row * 512 + ((quad ^ (row & 7)) << 4); }

// Shared memory is only reached through these. They are volatile, so they keep
// their order among themselves and with the barriers; they do not clobber
// memory, which would send the kernel's own variables through local memory.
__device__ __forceinline__ void st_shared16(uint32_t a, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v));
}
__device__ __forceinline__ void st_shared_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w));
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t a) {
  float4 r;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct Small {
  uint32_t x, s0, s1, s2, part, bar, tmem;
  uint32_t parity;
  int rank, ranks, warp, lane;
  int row, quarter;  // of the accumulator: the thread's row, the warp's quarter of 128 columns
  int depth;         // m rounded up to 16: the rows and columns of S that are used
  bool ok;

  __device__ __forceinline__ uint32_t lanes() const { return tmem + (static_cast<uint32_t>(row & ~31) << 16); }

  // Operands written and visible, then `issue` by one thread, then everyone
  // waits for its products.
  template <class Issue>
  __device__ __forceinline__ void multiply(Issue issue) {
    tc::fence_async_proxy_cta();
    tc::fence_before();
    __syncthreads();
    if (warp == 0) {
      tc::fence_after();
      if (tc::elect_one()) {
        issue();
        tc::mma_commit(bar);
      }
      __syncwarp();
    }
    if (ok) ok = tc::mbar_wait(bar, parity);
    parity ^= 1;
    tc::fence_after();
    __syncwarp();
  }

  // out = alpha a b + beta a + diag I, in fp16. Rows beyond `depth` hold what
  // they will: a row of a product depends on no other row of its first factor,
  // and sums and columns end at `depth`.
  __device__ __forceinline__ void product(uint32_t out, uint32_t a, uint32_t b, float alpha, float beta, float diag) {
    const uint32_t d = tmem;
    const int steps = depth / 16;
    multiply([=]() {
      const uint32_t idesc = tc::instr_desc(kM, 16 * steps, false, false, false);
#pragma unroll 1
      for (int k = 0; k < steps; ++k) {
        const uint32_t off = (k >> 2) * kChunk + (k & 3) * 32;
        tc::mma_f16(d, tc::smem_desc(a + off, false), tc::smem_desc(b + off, false), idesc, k != 0);
      }
    });
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col0 = quarter * 32 + j * 16;
      if (col0 >= depth) break;
      float v[16];
      tc::tmem_ld16(lanes() + col0, v);
      const uint32_t at0 = (quarter >> 1) * kChunk + chunk_at(row, (quarter & 1) * 32 + j * 16);
      const uint32_t at1 = (quarter >> 1) * kChunk + chunk_at(row, (quarter & 1) * 32 + j * 16 + 8);
      const uint4 y0 = ld_shared_v4(a + at0), y1 = ld_shared_v4(a + at1);
      const uint32_t y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
      tc::tmem_ld_wait();
      const int at_diag = row - col0;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
        w[i] = half2_bits(__fmaf_rn(beta, f.x, v[2 * i] * alpha) + (at_diag == 2 * i ? diag : 0.0f),
                          __fmaf_rn(beta, f.y, v[2 * i + 1] * alpha) + (at_diag == 2 * i + 1 ? diag : 0.0f));
      }
      st_shared_v4(out + at0, w[0], w[1], w[2], w[3]);
      st_shared_v4(out + at1, w[4], w[5], w[6], w[7]);
    }
  }

  // Adds up the partial Gram matrices of C CTAs and gives s0 to all of them: CTA
  // `rank` takes every C-th row.
  template <int C>
  __device__ __forceinline__ void exchange(float alpha) {
    constexpr int kRounds = kM / C / kSmallWarps;
    float4 v[kRounds][C];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int r = (warp + i * kSmallWarps) * C + rank;
      if (r < depth && 4 * lane < depth)
#pragma unroll
        for (int c = 0; c < C; ++c) v[i][c] = ld_cluster_v4(tc::map_to_rank(part + part_at(r, lane), c));
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int r = (warp + i * kSmallWarps) * C + rank;
      if (r < depth && 4 * lane < depth) {
        float4 sum = v[i][0];
#pragma unroll
        for (int c = 1; c < C; ++c)
          sum = make_float4(sum.x + v[i][c].x, sum.y + v[i][c].y, sum.z + v[i][c].z, sum.w + v[i][c].w);
        const uint32_t lo = half2_bits(sum.x * alpha, sum.y * alpha), hi = half2_bits(sum.z * alpha, sum.w * alpha);
        const uint32_t at = s0 + (lane >> 4) * kChunk + chunk_at(r, (lane & 15) * 4);
#pragma unroll
        for (int c = 0; c < C; ++c)
          asm volatile("st.shared::cluster.v2.b32 [%0], {%1,%2};" ::"r"(tc::map_to_rank(at, c)), "r"(lo), "r"(hi));
      }
    }
  }

  // s0 = X X^T summed over the cluster. Uses the space of s1 and s2.
  __device__ __forceinline__ void gram(int chunks) {
    const uint32_t xs = x, d = tmem;
    const int columns = depth;
    multiply([=]() {
      const uint32_t idesc = tc::instr_desc(kM, columns, false, false, false);
#pragma unroll 1
      for (int c = 0; c < 4 * chunks; ++c) {
        const uint64_t o = tc::smem_desc(xs + (c >> 2) * kChunk + (c & 3) * 32, false);
        tc::mma_f16(d, o, o, idesc, c != 0);
      }
    });
    constexpr float alpha = kScaleA / (kScaleX * kScaleX);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col0 = quarter * 32 + j * 16;
      if (col0 >= depth) break;
      float v[16];
      tc::tmem_ld16(lanes() + col0, v);
      tc::tmem_ld_wait();
      if (ranks == 1) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = half2_bits(v[2 * i] * alpha, v[2 * i + 1] * alpha);
        const uint32_t at = s0 + (quarter >> 1) * kChunk;
        st_shared_v4(at + chunk_at(row, (quarter & 1) * 32 + j * 16), w[0], w[1], w[2], w[3]);
        st_shared_v4(at + chunk_at(row, (quarter & 1) * 32 + j * 16 + 8), w[4], w[5], w[6], w[7]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
          st_shared_v4(part + part_at(row, col0 / 4 + u), __float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                       __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
      }
    }
    if (ranks == 1) return;
    __syncwarp();
    tc::cluster_sync();
    if (ranks == 2) exchange<2>(alpha);
    if (ranks == 4) exchange<4>(alpha);
    if (ranks == 8) exchange<8>(alpha);
    tc::fence_async_proxy();
    __syncwarp();
    tc::cluster_sync();
  }

  // tensor memory = sa X, all columns of the slice
  __device__ __forceinline__ void apply(uint32_t sa, int chunks) {
    const uint32_t xs = x, d = tmem;
    const int steps = depth / 16;
    multiply([=]() {
#pragma unroll 1
      for (int c = 0; c < chunks; c += 4) {
        const uint32_t idesc = tc::instr_desc(kM, min(4, chunks - c) * 64, false, false, true);
#pragma unroll 1
        for (int k = 0; k < steps; ++k)
          tc::mma_f16(d + c * 64, tc::smem_desc(sa + (k >> 2) * kChunk + (k & 3) * 32, false),
                      tc::smem_desc(xs + c * kChunk + k * 2048, true, kChunk), idesc, k != 0);
      }
    });
  }
};

template <bool F32>
__device__ __forceinline__ float load_value(const void* p, int64_t i) {
  return F32 ? static_cast<const float*>(p)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

// `format` < 0: the bf16 result; otherwise the weight's update.
__device__ __forceinline__ void finish(const NsSmallItem& it, int format, float decay, int64_t i, float o) {
  if (format < 0) {
    static_cast<__nv_bfloat16*>(it.out)[i] = __float2bfloat16_rn(o);
  } else if (format == LST_L12_BF16) {
    const float w = __uint_as_float(static_cast<uint32_t>(static_cast<uint16_t*>(it.out)[i]) << 16);
    static_cast<__nv_bfloat16*>(it.out)[i] = __float2bfloat16_rn(__fsub_rn(__fmul_rn(w, decay), __fmul_rn(it.step, o)));
  } else {
    const float w = __fsub_rn(__fmul_rn(static_cast<float*>(it.out)[i], decay), __fmul_rn(it.step, o));
    static_cast<float*>(it.out)[i] = w;
    if (format == LST_L16_MIXED) reinterpret_cast<__nv_bfloat16*>(it.w16)[i] = __float2bfloat16_rn(w);
  }
}

template <bool F32, bool MOM>
__global__ void __launch_bounds__(kSmallThreads, 1)
    ns_small_kernel(const __grid_constant__ SmallTable table, const __grid_constant__ NsSmallCall call, int ranks,
                    int chunks) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (tc::smem_addr(smem_raw) + 1023) & ~1023u;
  Small k;
  k.x = base;
  k.s0 = base + kMaxChunks * kChunk;
  k.s1 = k.s0 + kMatrix;
  k.s2 = k.s1 + kMatrix;
  k.part = k.s1;
  k.bar = base + kMaxChunks * kChunk + 3 * kMatrix;
  const uint32_t sums = k.bar + 16, slot = sums + 8 * kMaxCluster;
  k.warp = threadIdx.x >> 5;
  k.lane = threadIdx.x & 31;
  k.row = 32 * (k.warp & 3) + k.lane;
  k.quarter = k.warp >> 2;
  k.rank = static_cast<int>(tc::cluster_rank());
  k.ranks = ranks;
  k.parity = 0;
  k.ok = true;
  let_next_start();
  if (threadIdx.x == 0) {
    tc::mbar_init(k.bar, 1);
    tc::mbar_init_fence();
  }
  if (k.warp == 0) {
    __syncwarp();
    tc::tmem_alloc(slot, 512);
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(k.tmem) : "r"(slot));
  wait_for_previous();

  const NsSmallItem& it = table.it[blockIdx.x / ranks];
  const int rows = static_cast<int>(call.rows), cols = static_cast<int>(call.cols);
  const bool tall = rows > cols;
  const int m = tall ? cols : rows, n = tall ? rows : cols;
  k.depth = (m + 15) & ~15;
  const int width = chunks * 64, n0 = k.rank * width;
  const int mine = max(0, min(width, n - n0));  // columns of X (rows of a tall matrix) held here
  // the matrix elements held here: `outer` rows of `inner` contiguous ones
  const int outer = tall ? mine : m, inner = tall ? m : mine;
  const int64_t first = tall ? static_cast<int64_t>(n0) * it.ld : n0;
  const int64_t first_m = tall ? static_cast<int64_t>(n0) * cols : n0;  // momentum: rows of `cols`

  // 128 rows x 32 columns at a time, a warp's 8 loads in flight together
  auto for_values = [&](auto visit) {
#pragma unroll 1
    for (int r0 = k.warp; r0 < outer; r0 += 8 * kSmallWarps)
#pragma unroll 1
      for (int c = k.lane; c < inner; c += 32) {
        float g[8], mom[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = r0 + j * kSmallWarps;
          if (r < outer) {
            g[j] = load_value<F32>(it.g, first + r * it.ld + c);
            if (MOM) mom[j] = it.mom[first_m + static_cast<int64_t>(r) * cols + c];
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = r0 + j * kSmallWarps;
          if (r < outer) visit(r, c, g[j], mom[j]);
        }
      }
  };

  // momentum, and the sum of squares; once more over scaled values where the sum is out
  // of range (all CTAs of the cluster see the same sum)
  __shared__ float warp_sum[kSmallWarps];
  __shared__ float shared_sum;
  float pre = 1.0f, total;
#pragma unroll 1
  for (int pass = 0;; ++pass) {
    float sum = 0.0f;
    for_values([&](int r, int c, float g, float mom) {
      if (MOM) {
        if (pass == 0) {
          mom = new_momentum(mom, g, call.s);
          it.mom[first_m + static_cast<int64_t>(r) * cols + c] = mom;
        }
        g = muon_u(g, mom, call.s);
      }
      g *= pre;
      sum = __fmaf_rn(g, g, sum);
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_down_sync(0xffffffffu, sum, o);
    if (k.lane == 0) warp_sum[k.warp] = sum;
    // rows and columns beyond the matrix are zero
    if (pass == 0)
      for (int i = threadIdx.x; i < chunks * kChunk / 16; i += kSmallThreads) st_shared_v4(k.x + 16 * i, 0, 0, 0, 0);
    __syncthreads();
    const uint32_t now = sums + 4 * kMaxCluster * pass;
    if (threadIdx.x < ranks) {
      float x = 0.0f;
#pragma unroll
      for (int i = 0; i < kSmallWarps; ++i) x += warp_sum[i];
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::map_to_rank(now + 4 * k.rank, threadIdx.x)), "f"(x));
    }
    __syncwarp();
    tc::cluster_sync();
    if (threadIdx.x == 0) {
      float x = 0.0f;
      for (int i = 0; i < ranks; ++i) {
        float y;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y) : "r"(now + 4 * i));
        x += y;
      }
      shared_sum = x;
    }
    __syncthreads();
    total = shared_sum;
    if (pass == 1 || ordinary_sum(total)) break;
    pre = other_pre(total);
  }
  const float inv = ns_inv(total, pre, call.s.eps);
  for_values([&](int r, int c, float g, float mom) {
    if (MOM) g = muon_u(g, mom, call.s);
    const int xr = tall ? c : r, xc = tall ? r : c;
    st_shared16(k.x + (xc >> 6) * kChunk + chunk_at(xr, xc & 63), __half_as_ushort(__float2half_rn(g * pre * inv)));
  });

  bool pair = true;
  for (int done = 0; done < call.steps;) {
    const bool two = pair && call.steps - done >= 2;
    pair = !pair;
    k.gram(chunks);
    // Q = s1 from A = s0; for two steps also Q A = s2, A' = s0, Q' = s2, Q' Q = s0.
    // One loop, not five calls: a kernel that runs once is bound by fetching its
    // instructions where its code is long (inlined five times: 3 x slower).
#pragma unroll 1
    for (int op = 0; op < (two ? 5 : 1); ++op) {
      const bool poly = op == 0 || op == 3;
      const uint32_t out = op == 0 ? k.s1 : op == 1 || op == 3 ? k.s2 : k.s0;
      const uint32_t a = poly ? k.s0 : op == 1 ? k.s1 : k.s2;
      const uint32_t b = poly || op == 1 ? k.s0 : k.s1;
      const float alpha = poly      ? kNsC * kScaleQ / (kScaleA * kScaleA)
                          : op == 1 ? kScaleQA / (kScaleQ * kScaleA)
                          : op == 2 ? kScaleA / (kScaleQA * kScaleQ)
                                    : kScaleR / (kScaleQ * kScaleQ);
      k.product(out, a, b, alpha, poly ? kNsB * kScaleQ / kScaleA : 0.0f, poly ? kNsA * kScaleQ : 0.0f);
    }
    const float scale = two ? kScaleR : kScaleQ;
    done += two ? 2 : 1;
    k.apply(two ? k.s0 : k.s1, chunks);
    const bool final = done >= call.steps;
    const float back = final ? 1.0f / (scale * kScaleX) : 1.0f / scale;
#pragma unroll 1
    for (int c = k.quarter; c < 4 * chunks; c += 4) {  // 16 columns at a time
      float v[16];
      __syncwarp();
      tc::tmem_ld16(k.lanes() + 16 * c, v);
      tc::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= back;
      if (!final) {
        if (k.row >= k.depth) continue;  // X stays zero there
        const uint32_t at = k.x + (c >> 2) * kChunk;
        st_shared_v4(at + chunk_at(k.row, (c & 3) * 16), half2_bits(v[0], v[1]), half2_bits(v[2], v[3]),
                     half2_bits(v[4], v[5]), half2_bits(v[6], v[7]));
        st_shared_v4(at + chunk_at(k.row, (c & 3) * 16 + 8), half2_bits(v[8], v[9]), half2_bits(v[10], v[11]),
                     half2_bits(v[12], v[13]), half2_bits(v[14], v[15]));
        continue;
      }
      // the result: a column of X is a row of a tall matrix, with the lanes
      // consecutive in it; a wide one goes through the warp's own 32 x 17 words
      // to have 16 lanes consecutive in a row
      const uint32_t stage = k.s1 + k.warp * (32 * 17 * 4);
      if (!tall) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + (k.lane * 17 + i) * 4), "f"(v[i]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          asm volatile("ld.shared.f32 %0, [%1];"
                       : "=f"(v[i])
                       : "r"(stage + ((2 * i + (k.lane >> 4)) * 17 + (k.lane & 15)) * 4));
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int r = tall ? k.row : (k.row & ~31) + 2 * i + (k.lane >> 4);   // of X
        const int col = 16 * c + (tall ? i : k.lane & 15);
        if (r < m && col < mine) {
          const int64_t at = tall ? static_cast<int64_t>(n0 + col) * it.out_ld + r : static_cast<int64_t>(r) * it.out_ld + n0 + col;
          finish(it, call.format, call.decay, at, v[i]);
        }
      }
    }
  }
  if (!k.ok) {
    atomicExch(&g_ns_small_error, 1);
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);  // products in flight land
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  if (k.warp == 0) {
    __syncwarp();
    tc::tmem_free(k.tmem, 512);
  }
}

// ---- two steps of a Gram matrix of up to 256 rows -------------------------------------
// The five products between A and Q' Q of one matrix, by a CTA pair with the
// matrices in shared memory: CTA r holds rows 128 r .. 128 r + 127, which are its
// rows of every first factor and, all being symmetric, its half of every second
// one. As five launches of the tiled kernel they cost 5 us each whatever their size.
constexpr int kHalf = 4 * kChunk;  // bytes of 128 rows x 256 columns
constexpr int kChainSmem = 3 * kHalf + 1024 + 64;

struct Chain {
  uint32_t s0, s1, s2, ready, bar, tmem, parity;
  int rank, warp, lane, row, quarter, depth;
  bool ok;

  __device__ __forceinline__ void product(uint32_t out, uint32_t a, uint32_t b, float alpha, float beta, float diag) {
    tc::fence_async_proxy_cta();
    tc::fence_before();
    __syncthreads();
    if (threadIdx.x == 0) tc::mbar_arrive_cluster(tc::map_to_rank(ready, 0));
    if (warp == 0) {
      __syncwarp();
      if (rank == 0) {
        ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(ready, parity));
        tc::fence_async_proxy();
        tc::fence_after();
        if (ok && tc::elect_one()) {
          constexpr uint32_t idesc = tc::instr_desc(256, 256, false, false, false);
#pragma unroll 1
          for (int k = 0; k < depth / 16; ++k) {
            const uint32_t off = (k >> 2) * kChunk + (k & 3) * 32;
            tc::mma_f16_pair(tmem, tc::smem_desc(a + off, false), tc::smem_desc(b + off, false), idesc, k != 0);
          }
          tc::mma_commit_pair(bar);
        }
        __syncwarp();
      }
    }
    ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(bar, parity));
    parity ^= 1;
    tc::fence_after();
    __syncwarp();
    const int row_global = 128 * rank + row;
#pragma unroll 1
    for (int j = 0; j < 4; ++j) {
      const int col0 = quarter * 64 + j * 16;
      if (col0 >= depth) break;
      float v[16];
      tc::tmem_ld16(tmem + (static_cast<uint32_t>(row & ~31) << 16) + col0, v);
      const uint32_t at0 = quarter * kChunk + chunk_at(row, j * 16), at1 = quarter * kChunk + chunk_at(row, j * 16 + 8);
      const uint4 y0 = ld_shared_v4(a + at0), y1 = ld_shared_v4(a + at1);
      const uint32_t y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
      tc::tmem_ld_wait();
      const int at_diag = row_global - col0;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&y[i]));
        w[i] = half2_bits(__fmaf_rn(beta, f.x, v[2 * i] * alpha) + (at_diag == 2 * i ? diag : 0.0f),
                          __fmaf_rn(beta, f.y, v[2 * i + 1] * alpha) + (at_diag == 2 * i + 1 ? diag : 0.0f));
      }
      st_shared_v4(out + at0, w[0], w[1], w[2], w[3]);
      st_shared_v4(out + at1, w[4], w[5], w[6], w[7]);
    }
  }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kSmallThreads, 1)
    ns_chain_kernel(__half* s, int m, int64_t ld, int64_t pitch) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (tc::smem_addr(smem_raw) + 1023) & ~1023u;
  Chain k;
  k.s0 = base;
  k.s1 = base + kHalf;
  k.s2 = base + 2 * kHalf;
  k.ready = base + 3 * kHalf;
  k.bar = k.ready + 8;
  const uint32_t slot = k.bar + 8;
  k.warp = threadIdx.x >> 5;
  k.lane = threadIdx.x & 31;
  k.row = 32 * (k.warp & 3) + k.lane;
  k.quarter = k.warp >> 2;
  k.rank = static_cast<int>(tc::cluster_rank());
  k.depth = (m + 15) & ~15;
  k.parity = 0;
  k.ok = true;
  let_next_start();
  if (threadIdx.x == 0) {
    tc::mbar_init(k.ready, 2);
    tc::mbar_init(k.bar, 1);
    tc::mbar_init_fence();
  }
  if (k.warp == 1) {
    __syncwarp();
    tc::tmem_alloc_pair(slot, 256);
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(k.tmem) : "r"(slot));
  wait_for_previous();

  // 128 rows x 32 pieces of 16 bytes; what lies beyond m is zero
  __half* const mine = s + static_cast<int64_t>(blockIdx.x >> 1) * pitch;
  const int piece = k.lane;
  uint4 v[kM / kSmallWarps];
#pragma unroll
  for (int i = 0; i < kM / kSmallWarps; ++i) {
    const int r = 128 * k.rank + k.warp + i * kSmallWarps;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < m && 8 * piece < m) {
      v[i] = *reinterpret_cast<const uint4*>(mine + r * ld + 8 * piece);
      uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      if (8 * piece + 8 > m)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * piece + e >= m) w[e >> 1] &= (e & 1) ? 0x0000ffffu : 0xffff0000u;
      v[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < kM / kSmallWarps; ++i)
    st_shared_v4(k.s0 + (piece >> 3) * kChunk + chunk_at(k.warp + i * kSmallWarps, (piece & 7) * 8), v[i].x, v[i].y, v[i].z, v[i].w);

  // Q = s1 from A = s0, Q A = s2, A' = s0, Q' = s2, Q' Q = s0
#pragma unroll 1
  for (int op = 0; op < 5; ++op) {
    const bool poly = op == 0 || op == 3;
    const uint32_t out = op == 0 ? k.s1 : op == 1 || op == 3 ? k.s2 : k.s0;
    const uint32_t a = poly ? k.s0 : op == 1 ? k.s1 : k.s2;
    const uint32_t b = poly || op == 1 ? k.s0 : k.s1;
    const float alpha = poly      ? kNsC * kScaleQ / (kScaleA * kScaleA)
                        : op == 1 ? kScaleQA / (kScaleQ * kScaleA)
                        : op == 2 ? kScaleA / (kScaleQA * kScaleQ)
                                  : kScaleR / (kScaleQ * kScaleQ);
    k.product(out, a, b, alpha, poly ? kNsB * kScaleQ / kScaleA : 0.0f, poly ? kNsA * kScaleQ : 0.0f);
  }
  __syncthreads();
#pragma unroll 4
  for (int i = 0; i < kM / kSmallWarps; ++i) {
    const int r = k.warp + i * kSmallWarps, row = 128 * k.rank + r;
    if (row < m && 8 * piece < m) {  // ld is a multiple of 64: a last piece may reach past m
      const uint4 w = ld_shared_v4(k.s0 + (piece >> 3) * kChunk + chunk_at(r, (piece & 7) * 8));
      *reinterpret_cast<uint4*>(mine + row * ld + 8 * piece) = w;
    }
  }
  if (!k.ok) {
    atomicExch(&g_ns_small_error, 1);
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);  // products in flight land
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  if (k.warp == 1) {
    __syncwarp();
    tc::tmem_free_pair(k.tmem, 256);
  }
}

}  // namespace

bool ns_small_fits(int64_t rows, int64_t cols) {
  return std::min(rows, cols) <= kM && std::max(rows, cols) <= kMaxCluster * kMaxChunks * 64;
}

cudaError_t ns_small(const NsSmallItem* items, int count, const NsSmallCall& call, cudaStream_t stream) {
  constexpr int kMaxDevices = 16;
  static std::mutex mu;
  static bool ready[kMaxDevices][4] = {};
  const bool mom = count > 0 && items[0].mom != nullptr;
  const int which = (call.f32 ? 2 : 0) + (mom ? 1 : 0);
  auto kernel = call.f32 ? (mom ? ns_small_kernel<true, true> : ns_small_kernel<true, false>)
                         : (mom ? ns_small_kernel<false, true> : ns_small_kernel<false, false>);
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= kMaxDevices || !ready[dev][which]) {
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
      if (err != cudaSuccess) return err;
      if (dev < kMaxDevices) ready[dev][which] = true;
    }
  }
  const int64_t n = std::max(call.rows, call.cols);
  for (int first = 0; first < count; first += kNsSmallItems) {
    const int now = std::min(kNsSmallItems, count - first);
    SmallTable table;
    for (int i = 0; i < now; ++i) table.it[i] = items[first + i];
    // as many CTAs to a matrix as the GPU has for each, one for every 64 columns
    // at most, and as many as its columns need
    int ranks = 1;
    while (ranks < kMaxCluster && (n > ranks * kMaxChunks * 64 || (2 * ranks * now <= 144 && n > ranks * 64))) ranks *= 2;
    const int chunks = static_cast<int>(ops_ceil_div(ops_ceil_div(n, 64), ranks));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(now * ranks));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = kSmallSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    err = cudaLaunchKernelEx(&cfg, kernel, table, call, ranks, chunks);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t ns_chain(__half* s, int64_t m, int64_t ld, int64_t pitch, int64_t count, cudaStream_t stream) {
  // per device, host only, under a microsecond
  cudaError_t err = cudaFuncSetAttribute(ns_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChainSmem);
  for (int64_t first = 0; err == cudaSuccess && first < count; first += 1 << 20) {
    const int64_t now = std::min<int64_t>(count - first, 1 << 20);
    err = launch_chained(ns_chain_kernel, dim3(static_cast<unsigned>(2 * now)), dim3(kSmallThreads), kChainSmem, stream,
                         s + first * pitch, static_cast<int>(m), ld, pitch);
  }
  return err;
}

cudaError_t ns_small_take_error(int* out) {
  cudaError_t err = cudaMemcpyFromSymbol(out, g_ns_small_error, sizeof(int));
  if (err != cudaSuccess || *out == 0) return err;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_ns_small_error, &zero, sizeof(int));
}

}  // namespace lst
