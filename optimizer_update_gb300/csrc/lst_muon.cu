// Newton-Schulz orthogonalisation and the Muon step over packed blocks.
//
// Mathematics, for a wide matrix (m rows, n >= m columns; a tall one is the
// same from the other side, X <- X Q with A = X^T X, in its own row order). With
// X_0 = U / (|U|_F + eps) a step is X <- Q X, Q = a I + b A + c A^2, A = X X^T. All Q and A are polynomials of
// X_0 X_0^T: symmetric, and they commute. So two steps can share one Gram
// matrix: with Q_1 from A, the next Gram matrix is A' = Q_1 A Q_1, Q_2 comes
// from A', and X <- (Q_2 Q_1) X. A pair so formed costs five m x m products and
// two products with X where two single steps cost two and four; products with a
// symmetric result are formed on one triangle only and cost half. For 5 steps,
// counting m^2 n and m^3 in units of two operations per half product:
//   single steps  15 m^2 n +  5 m^3
//   2 + 1 + 2      9 m^2 n + 11 m^3    equal at n = m, 1.5 x less at n = 8 m
// Carrying the Gram matrix further than two steps would cost less still, but
// its rounding error grows with the square of the conditioning: on matrices
// with singular values falling as 1/i, 2 + 3 steps put the result 8e-3 from the
// 64-bit one where 2 + 1 + 2 and single steps both put it 4e-3 (fp16, below).
//
// Precision. Values are held in fp16, not bf16: at 11 bits instead of 8 the
// result is 1.2e-3 from the 64-bit one where bf16 leaves 1e-2, at the same
// tensor-core rate. Their range needs no watching: |X| <= 1.21 in the 2-norm
// after any step (the largest value of a s + b s^3 + c s^5 on [0, 1.21]), so
// no entry of X, A, Q, Q A and Q_2 Q_1 exceeds 1.21, 1.46, 3.5, 1.3, 11.9, and each
// kind is stored times a power of two that leaves these below 65504 and the
// smallest normal number at 1e-9 to 1e-8. Q is stored whole, not as Q - a I:
// a I + (Q - a I) cancels to about 1 where singular values have converged, and
// would take the rounding of the larger parts into X (measured 2 x the error).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <vector>

#include "lst_device.cuh"
#include "lst_gemm.h"
#include "lst_ns.h"
#include "lst_ops.h"

namespace lst {

namespace {

constexpr int kItemsPerLaunch = 32;
constexpr int kNormBlocks = 1024;  // partial sums per matrix
// Inputs of the matrices whose norms are taken together: their second read, to
// scale them, then comes from L2 (129 MB) for the most part.
constexpr int64_t kIngestBytes = int64_t(64) << 20;

// One matrix on its way in.
struct Item {
  const void* g;      // gradient, or the matrix itself
  float* mom;         // momentum, or null
  __half* x;          // rows x ldx values
  float2* part;       // kNormBlocks partial sums of (u * pre)^2, and pre
  int64_t rows, cols, ld, ldx;
};
struct ItemTable {
  Item it[kItemsPerLaunch];
};
__device__ __forceinline__ float load_in(const void* p, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}
template <bool F32>
__device__ __forceinline__ void load_in8(const void* p, int64_t i, float (&v)[8]) {
  if (F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
  }
}

// Whether every row of the matrix can be read in vectors of 8.
template <bool MOM>
__device__ __forceinline__ bool vector_rows(const Item& it) {
  return it.cols % 8 == 0 && it.ld % 8 == 0 && (reinterpret_cast<uintptr_t>(it.g) & 15) == 0 &&
         (!MOM || (reinterpret_cast<uintptr_t>(it.mom) & 15) == 0);
}

// Row and first column of vector q of 8, with 32-bit division where it suffices.
__device__ __forceinline__ void vector_at(int64_t q, uint32_t per_row, int64_t* r, int64_t* c) {
  *r = q <= 0xffffffffll ? static_cast<int64_t>(static_cast<uint32_t>(q) / per_row) : q / per_row;
  *c = (q - *r * per_row) * 8;
}

// A block's share of the sum of (u * pre)^2, by thread. kFirst: with m = momentum m + g in
// place, and pre = 1.
template <bool F32, bool MOM, bool kFirst>
__device__ __forceinline__ float squares(const Item& it, const NsMomentum& s, float pre) {
  float sum = 0.0f;
  if (vector_rows<MOM>(it)) {
    const uint32_t per_row = static_cast<uint32_t>(it.cols / 8);
    const int64_t total = it.rows * per_row;
    const bool flat = it.ld == it.cols;
#pragma unroll (kFirst ? 4 : 1)
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < total; q += static_cast<int64_t>(gridDim.x) * 256) {
      int64_t r = 0, c = q * 8;
      if (!flat) vector_at(q, per_row, &r, &c);
      const int64_t at = r * it.ld + c;
      float g[8];
      load_in8<F32>(it.g, at, g);
      if (MOM) {
        float4* p = reinterpret_cast<float4*>(it.mom) + 2 * q;
        float4 a = p[0], b = p[1];
        if (kFirst) {
          a = make_float4(new_momentum(a.x, g[0], s), new_momentum(a.y, g[1], s), new_momentum(a.z, g[2], s),
                          new_momentum(a.w, g[3], s));
          b = make_float4(new_momentum(b.x, g[4], s), new_momentum(b.y, g[5], s), new_momentum(b.z, g[6], s),
                          new_momentum(b.w, g[7], s));
          p[0] = a;
          p[1] = b;
        }
        const float m[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = muon_u(g[i], m[i], s);
      }
      float x = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!kFirst) g[i] *= pre;
        x = __fmaf_rn(g[i], g[i], x);
      }
      sum += x;
    }
  } else {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < it.rows; r += warps) {
#pragma unroll (kFirst ? 4 : 1)
      for (int64_t c = lane; c < it.cols; c += 32) {
        float u = load_in(it.g, r * it.ld + c, F32);
        if (MOM) {
          float* p = it.mom + r * it.cols + c;
          float m = *p;
          if (kFirst) *p = m = new_momentum(m, u, s);
          u = muon_u(u, m, s);
        }
        if (!kFirst) u *= pre;
        sum = __fmaf_rn(u, u, sum);
      }
    }
  }
  return sum;
}

// The sum over the block's threads, in all of them.
__device__ __forceinline__ float block_sum(float sum, float (&red)[8]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_down_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) sum += red[i];
  return sum;
}

// Outside the kernels' own code, which it would cost registers (a TinyLlama layer by Muon
// 1200 -> 1210 us): the block's sum again, scaled; and the join of sums of three ranges,
// of which the largest there is sets `pre`.
template <bool F32, bool MOM>
__device__ __noinline__ float2 sum_again(const Item& it, const NsMomentum& s, float sum, float (&red)[8]) {
  const float pre = other_pre(sum);
  sum = block_sum(squares<F32, MOM, false>(it, s, pre), red);
  return make_float2(sum, sum == 0.0f ? 1.0f : pre);  // nothing but zeros, or nothing at all
}
__device__ __noinline__ float2 join_ranges(const float2* part, int parts, float sum, float (&red)[2][8]) {
  float small = 0.0f, large = 0.0f;
  for (int i = threadIdx.x; i < parts; i += 256) {
    const float2 p = part[i];
    if (p.y == kSmallPre) small += p.x;
    if (p.y == kLargePre) large += p.x;
  }
  small = block_sum(small, red[0]);
  large = block_sum(large, red[1]);
  if (large != 0.0f) return make_float2(large + sum * kLargePre * kLargePre, kLargePre);  // or NaN
  if (sum > 0.0f) return make_float2(sum + small * 0x1p-100f * 0x1p-100f, 1.0f);
  return make_float2(small, kSmallPre);
}

// m = momentum m + g in place, and the sum of u^2 in fp32: over a thread's
// elements, a warp, a block and at last the blocks (each level adds at most a
// few hundred terms, an error under 1e-5 of the norm in the worst case, against
// the 5e-4 of the fp16 that it scales; fp64 would cost more than the loads do).
// A block whose sum is out of range reads its share again (from L2), scaled.
// Bound by memory: reads g and m, writes m.
template <bool F32, bool MOM>
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ ItemTable t, NsMomentum s) {
  let_next_start();
  wait_for_previous();
  const Item& it = t.it[blockIdx.y];
  __shared__ float red[2][8];
  const float sum = block_sum(squares<F32, MOM, true>(it, s, 1.0f), red[0]);
  float2 part = make_float2(sum, 1.0f);
  if (!ordinary_sum(sum)) part = sum_again<F32, MOM>(it, s, sum, red[1]);
  if (threadIdx.x == 0) it.part[blockIdx.x] = part;
}

// X_0 = u / (|u|_F + eps), in fp16 times kScaleX.
template <bool F32, bool MOM>
__global__ void __launch_bounds__(256, MOM ? 6 : 8) scale_kernel(const __grid_constant__ ItemTable t, NsMomentum s, int parts) {
  let_next_start();
  wait_for_previous();
  const Item& it = t.it[blockIdx.y];
  __shared__ float red[8], again[2][8];
  __shared__ int scaled;
  if (threadIdx.x == 0) scaled = 0;
  __syncthreads();
  float sum = 0.0f, pre = 1.0f;
  for (int i = threadIdx.x; i < parts; i += 256) {
    const float2 p = it.part[i];
    if (p.y == 1.0f)
      sum += p.x;
    else
      scaled = 1;
  }
  sum = block_sum(sum, red);
  if (scaled || sum == 0.0f) {
    const float2 joined = join_ranges(it.part, parts, sum, again);
    sum = joined.x;
    pre = joined.y;
  }
  const float inv = ns_inv(sum, pre, s.eps);
  if (vector_rows<MOM>(it)) {
    const uint32_t per_row = static_cast<uint32_t>(it.cols / 8);
    const int64_t total = it.rows * per_row;
#pragma unroll 4
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < total; q += static_cast<int64_t>(gridDim.x) * 256) {
      int64_t r, c;
      vector_at(q, per_row, &r, &c);
      float u[8];
      load_in8<F32>(it.g, r * it.ld + c, u);
      if (MOM) {
        float m[8];
        load_in8<true>(it.mom, q * 8, m);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = muon_u(u[i], m[i], s);
      }
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(u[2 * i] * pre * inv, u[2 * i + 1] * pre * inv);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(it.x + r * it.ldx + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < it.rows; r += warps) {
#pragma unroll 4
      for (int64_t c = lane; c < it.cols; c += 32) {
        float u = load_in(it.g, r * it.ld + c, F32);
        if (MOM) u = muon_u(u, it.mom[r * it.cols + c], s);
        it.x[r * it.ldx + c] = __float2half_rn(u * pre * inv);
      }
    }
  }
}

// AdamW on the tensors that do not take the Muon rule: the operations of
// lst_adamw_step, element by element.
struct AdamItem {
  const void* g;
  void* w;
  float *m, *v;
  uint16_t* w16;
  int64_t n;
};
struct AdamTable {
  AdamItem it[kItemsPerLaunch];
};
template <int FMT>
__global__ void __launch_bounds__(256) adam_kernel(const __grid_constant__ AdamTable t, Scalars s) {
  let_next_start();
  wait_for_previous();
  const AdamItem& it = t.it[blockIdx.y];
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < it.n;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const float g = load_in(it.g, i, FMT == F_L16F);
    float w = FMT == F_L12 ? bf16_lo(static_cast<uint16_t*>(it.w)[i]) : static_cast<float*>(it.w)[i];
    float m = it.m[i], v = it.v[i];
    adam_moments(g, m, v, s);
    w = adamw_finish<true>(w, m, v, s);
    it.m[i] = m;
    it.v[i] = v;
    if (FMT == F_L12) {
      static_cast<__nv_bfloat16*>(it.w)[i] = __float2bfloat16_rn(w);
    } else {
      static_cast<float*>(it.w)[i] = w;
      if (FMT == F_L16M) reinterpret_cast<__nv_bfloat16*>(it.w16)[i] = __float2bfloat16_rn(w);
    }
  }
}

// ---- a batch of matrices: buffers and products -----------------------------------

struct Shape2 {
  int64_t rows, cols;
  int64_t m() const { return rows < cols ? rows : cols; }
  int64_t n() const { return rows < cols ? cols : rows; }
  bool operator==(const Shape2& o) const { return rows == o.rows && cols == o.cols; }
  bool operator<(const Shape2& o) const {
    return m() != o.m() ? m() < o.m() : n() != o.n() ? n() < o.n() : rows < o.rows;
  }
};

// Matrices in the order of Shape2: `groups` of one shape, `classes` of one m. A
// class keeps three stacks of m x m matrices, a group two stacks of its shape.
struct Batch {
  struct Group {
    Shape2 s;
    int64_t ldx, first, count, x_off[2], cls, first_in_class;
    int64_t x_elems() const { return s.rows * ldx; }
  };
  struct Class {
    int64_t m, lds, count, s_off[3];
  };
  std::vector<Group> groups;
  std::vector<Class> classes;
  int64_t part_off = 0, bytes = 0;

  static int64_t ld(int64_t n) { return ops_round_up(n, 64); }
  static int64_t item_bytes(const Shape2& s) {  // upper bound of what one more matrix adds, tall or wide
    return 2 * std::max(s.rows * ld(s.cols), s.cols * ld(s.rows)) * 2 + 3 * s.m() * ld(s.m()) * 2 + kNormBlocks * 8 + 8 * 256;
  }

  void build(const Shape2* shapes, int64_t count) {
    groups.clear();
    classes.clear();
    int64_t at = 0;
    part_off = at;
    at += ops_round_up(count * kNormBlocks * 8, 256);
    for (int64_t i = 0; i < count; ++i) {
      const int64_t m = shapes[i].m();
      if (classes.empty() || classes.back().m != m) classes.push_back({m, ld(m), 0, {0, 0, 0}});
      if (groups.empty() || !(groups.back().s == shapes[i]))
        groups.push_back({shapes[i], ld(shapes[i].cols), i, 0, {0, 0}, (int64_t)classes.size() - 1, classes.back().count});
      groups.back().count++;
      classes.back().count++;
    }
    for (Group& g : groups)
      for (int k = 0; k < 2; ++k) {
        g.x_off[k] = at;
        at += ops_round_up(g.count * g.x_elems() * 2, 256);
      }
    for (Class& c : classes)
      for (int k = 0; k < 3; ++k) {
        c.s_off[k] = at;
        at += ops_round_up(c.count * c.m * c.lds * 2, 256);
      }
    bytes = at;
  }
};

struct Runner {
  const Batch& b;
  char* ws;
  cudaStream_t stream;
  std::vector<GemmProblem> pending;

  cudaError_t flush(GemmKind kind) {
    for (size_t i = 0; i < pending.size(); i += kGemmMaxProblems) {
      const int n = static_cast<int>(std::min<size_t>(kGemmMaxProblems, pending.size() - i));
      const cudaError_t err = launch_gemm(kind, pending.data() + i, n, stream);
      if (err != cudaSuccess) return err;
    }
    pending.clear();
    return cudaSuccess;
  }

  // Matrices first .. first + count of a group; `transposed` as in GemmOperand.
  GemmOperand x_operand(const Batch::Group& g, int k, int64_t first, int64_t count, bool transposed) const {
    return {ws + g.x_off[k] + first * g.x_elems() * 2, g.s.cols, g.s.rows, g.ldx, transposed, count, g.x_elems()};
  }
  GemmOperand s_operand(const Batch::Class& c, int k, int64_t first, int64_t count) const {
    return {ws + c.s_off[k] + first * c.m * c.lds * 2, c.m, c.m, c.lds, false, count, c.m * c.lds};
  }
  static StoreParams s_store(const Batch::Class& c, void* out, const void* cc, float alpha, float beta, float diag) {
    return {out, cc, c.lds, c.m * c.lds, alpha, beta, diag, 0, 16};
  }

  // A = X X^T (or X^T X) into stack 0
  cudaError_t gram(int x) {
    // the longest sums first: the short tiles then even out the pairs' ends
    for (size_t i = b.groups.size(); i-- > 0;) {
      const Batch::Group& g = b.groups[i];
      const Batch::Class& c = b.classes[(size_t)g.cls];
      GemmProblem p;
      p.a = p.b = x_operand(g, x, 0, g.count, g.s.rows > g.s.cols);
      p.m = p.n = c.m;
      p.k = g.s.n();
      p.batch = g.count;
      p.symmetric = true;
      p.store = s_store(c, ws + c.s_off[0] + g.first_in_class * c.m * c.lds * 2, nullptr, kScaleA / (kScaleX * kScaleX),
                        0.0f, 0.0f);
      pending.push_back(p);
    }
    return flush(GEMM_F16);
  }
  // out = alpha s1 s2 + beta s3 + diag I, all symmetric and commuting
  cudaError_t product(int out, int s1, int s2, float alpha, int s3 = -1, float beta = 0.0f, float diag = 0.0f) {
    for (size_t i = b.classes.size(); i-- > 0;) {
      const Batch::Class& c = b.classes[i];
      GemmProblem p;
      p.a = s_operand(c, s1, 0, c.count);
      p.b = s_operand(c, s2, 0, c.count);
      p.m = p.n = p.k = c.m;
      p.batch = c.count;
      p.symmetric = true;
      p.store = s_store(c, ws + c.s_off[out], s3 < 0 ? nullptr : ws + c.s_off[s3], alpha, beta, diag);
      pending.push_back(p);
    }
    return flush(GEMM_F16);
  }
  // stack `out` = Q of the Gram matrices in stack `a`
  cudaError_t polynomial(int out, int a) {
    return product(out, a, a, kNsC * kScaleQ / (kScaleA * kScaleA), a, kNsB * kScaleQ / kScaleA, kNsA * kScaleQ);
  }
  // S X (or X S) of matrices first .. first + count of a group, without a destination.
  GemmProblem applied(const Batch::Group& g, int s, int x, int64_t first, int64_t count) const {
    const Batch::Class& c = b.classes[(size_t)g.cls];
    const bool tall = g.s.rows > g.s.cols;
    GemmProblem p;
    p.a = tall ? x_operand(g, x, first, count, false) : s_operand(c, s, g.first_in_class + first, count);
    p.b = tall ? s_operand(c, s, g.first_in_class + first, count) : x_operand(g, x, first, count, true);
    p.m = g.s.rows;
    p.n = g.s.cols;
    p.k = c.m;
    p.batch = count;
    return p;
  }
  // X_out = S X_in, S in stack s stored times `scale`
  cudaError_t apply(int s, float scale, int x_in, int x_out) {
    for (size_t i = b.groups.size(); i-- > 0;) {
      const Batch::Group& g = b.groups[i];
      pending.push_back(applied(g, s, x_in, 0, g.count));
      pending.back().store = {ws + g.x_off[x_out], nullptr, g.ldx, g.x_elems(), 1.0f / scale, 0.0f, 0.0f, 0, 16};
    }
    return flush(GEMM_F16);
  }

  // `steps` steps from X in buffer 0, as single steps or as 2 + 1 + 2 + 1 + ...
  // The last product is left to the caller: *s, *scale, *x say which stack
  // times which X it is.
  cudaError_t iterate(int steps, bool pairs, int* s, float* scale, int* x) {
    int at = 0;
    bool pair = pairs;
    for (int done = 0;;) {
      const int now = pair && steps - done >= 2 ? 2 : 1;
      cudaError_t err;
      if ((err = gram(at)) != cudaSuccess) return err;
      if (now == 2 && b.classes.back().m <= kNsChain) {  // the largest m
        for (const Batch::Class& c : b.classes)
          if ((err = ns_chain(reinterpret_cast<__half*>(ws + c.s_off[0]), c.m, c.lds, c.m * c.lds, c.count, stream)) != cudaSuccess)
            return err;
        *s = 0;
        *scale = kScaleR;
      } else if ((err = polynomial(1, 0)) != cudaSuccess) {
        return err;
      } else if (now == 1) {
        *s = 1;
        *scale = kScaleQ;
      } else {
        if ((err = product(2, 1, 0, kScaleQA / (kScaleQ * kScaleA))) != cudaSuccess) return err;   // Q A
        if ((err = product(0, 2, 1, kScaleA / (kScaleQA * kScaleQ))) != cudaSuccess) return err;   // A' = (Q A) Q
        if ((err = polynomial(2, 0)) != cudaSuccess) return err;                                   // Q'
        if ((err = product(0, 2, 1, kScaleR / (kScaleQ * kScaleQ))) != cudaSuccess) return err;    // Q' Q
        *s = 0;
        *scale = kScaleR;
      }
      done += now;
      if (pairs) pair = !pair;
      *x = at;
      if (done == steps) return cudaSuccess;
      if ((err = apply(*s, *scale, at, at ^ 1)) != cudaSuccess) return err;
      at ^= 1;
    }
  }
};

// Whether carrying the Gram matrix over two steps costs fewer operations (see
// the counts above) for these matrices.
bool use_pairs(const Shape2* s, int64_t count) {
  double single = 0, paired = 0;
  for (int64_t i = 0; i < count; ++i) {
    const double m = (double)s[i].m(), n = (double)s[i].n();
    single += 15 * m * m * n + 5 * m * m * m;
    paired += 9 * m * m * n + 11 * m * m * m;
  }
  return paired < single;
}

// Norms and X_0 of a batch's items, a few at a time (kIngestBytes).
cudaError_t ingest(const std::vector<Item>& items, bool f32, bool mom, const NsMomentum& s, cudaStream_t stream) {
  const int64_t size = (f32 ? 4 : 2) + (mom ? 4 : 0);
  for (size_t i = 0; i < items.size();) {
    ItemTable t;
    int n = 0;
    int64_t bytes = 0, largest = 0;
    while (n < kItemsPerLaunch && i < items.size()) {
      const int64_t z = items[i].rows * items[i].cols;
      if (n > 0 && bytes + z * size > kIngestBytes) break;
      bytes += z * size;
      largest = std::max(largest, z);
      t.it[n++] = items[i++];
    }
    // 8 elements a thread, twice, until the grid is large enough to walk on
    const int parts = static_cast<int>(std::min<int64_t>(kNormBlocks, ops_ceil_div(largest, 4096)));
    const dim3 g1(parts, n), g2(static_cast<unsigned>(std::min<int64_t>(1024, ops_ceil_div(largest, 4096))), n);
    auto norm = f32 ? (mom ? norm_kernel<true, true> : norm_kernel<true, false>)
                    : (mom ? norm_kernel<false, true> : norm_kernel<false, false>);
    auto scale = f32 ? (mom ? scale_kernel<true, true> : scale_kernel<true, false>)
                     : (mom ? scale_kernel<false, true> : scale_kernel<false, false>);
    cudaError_t err = launch_chained(norm, g1, dim3(256), 0, stream, t, s);
    if (err == cudaSuccess) err = launch_chained(scale, g2, dim3(256), 0, stream, t, s, parts);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

// No device holds a matrix of more elements; sizes up to here stay within 64 bits.
constexpr int64_t kMaxElems = int64_t(1) << 40;
// A workspace for all matrices at once, or for as many as 4 GiB hold, at least one.
constexpr int64_t kMaxBatchBytes = int64_t(4) << 30;

}  // namespace
}  // namespace lst

using namespace lst;

extern "C" int64_t lst_orthogonalize_workspace_bytes(int32_t count, int64_t rows, int64_t cols) {
  if (count <= 0 || rows <= 0 || cols <= 0 || rows > INT32_MAX || cols > INT32_MAX || rows > kMaxElems / cols) return 0;
  const Shape2 s = {rows, cols};
  const int64_t fit = std::max<int64_t>(1, kMaxBatchBytes / Batch::item_bytes(s));
  return std::min<int64_t>(count, fit) * Batch::item_bytes(s);
}

extern "C" lst_status lst_orthogonalize(int32_t count, const lst_matrix* in, const lst_matrix* out,
                                        const lst_ns_params* params, void* workspace, int64_t workspace_bytes,
                                        void* cuda_stream) {
  clear_error();
  const char* who = "lst_orthogonalize";
  if (count < 0) return fail(LST_ERR_INVALID_ARG, "%s: count < 0", who);
  if (!params) return fail(LST_ERR_INVALID_ARG, "%s: params is null", who);
  if (params->steps < 1 || params->steps > 20 || !(params->eps > 0.0f) || !std::isfinite(params->eps))
    return fail(LST_ERR_INVALID_ARG, "%s: steps outside 1..20 or eps not positive", who);
  if (count == 0) return LST_OK;
  if (!in || !out) return fail(LST_ERR_INVALID_ARG, "%s: in or out is null", who);
  for (int32_t i = 0; i < count; ++i) {
    LST_TRY(check_matrix(in + i, "in", who));
    LST_TRY(check_matrix(out + i, "out", who));
    if (in[i].rows != in[0].rows || in[i].cols != in[0].cols || in[i].dtype != in[0].dtype ||
        out[i].rows != in[0].rows || out[i].cols != in[0].cols)
      return fail(LST_ERR_INVALID_ARG, "%s: matrix %d differs in shape or type from the first", who, (int)i);
    if (out[i].dtype != LST_BF16) return fail(LST_ERR_INVALID_ARG, "%s: out must be bf16", who);
  }
  if (in[0].rows == 0 || in[0].cols == 0) return LST_OK;
  const Shape2 shape = {in[0].rows, in[0].cols};
  if (shape.rows > kMaxElems / shape.cols) return fail(LST_ERR_INVALID_ARG, "%s: matrix of more than 2^40 elements", who);
  LST_TRY(check_workspace(workspace, workspace_bytes, Batch::item_bytes(shape), who));
  if (ns_small_fits(shape.rows, shape.cols)) {
    const NsSmallCall call = {shape.rows, shape.cols, in[0].dtype == LST_F32, -1, params->steps, 1.0f, {0.0f, params->eps, 0}};
    NsSmallItem items[kNsSmallItems];
    for (int32_t first = 0; first < count; first += kNsSmallItems) {
      const int now = std::min(kNsSmallItems, count - first);
      for (int i = 0; i < now; ++i)
        items[i] = {in[first + i].data, nullptr, out[first + i].data, nullptr, in[first + i].stride, out[first + i].stride, 0.0f};
      LST_TRY_CUDA(ns_small(items, now, call, static_cast<cudaStream_t>(cuda_stream)), who);
    }
    return LST_OK;
  }
  const int64_t fit = workspace_bytes / Batch::item_bytes(shape);
  const NsMomentum s = {0.0f, params->eps, 0};
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  char* ws = static_cast<char*>(workspace);
  try {
    for (int64_t first = 0; first < count; first += fit) {
      const int64_t n = std::min<int64_t>(fit, count - first);
      std::vector<Shape2> shapes((size_t)n, shape);
      Batch b;
      b.build(shapes.data(), n);
      const Batch::Group& g = b.groups[0];
      std::vector<Item> items((size_t)n);
      for (int64_t i = 0; i < n; ++i) {
        const lst_matrix& src = in[first + i];
        Item& it = items[(size_t)i];
        it = {};
        it.g = src.data;
        it.rows = src.rows;
        it.cols = src.cols;
        it.ld = src.stride;
        it.x = reinterpret_cast<__half*>(ws + g.x_off[0]) + i * g.x_elems();
        it.ldx = g.ldx;
        it.part = reinterpret_cast<float2*>(ws + b.part_off) + i * kNormBlocks;
      }
      LST_TRY_CUDA(ingest(items, in[0].dtype == LST_F32, false, s, stream), who);
      Runner run{b, ws, stream, {}};
      int si, xi;
      float scale;
      LST_TRY_CUDA(run.iterate(params->steps, use_pairs(shapes.data(), n), &si, &scale, &xi), who);
      // the last product goes to the caller's matrices
      for (int64_t i = 0; i < n; ++i) {
        const lst_matrix& dst = out[first + i];
        const uintptr_t align = reinterpret_cast<uintptr_t>(dst.data) | static_cast<uintptr_t>(dst.stride * 2);
        const int vec = align % 16 == 0 ? 16 : 2;
        run.pending.push_back(run.applied(g, si, xi, i, 1));
        run.pending.back().store = {dst.data, nullptr, dst.stride, 0, 1.0f / (scale * kScaleX), 0.0f, 0.0f, 1, vec};
      }
      LST_TRY_CUDA(run.flush(GEMM_F16), who);
    }
  } catch (...) {
    return fail(LST_ERR_OOM, "%s: out of host memory", who);
  }
  return LST_OK;
}

extern "C" int64_t lst_muon_workspace_bytes(const lst_layout* L) {
  if (!L) return 0;
  int64_t all = 0, largest = 0;
  for (const Tensor& t : L->tensors) {
    if (t.ndim != 2 || t.numel == 0) continue;
    const int64_t z = Batch::item_bytes({t.dims[0], t.dims[1]});
    all += z;
    largest = std::max(largest, z);
  }
  return std::min(all, std::max(largest, kMaxBatchBytes));
}

extern "C" lst_status lst_muon_step(const lst_layout* L, void* const* dev_blocks, const lst_muon_hparams* hp,
                                    const lst_adamw_hparams* adamw, const uint8_t* use_muon, void* workspace,
                                    int64_t workspace_bytes, void* cuda_stream) {
  clear_error();
  const char* who = "lst_muon_step";
  if (!L) return fail(LST_ERR_INVALID_ARG, "%s: null layout", who);
  if (!hp) return fail(LST_ERR_INVALID_ARG, "%s: null muon hparams", who);
  if (!std::isfinite(hp->lr) || !std::isfinite(hp->weight_decay) || !(hp->momentum >= 0.0f && hp->momentum < 1.0f) ||
      !(hp->rms_scale >= 0.0f) || !std::isfinite(hp->rms_scale) || !(hp->eps > 0.0f) || !std::isfinite(hp->eps) ||
      hp->ns_steps < 1 || hp->ns_steps > 20)
    return fail(LST_ERR_INVALID_ARG, "%s: muon hyperparameters outside their domain", who);
  Scalars as{};
  if (adamw && !make_scalars(*adamw, &as))
    return fail(LST_ERR_INVALID_ARG,
                "%s: hyperparameters outside their domain (step >= 1, 0 <= beta < 1, finite)", who);
  const int64_t nt = (int64_t)L->tensors.size();
  if (L->blocks.empty()) return LST_OK;
  if (!dev_blocks) return fail(LST_ERR_INVALID_ARG, "%s: dev_blocks is null", who);
  for (size_t i = 0; i < L->blocks.size(); ++i) {
    if (L->blocks[i].bytes == 0) continue;
    if (!dev_blocks[i]) return fail(LST_ERR_INVALID_ARG, "%s: block %lld pointer is null", who, (long long)i);
    if (reinterpret_cast<uintptr_t>(dev_blocks[i]) % 16 != 0)
      return fail(LST_ERR_ALIGNMENT, "%s: block %lld pointer not 16-byte aligned", who, (long long)i);
  }
  try {
    struct Pick {
      Shape2 s;
      int64_t tensor;
    };
    std::vector<Pick> picks;
    std::vector<AdamItem> adam;
    int64_t largest = 0;
    auto run_of = [&](const Tensor& t) {
      const Block& b = L->blocks[(size_t)t.layer];
      return block_run(*L, b, static_cast<char*>(dev_blocks[t.layer]), t.elem_off, t.elem_off + t.numel);
    };
    for (int64_t i = 0; i < nt; ++i) {
      const Tensor& t = L->tensors[(size_t)i];
      const bool matrix = t.ndim == 2;
      if (use_muon && use_muon[i] && !matrix)
        return fail(LST_ERR_INVALID_ARG, "%s: tensor %lld is not a matrix", who, (long long)i);
      if (t.numel == 0) continue;
      if (use_muon ? use_muon[i] != 0 : matrix) {
        if (t.dims[0] > INT32_MAX || t.dims[1] > INT32_MAX)
          return fail(LST_ERR_INVALID_ARG, "%s: tensor %lld: dimension above 2^31-1", who, (long long)i);
        picks.push_back({{t.dims[0], t.dims[1]}, i});
        largest = std::max(largest, Batch::item_bytes(picks.back().s));
      } else if (adamw) {
        const Run r = run_of(t);
        adam.push_back({r.g, r.w, r.m, r.v, static_cast<uint16_t*>(r.w16), t.numel});
      }
    }
    LST_TRY(check_workspace(workspace, workspace_bytes, largest, who));
    std::stable_sort(picks.begin(), picks.end(), [](const Pick& a, const Pick& b) { return a.s < b.s; });
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    char* ws = static_cast<char*>(workspace);
    const NsMomentum ms = {hp->momentum, hp->eps, hp->nesterov ? 1 : 0};
    const float decay = (float)(1.0 - (double)hp->lr * (double)hp->weight_decay);
    const bool f32 = L->fmt == LST_L16_FP32;

    auto step_of = [&](const Shape2& z) {
      const double rows = (double)z.rows, cols = (double)z.cols;
      return (double)hp->lr * (hp->rms_scale > 0.0f ? (double)hp->rms_scale * std::sqrt(std::max(rows, cols))
                                                    : std::sqrt(std::max(1.0, rows / cols)));
    };
    // small matrices: one kernel for those of a shape
    std::vector<Pick> large;
    std::vector<NsSmallItem> small;
    for (size_t i = 0; i < picks.size(); ++i) {
      const Shape2& z = picks[i].s;
      if (!ns_small_fits(z.rows, z.cols)) {
        large.push_back(picks[i]);
        continue;
      }
      const Run r = run_of(L->tensors[(size_t)picks[i].tensor]);
      small.push_back({r.g, r.m, r.w, static_cast<uint16_t*>(r.w16), z.cols, z.cols, (float)step_of(z)});
      if (i + 1 == picks.size() || !(picks[i + 1].s == z)) {
        const NsSmallCall call = {z.rows, z.cols, f32, L->fmt, hp->ns_steps, decay, ms};
        LST_TRY_CUDA(ns_small(small.data(), (int)small.size(), call, stream), who);
        small.clear();
      }
    }
    picks.swap(large);

    for (size_t first = 0; first < picks.size();) {
      std::vector<Shape2> shapes;
      int64_t used = 0;
      size_t last = first;
      while (last < picks.size() && used + Batch::item_bytes(picks[last].s) <= workspace_bytes) {
        used += Batch::item_bytes(picks[last].s);
        shapes.push_back(picks[last].s);
        ++last;
      }
      Batch b;
      b.build(shapes.data(), (int64_t)shapes.size());
      std::vector<Item> items(shapes.size());
      for (const Batch::Group& g : b.groups)
        for (int64_t k = 0; k < g.count; ++k) {
          const Run r = run_of(L->tensors[(size_t)picks[first + (size_t)(g.first + k)].tensor]);
          items[(size_t)(g.first + k)] = {r.g, r.m, reinterpret_cast<__half*>(ws + g.x_off[0]) + k * g.x_elems(),
                                          reinterpret_cast<float2*>(ws + b.part_off) + (g.first + k) * kNormBlocks,
                                          g.s.rows, g.s.cols, g.s.cols, g.ldx};
        }
      LST_TRY_CUDA(ingest(items, f32, true, ms, stream), who);
      Runner run{b, ws, stream, {}};
      int si, xi;
      float scale;
      LST_TRY_CUDA(run.iterate(hp->ns_steps, use_pairs(shapes.data(), (int64_t)shapes.size()), &si, &scale, &xi), who);
      // the last product updates the weights
      UpdateTable table;
      int entries = 0;
      auto flush = [&]() {
        const cudaError_t err = launch_gemm(GEMM_F16_UPDATE, run.pending.data(), (int)run.pending.size(), stream, &table);
        run.pending.clear();
        entries = 0;
        return err;
      };
      for (size_t i = b.groups.size(); i-- > 0;) {
        const Batch::Group& g = b.groups[i];
        for (int64_t k = 0; k < g.count;) {
          if (entries == kGemmMaxUpdates || run.pending.size() == kGemmMaxProblems) LST_TRY_CUDA(flush(), who);
          const int64_t now = std::min<int64_t>(g.count - k, kGemmMaxUpdates - entries);
          run.pending.push_back(run.applied(g, si, xi, k, now));
          // tensors start at multiples of 8 elements: rows of such a length are on 16 bytes in every field
          run.pending.back().update = {g.s.cols, entries, L->fmt, g.s.cols % 8 == 0 ? 16 : 2, decay};
          for (int64_t j = 0; j < now; ++j, ++entries) {
            const Run r = run_of(L->tensors[(size_t)picks[first + (size_t)(g.first + k + j)].tensor]);
            table.w[entries] = r.w;
            table.w16[entries] = static_cast<uint16_t*>(r.w16);
            table.step[entries] = (float)(step_of(g.s) / ((double)kScaleX * (double)scale));
          }
          k += now;
        }
      }
      LST_TRY_CUDA(flush(), who);
      first = last;
    }
    for (size_t i = 0; i < adam.size(); i += kItemsPerLaunch) {
      AdamTable t;
      const int n = static_cast<int>(std::min<size_t>(kItemsPerLaunch, adam.size() - i));
      int64_t big = 0;
      for (int k = 0; k < n; ++k) {
        t.it[k] = adam[i + (size_t)k];
        big = std::max(big, t.it[k].n);
      }
      const dim3 grid(static_cast<unsigned>(std::min<int64_t>(4096, ops_ceil_div(big, 1024))), n);
      auto kernel = L->fmt == LST_L12_BF16    ? adam_kernel<F_L12>
                    : L->fmt == LST_L16_MIXED ? adam_kernel<F_L16M>
                                              : adam_kernel<F_L16F>;
      LST_TRY_CUDA(launch_chained(kernel, grid, dim3(256), 0, stream, t, as), who);
    }
  } catch (...) {
    return fail(LST_ERR_OOM, "%s: out of host memory", who);
  }
  return LST_OK;
}

extern "C" lst_status lst_operator_status(void) {
  clear_error();
  int err = 0;
  LST_TRY_CUDA(cudaDeviceSynchronize(), "lst_operator_status");
  LST_TRY_CUDA(gemm_take_error(&err), "lst_operator_status");
  int small = 0;
  LST_TRY_CUDA(ns_small_take_error(&small), "lst_operator_status");
  if (err || small) return fail(LST_ERR_TIMEOUT, "a wait inside a matrix kernel ran out");
  return LST_OK;
}
