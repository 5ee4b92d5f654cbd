// Newton-Schulz orthogonalisation and the Muon step over packed blocks.
//
// Mathematics. With X_0 = U / (|U|_F + eps) (transposed so that m <= n) a step
// is X <- Q X, Q = a I + b A + c A^2, A = X X^T. All Q and A are polynomials of
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
#include "lst_ops.h"

namespace lst {

namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
// power-of-two scales of the stored fp16 values
constexpr float kScaleX = 16384.0f, kScaleA = 16384.0f, kScaleQ = 8192.0f, kScaleQA = 16384.0f, kScaleR = 4096.0f;

constexpr int kItemsPerLaunch = 32;
constexpr int kNormBlocks = 512;   // partial sums per matrix
constexpr int kTile = 64;

// One matrix on its way in (u = its values) and out (its orthogonalised form).
struct Item {
  const void* g;      // gradient, or the matrix itself
  float* mom;         // momentum, or null
  void* w;            // weight to update, or null
  uint16_t* w16;      // derived bf16 weight, or null
  __half* x;          // m x ldx values
  const __half* o;    // result
  double* part;       // kNormBlocks partial sums of squares
  int64_t rows, cols, ld, ldx;
  int32_t tall;       // rows > cols: x is the transpose
  float step;         // lr * update scale / kScaleX
};
struct ItemTable {
  Item it[kItemsPerLaunch];
};
struct MuonScalars {
  float momentum, decay, eps;
  int32_t nesterov;
};

__device__ __forceinline__ float load_in(const void* p, int64_t i, bool f32) {
  return f32 ? static_cast<const float*>(p)[i]
             : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}

// u of one element; `m` is the momentum already updated.
__device__ __forceinline__ float muon_u(float g, float m, const MuonScalars& s) {
  return s.nesterov ? __fadd_rn(g, __fmul_rn(s.momentum, m)) : m;
}

// m = momentum m + g in place, and the sum of u^2 (in fp32 over a thread's
// elements of one stride, in fp64 above that). Bound by memory: reads g and m,
// writes m.
template <bool F32, bool MOM>
__global__ void __launch_bounds__(256) norm_kernel(const __grid_constant__ ItemTable t, MuonScalars s) {
  const Item& it = t.it[blockIdx.y];
  double sum = 0.0;
  const bool flat = it.ld == it.cols && (reinterpret_cast<uintptr_t>(it.g) & 15) == 0 &&
                    (!MOM || (reinterpret_cast<uintptr_t>(it.mom) & 15) == 0);
  const int64_t total = it.rows * it.cols;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  int64_t tail = 0;
  if (flat) {
    const int64_t quads = total / 4;
    tail = quads * 4;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < quads; q += stride) {
      float g[4], u[4];
      if (F32) {
        const float4 x = static_cast<const float4*>(it.g)[q];
        g[0] = x.x, g[1] = x.y, g[2] = x.z, g[3] = x.w;
      } else {
        const uint2 x = static_cast<const uint2*>(it.g)[q];
        g[0] = bf16_lo(x.x), g[1] = bf16_hi(x.x), g[2] = bf16_lo(x.y), g[3] = bf16_hi(x.y);
      }
      if (MOM) {
        float4 m = reinterpret_cast<float4*>(it.mom)[q];
        m.x = __fadd_rn(__fmul_rn(s.momentum, m.x), g[0]);
        m.y = __fadd_rn(__fmul_rn(s.momentum, m.y), g[1]);
        m.z = __fadd_rn(__fmul_rn(s.momentum, m.z), g[2]);
        m.w = __fadd_rn(__fmul_rn(s.momentum, m.w), g[3]);
        reinterpret_cast<float4*>(it.mom)[q] = m;
        u[0] = muon_u(g[0], m.x, s), u[1] = muon_u(g[1], m.y, s);
        u[2] = muon_u(g[2], m.z, s), u[3] = muon_u(g[3], m.w, s);
      } else {
        u[0] = g[0], u[1] = g[1], u[2] = g[2], u[3] = g[3];
      }
      sum += static_cast<double>((u[0] * u[0] + u[1] * u[1]) + (u[2] * u[2] + u[3] * u[3]));
    }
  }
  for (int64_t i = tail + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += stride) {
    const int64_t at = it.ld == it.cols ? i : i / it.cols * it.ld + i % it.cols;
    float u = load_in(it.g, at, F32);
    if (MOM) {
      const float m = __fadd_rn(__fmul_rn(s.momentum, it.mom[i]), u);
      it.mom[i] = m;
      u = muon_u(u, m, s);
    }
    sum += static_cast<double>(u * u);
  }
  __shared__ double red[8];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_down_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double x = red[0];
    for (int i = 1; i < 8; ++i) x += red[i];
    it.part[blockIdx.x] = x;
  }
}

// X_0 = u / (|u|_F + eps), in fp16 times kScaleX, transposed where rows > cols.
template <bool F32, bool MOM>
__global__ void __launch_bounds__(256) scale_kernel(const __grid_constant__ ItemTable t, MuonScalars s, int parts) {
  const Item& it = t.it[blockIdx.y];
  const int64_t tiles_c = (it.cols + kTile - 1) / kTile, tiles = (it.rows + kTile - 1) / kTile * tiles_c;
  if (blockIdx.x >= tiles) return;
  __shared__ double red[8];
  __shared__ __half tile[kTile][kTile + 2];
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += 256) sum += it.part[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_down_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  sum = red[0];
  for (int i = 1; i < 8; ++i) sum += red[i];
  const float inv = static_cast<float>(static_cast<double>(kScaleX) / (sqrt(sum) + static_cast<double>(s.eps)));
  const int c = threadIdx.x & 63, r4 = threadIdx.x >> 6;
  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    const int64_t r0 = b / tiles_c * kTile, c0 = b % tiles_c * kTile;
#pragma unroll 4
    for (int k = 0; k < kTile / 4; ++k) {
      const int r = r4 + 4 * k;
      if (r0 + r >= it.rows || c0 + c >= it.cols) continue;
      float u = load_in(it.g, (r0 + r) * it.ld + c0 + c, F32);
      if (MOM) u = muon_u(u, it.mom[(r0 + r) * it.cols + c0 + c], s);
      const __half h = __float2half_rn(u * inv);
      if (it.tall)
        tile[r][c] = h;
      else
        it.x[(r0 + r) * it.ldx + c0 + c] = h;
    }
    if (it.tall) {
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kTile / 4; ++k) {
        const int col = r4 + 4 * k;  // column of the source
        if (c0 + col < it.cols && r0 + c < it.rows) it.x[(c0 + col) * it.ldx + r0 + c] = tile[c][col];
      }
      __syncthreads();
    }
  }
}

// w = w decay - step O (and the derived bf16 W). FMT as in lst_device.cuh.
template <int FMT>
__global__ void __launch_bounds__(256) apply_kernel(const __grid_constant__ ItemTable t, MuonScalars s) {
  const Item& it = t.it[blockIdx.y];
  const int64_t tiles_c = (it.cols + kTile - 1) / kTile, tiles = (it.rows + kTile - 1) / kTile * tiles_c;
  __shared__ __half tile[kTile][kTile + 2];
  const int c = threadIdx.x & 63, r4 = threadIdx.x >> 6;
  for (int64_t b = blockIdx.x; b < tiles; b += gridDim.x) {
    const int64_t r0 = b / tiles_c * kTile, c0 = b % tiles_c * kTile;
    if (it.tall) {
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kTile / 4; ++k) {
        const int col = r4 + 4 * k;
        if (c0 + col < it.cols && r0 + c < it.rows) tile[c][col] = it.o[(c0 + col) * it.ldx + r0 + c];
      }
      __syncthreads();
    }
#pragma unroll 4
    for (int k = 0; k < kTile / 4; ++k) {
      const int r = r4 + 4 * k;
      if (r0 + r >= it.rows || c0 + c >= it.cols) continue;
      const float o = __half2float(it.tall ? tile[r][c] : it.o[(r0 + r) * it.ldx + c0 + c]);
      const int64_t i = (r0 + r) * it.cols + c0 + c;
      float w = FMT == F_L12 ? bf16_lo(static_cast<uint16_t*>(it.w)[i]) : static_cast<float*>(it.w)[i];
      w = __fsub_rn(__fmul_rn(w, s.decay), __fmul_rn(it.step, o));
      if (FMT == F_L12) {
        static_cast<__nv_bfloat16*>(it.w)[i] = __float2bfloat16_rn(w);
      } else {
        static_cast<float*>(it.w)[i] = w;
        if (FMT == F_L16M) reinterpret_cast<__nv_bfloat16*>(it.w16)[i] = __float2bfloat16_rn(w);
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
  int64_t m, n;  // m <= n
};

// Matrices sorted by (m, n): `groups` of one shape, `classes` of one m. A class
// keeps three stacks of m x m matrices, a group two stacks of m x n.
struct Batch {
  struct Group {
    int64_t m, n, ldx, first, count, x_off[2], cls, first_in_class;
  };
  struct Class {
    int64_t m, lds, count, s_off[3];
  };
  std::vector<Group> groups;
  std::vector<Class> classes;
  int64_t part_off = 0, bytes = 0;

  static int64_t ld(int64_t n) { return ops_round_up(n, 64); }
  static int64_t item_bytes(const Shape2& s) {  // upper bound of what one more matrix adds
    return 2 * s.m * ld(s.n) * 2 + 3 * s.m * ld(s.m) * 2 + kNormBlocks * 8 + 8 * 256;
  }

  void build(const Shape2* shapes, int64_t count) {
    groups.clear();
    classes.clear();
    int64_t at = 0;
    part_off = at;
    at += ops_round_up(count * kNormBlocks * 8, 256);
    for (int64_t i = 0; i < count; ++i) {
      if (classes.empty() || classes.back().m != shapes[i].m) classes.push_back({shapes[i].m, ld(shapes[i].m), 0, {0, 0, 0}});
      if (groups.empty() || groups.back().m != shapes[i].m || groups.back().n != shapes[i].n)
        groups.push_back({shapes[i].m, shapes[i].n, ld(shapes[i].n), i, 0, {0, 0}, (int64_t)classes.size() - 1,
                          classes.back().count});
      groups.back().count++;
      classes.back().count++;
    }
    for (Group& g : groups)
      for (int k = 0; k < 2; ++k) {
        g.x_off[k] = at;
        at += ops_round_up(g.count * g.m * g.ldx * 2, 256);
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

  GemmOperand x_operand(const Batch::Group& g, int k) const {
    return {ws + g.x_off[k], g.n, g.m, g.ldx, g.count, g.m * g.ldx};
  }
  GemmOperand s_operand(const Batch::Class& c, int k, int64_t first, int64_t count) const {
    return {ws + c.s_off[k] + first * c.m * c.lds * 2, c.m, c.m, c.lds, count, c.m * c.lds};
  }
  static StoreParams s_store(const Batch::Class& c, void* out, const void* cc, float alpha, float beta, float diag) {
    return {out, cc, c.lds, c.m * c.lds, alpha, beta, diag, 0, 0, 32};
  }

  // A = X X^T into stack 0
  cudaError_t gram(int x) {
    for (const Batch::Group& g : b.groups) {
      const Batch::Class& c = b.classes[(size_t)g.cls];
      GemmProblem p;
      p.a = p.b = x_operand(g, x);
      p.m = p.n = g.m;
      p.k = g.n;
      p.batch = g.count;
      p.symmetric = true;
      p.store = s_store(c, ws + c.s_off[0] + g.first_in_class * c.m * c.lds * 2, nullptr, kScaleA / (kScaleX * kScaleX),
                        0.0f, 0.0f);
      pending.push_back(p);
    }
    return flush(GEMM_NS_SYM);
  }
  // out = alpha s1 s2 + beta s3 + diag I, all symmetric and commuting
  cudaError_t product(int out, int s1, int s2, float alpha, int s3 = -1, float beta = 0.0f, float diag = 0.0f) {
    for (const Batch::Class& c : b.classes) {
      GemmProblem p;
      p.a = s_operand(c, s1, 0, c.count);
      p.b = s_operand(c, s2, 0, c.count);
      p.m = p.n = p.k = c.m;
      p.batch = c.count;
      p.symmetric = true;
      p.store = s_store(c, ws + c.s_off[out], s3 < 0 ? nullptr : ws + c.s_off[s3], alpha, beta, diag);
      pending.push_back(p);
    }
    return flush(GEMM_NS_SYM);
  }
  // stack `out` = Q of the Gram matrices in stack `a`
  cudaError_t polynomial(int out, int a) {
    return product(out, a, a, kC * kScaleQ / (kScaleA * kScaleA), a, kB * kScaleQ / kScaleA, kA * kScaleQ);
  }
  // X_out = S X_in, S in stack s stored times `scale`
  cudaError_t apply(int s, float scale, int x_in, int x_out) {
    for (const Batch::Group& g : b.groups) {
      const Batch::Class& c = b.classes[(size_t)g.cls];
      GemmProblem p;
      p.a = s_operand(c, s, g.first_in_class, g.count);
      p.b = x_operand(g, x_in);
      p.m = g.m;
      p.n = g.n;
      p.k = g.m;
      p.batch = g.count;
      p.store = {ws + g.x_off[x_out], nullptr, g.ldx, g.m * g.ldx, 1.0f / scale, 0.0f, 0.0f, 0, 0, 32};
      pending.push_back(p);
    }
    return flush(GEMM_NS_APPLY);
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
      if ((err = polynomial(1, 0)) != cudaSuccess) return err;
      *s = 1;
      *scale = kScaleQ;
      if (now == 2) {
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
    const double m = (double)s[i].m, n = (double)s[i].n;
    single += 15 * m * m * n + 5 * m * m * m;
    paired += 9 * m * m * n + 11 * m * m * m;
  }
  return paired < single;
}

template <class F>
cudaError_t for_items(const std::vector<Item>& items, F launch) {
  for (size_t i = 0; i < items.size(); i += kItemsPerLaunch) {
    ItemTable t;
    const int n = static_cast<int>(std::min<size_t>(kItemsPerLaunch, items.size() - i));
    int64_t largest = 0;
    for (int k = 0; k < n; ++k) {
      t.it[k] = items[i + k];
      largest = std::max(largest, t.it[k].rows * t.it[k].cols);
    }
    launch(t, n, largest);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

int norm_blocks(int64_t elements) {
  return static_cast<int>(std::min<int64_t>(kNormBlocks, std::max<int64_t>(1, elements / 8192)));
}

// Norms and X_0 of a batch's items.
cudaError_t ingest(const std::vector<Item>& items, bool f32, bool mom, const MuonScalars& s, cudaStream_t stream) {
  return for_items(items, [&](const ItemTable& t, int n, int64_t largest) {
    const int parts = norm_blocks(largest);
    const unsigned tiles = static_cast<unsigned>(std::min<int64_t>(16384, std::max<int64_t>(1, largest / 2048)));
    const dim3 g1(parts, n), g2(tiles, n);
    if (f32 && mom) {
      norm_kernel<true, true><<<g1, 256, 0, stream>>>(t, s);
      scale_kernel<true, true><<<g2, 256, 0, stream>>>(t, s, parts);
    } else if (f32) {
      norm_kernel<true, false><<<g1, 256, 0, stream>>>(t, s);
      scale_kernel<true, false><<<g2, 256, 0, stream>>>(t, s, parts);
    } else if (mom) {
      norm_kernel<false, true><<<g1, 256, 0, stream>>>(t, s);
      scale_kernel<false, true><<<g2, 256, 0, stream>>>(t, s, parts);
    } else {
      norm_kernel<false, false><<<g1, 256, 0, stream>>>(t, s);
      scale_kernel<false, false><<<g2, 256, 0, stream>>>(t, s, parts);
    }
  });
}

Shape2 shape_of(int64_t rows, int64_t cols) { return {std::min(rows, cols), std::max(rows, cols)}; }
bool by_shape(const Shape2& a, const Shape2& b) { return a.m != b.m ? a.m < b.m : a.n < b.n; }

// A workspace for all matrices at once, or for as many as 4 GiB hold, at least one.
constexpr int64_t kMaxBatchBytes = int64_t(4) << 30;

}  // namespace
}  // namespace lst

using namespace lst;

extern "C" int64_t lst_orthogonalize_workspace_bytes(int32_t count, int64_t rows, int64_t cols) {
  if (count <= 0 || rows <= 0 || cols <= 0) return 0;
  const Shape2 s = shape_of(rows, cols);
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
  const Shape2 shape = shape_of(in[0].rows, in[0].cols);
  LST_TRY(check_workspace(workspace, workspace_bytes, Batch::item_bytes(shape), who));
  const int64_t fit = workspace_bytes / Batch::item_bytes(shape);
  const bool tall = in[0].rows > in[0].cols;
  const MuonScalars s = {0.0f, 1.0f, params->eps, 0};
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
        it.x = reinterpret_cast<__half*>(ws + g.x_off[0]) + i * g.m * g.ldx;
        it.ldx = g.ldx;
        it.part = reinterpret_cast<double*>(ws + b.part_off) + i * kNormBlocks;
        it.tall = tall;
      }
      LST_TRY_CUDA(ingest(items, in[0].dtype == LST_F32, false, s, stream), who);
      Runner run{b, ws, stream, {}};
      int si, xi;
      float scale;
      LST_TRY_CUDA(run.iterate(params->steps, use_pairs(shapes.data(), n), &si, &scale, &xi), who);
      // the last product goes to the caller's matrices, transposed back
      for (int64_t i = 0; i < n; ++i) {
        const lst_matrix& dst = out[first + i];
        GemmProblem p;
        p.a = run.s_operand(b.classes[0], si, i, 1);
        p.b = run.x_operand(g, xi);
        p.b.ptr = ws + g.x_off[xi] + i * g.m * g.ldx * 2;
        p.b.batch = 1;
        p.m = g.m;
        p.n = g.n;
        p.k = g.m;
        const uintptr_t align = reinterpret_cast<uintptr_t>(dst.data) | static_cast<uintptr_t>(dst.stride * 2);
        const int vec = align % 32 == 0 ? 32 : align % 16 == 0 ? 16 : 2;
        p.store = {dst.data, nullptr, dst.stride, 0, 1.0f / (scale * kScaleX), 0.0f, 0.0f, 1, tall ? 1 : 0, vec};
        run.pending.push_back(p);
      }
      LST_TRY_CUDA(run.flush(GEMM_NS_APPLY), who);
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
    const int64_t z = Batch::item_bytes(shape_of(t.dims[0], t.dims[1]));
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
        picks.push_back({shape_of(t.dims[0], t.dims[1]), i});
        largest = std::max(largest, Batch::item_bytes(picks.back().s));
      } else if (adamw) {
        const Run r = run_of(t);
        adam.push_back({r.g, r.w, r.m, r.v, static_cast<uint16_t*>(r.w16), t.numel});
      }
    }
    LST_TRY(check_workspace(workspace, workspace_bytes, largest, who));
    std::stable_sort(picks.begin(), picks.end(), [](const Pick& a, const Pick& b) { return by_shape(a.s, b.s); });
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    char* ws = static_cast<char*>(workspace);
    const MuonScalars ms = {hp->momentum, (float)(1.0 - (double)hp->lr * (double)hp->weight_decay), hp->eps,
                            hp->nesterov ? 1 : 0};
    const bool f32 = L->fmt == LST_L16_FP32;

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
          const Tensor& t = L->tensors[(size_t)picks[first + (size_t)(g.first + k)].tensor];
          const Run r = run_of(t);
          Item& it = items[(size_t)(g.first + k)];
          const double rows = (double)t.dims[0], cols = (double)t.dims[1];
          const double scale = hp->rms_scale > 0.0f ? (double)hp->rms_scale * std::sqrt(std::max(rows, cols))
                                                    : std::sqrt(std::max(1.0, rows / cols));
          it = {};
          it.g = r.g;
          it.mom = r.m;
          it.w = r.w;
          it.w16 = static_cast<uint16_t*>(r.w16);
          it.rows = t.dims[0];
          it.cols = it.ld = t.dims[1];
          it.x = reinterpret_cast<__half*>(ws + g.x_off[0]) + k * g.m * g.ldx;
          it.ldx = g.ldx;
          it.part = reinterpret_cast<double*>(ws + b.part_off) + (g.first + k) * kNormBlocks;
          it.tall = t.dims[0] > t.dims[1];
          it.step = (float)((double)hp->lr * scale / (double)kScaleX);
        }
      LST_TRY_CUDA(ingest(items, f32, true, ms, stream), who);
      Runner run{b, ws, stream, {}};
      int si, xi;
      float scale;
      LST_TRY_CUDA(run.iterate(hp->ns_steps, use_pairs(shapes.data(), (int64_t)shapes.size()), &si, &scale, &xi), who);
      LST_TRY_CUDA(run.apply(si, scale, xi, xi ^ 1), who);
      for (const Batch::Group& g : b.groups)
        for (int64_t k = 0; k < g.count; ++k)
          items[(size_t)(g.first + k)].o = reinterpret_cast<const __half*>(ws + g.x_off[xi ^ 1]) + k * g.m * g.ldx;
      LST_TRY_CUDA(for_items(items,
                             [&](const ItemTable& t, int n, int64_t big) {
                               const dim3 grid(
                                   static_cast<unsigned>(std::min<int64_t>(16384, std::max<int64_t>(1, big / 2048))), n);
                               if (L->fmt == LST_L12_BF16)
                                 apply_kernel<F_L12><<<grid, 256, 0, stream>>>(t, ms);
                               else if (L->fmt == LST_L16_MIXED)
                                 apply_kernel<F_L16M><<<grid, 256, 0, stream>>>(t, ms);
                               else
                                 apply_kernel<F_L16F><<<grid, 256, 0, stream>>>(t, ms);
                             }),
                   who);
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
      if (L->fmt == LST_L12_BF16)
        adam_kernel<F_L12><<<grid, 256, 0, stream>>>(t, as);
      else if (L->fmt == LST_L16_MIXED)
        adam_kernel<F_L16M><<<grid, 256, 0, stream>>>(t, as);
      else
        adam_kernel<F_L16F><<<grid, 256, 0, stream>>>(t, as);
      LST_TRY_CUDA(cudaGetLastError(), who);
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
  if (err) return fail(LST_ERR_TIMEOUT, "a wait inside a matrix kernel ran out");
  return LST_OK;
}
