// Tensor-core products of the training operators: one persistent kernel,
// instantiated for the operand layouts and epilogues of lst_gemm.h.
//
// A CTA pair (cluster of 2, tcgen05 cta_group::2) forms a 256 x 256 tile of
// C = A * B with fp32 accumulators in tensor memory: each CTA holds 128 rows
// of the tile, loads its 128 rows of A and its half of B, and the pair's MMAs
// read both halves of B, so a 64-deep K step costs each SM 32 KB of shared
// memory instead of the 48 KB a lone CTA would read for the same rows. Per CTA:
//   warp 0     one thread issues the TMA loads (six 32 KB stages),
//   warp 1     one thread of the leading CTA issues the MMAs,
//   warps 2-9  take finished accumulators from tensor memory: two warps per 32
//              rows, one for each half of the tile's columns.
// Two accumulators alternate, so the epilogue of a tile runs under the main loop
// of the next. Tiles are dealt to the pairs in a fixed order: every result is
// formed by one pair in one order of additions.
// Products that have fewer tiles than the GPU has pairs run with tiles of 256 x
// 128: twice the pairs at work, half the time to a tile's end.
#include "lst_gemm.h"

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "lst_ops.h"
#include "lst_tc.cuh"

namespace lst {

namespace {

constexpr int kTileK = 64;
constexpr int kStages = 6;
constexpr int kABytes = 128 * kTileK * 2;  // one CTA's rows of A
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kBarriers = 2 * kStages + 4;
__host__ __device__ constexpr int b_bytes(int tile_n) { return tile_n / 2 * kTileK * 2; }  // one CTA's half of B
constexpr int kTurnBytes = 32 * 33 * 4;  // a warp's 32 x 32 values on their way from rows to columns
__host__ __device__ constexpr int smem_bytes(int tile_n) {
  return kStages * (kABytes + b_bytes(tile_n)) + 1024 + 8 * kBarriers + 16 + kEpiWarps * kTurnBytes;
}

__device__ int g_gemm_error;

struct Shape {
  int32_t m, n;
  int32_t k_blocks, k_per_split, splits;
  int32_t tiles_m, tiles_n, tiles;  // tiles: of one matrix and one split
  int32_t symmetric;
  int32_t a_mn, b_mn;  // operand is MN-major in memory
  int32_t first_tile;
  int32_t part_blocks;  // K blocks of a part of B (weight gradients)
};

struct Nothing {};

template <class Epi>
struct Args {
  CUtensorMap a[kGemmMaxProblems], b[kGemmMaxProblems], b_half[kGemmMaxProblems];
  Shape shape[kGemmMaxProblems];
  typename Epi::Params epi[kGemmMaxProblems];
  typename Epi::Table table;
  int32_t count, whole_tiles, total_tiles;  // the tiles from whole_tiles on are halves
  int32_t mixed;                            // sums of different lengths
};

struct Tile {
  int problem, batch, split, tm, tn, kb0, kb1;
  int half;  // -1: the whole tile; 0, 1: these half of its columns
};

// Tiles of a matrix go down groups of 8 tile rows, column by column: the tiles
// in flight share 8 row panels of A and a few column panels of B, which stay
// in L2. A symmetric result has the tiles of its upper triangle, row by row.
template <int kTileN, class Epi>
__device__ __forceinline__ Tile decode(const Args<Epi>& g, int t) {
  Tile r;
  r.half = -1;
  if (kTileN == kGemmTile && t >= g.whole_tiles) {
    r.half = (t - g.whole_tiles) & 1;
    t = g.whole_tiles + ((t - g.whole_tiles) >> 1);
  }
  int p = 0;
  while (p + 1 < g.count && t >= g.shape[p + 1].first_tile) ++p;
  const Shape& s = g.shape[p];
  int i = t - s.first_tile;
  // divisions (some 20 dependent instructions) only where they are needed
  const int matrix = i < s.tiles ? 0 : i / s.tiles;
  i -= matrix * s.tiles;
  r.problem = p;
  r.batch = s.splits == 1 ? matrix : matrix / s.splits;
  r.split = matrix - r.batch * s.splits;
  if (s.symmetric) {
    constexpr int kAcross = kGemmTile / kTileN;
    int row = 0;
    while (i >= s.tiles_n - kAcross * row) {
      i -= s.tiles_n - kAcross * row;
      ++row;
    }
    r.tm = row;
    r.tn = kAcross * row + i;
  } else {
    const int per_group = 8 * s.tiles_n;
    const int group = i / per_group;
    const int rows = min(8, s.tiles_m - group * 8);
    i -= group * per_group;
    const int across = rows == 8 ? i >> 3 : i / rows;
    r.tm = group * 8 + i - across * rows;
    r.tn = across;
  }
  r.kb0 = r.split * s.k_per_split;
  r.kb1 = min(s.k_blocks, r.kb0 + s.k_per_split);
  return r;
}

// ---- epilogues ---------------------------------------------------------------
// Each warp calls run() with its accumulator address (32 lanes = 32 rows, kCols
// = half a tile's columns); prepare() runs before the tile is complete. `release`
// must be called once, by all lanes, when the accumulator has been read.

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float unpack16(uint16_t u, bool bf16) {
  return bf16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

// Epilogues go through a row 16 columns at a time in loops that are not unrolled:
// a launch of few tiles runs this code once, and fetching long unrolled code took
// longer (4 us for a 256 x 128 tile) than running it. What a group reads from
// memory is fetched one group ahead.

// 32 accumulator columns with the lanes turned from rows to columns, through the
// warp's words at `turn`: v[i] becomes row i of the lane's column. What is then
// read and written is consecutive over the lanes.
__device__ __forceinline__ void load_turned(uint32_t tmem, uint32_t turn, float (&v)[32]) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  tc::tmem_ld32(tmem, v);
  tc::tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("st.shared.f32 [%0], %1;" ::"r"(turn + (lane * 33 + i) * 4), "f"(v[i]));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i]) : "r"(turn + (i * 33 + lane) * 4));
}

// The same in units of kUnit = 4 or 8 consecutive columns a lane. Units of 4: v[i] is
// columns 4 (lane % 8) .. of row 4 i + lane / 8; of 8: v[2 i] and v[2 i + 1] are
// columns 8 (lane % 4) .. of row 8 i + lane / 4. 16-byte accesses, no bank conflicts.
template <int kUnit>
__device__ __forceinline__ void load_units(uint32_t tmem, uint32_t turn, float4 (&v)[8]) {
  const int lane = threadIdx.x & 31;
  auto word = [&](int r, int u) { return turn + r * 128 + ((u ^ (r & 7)) << 4); };
  float a[32];
  __syncwarp();
  tc::tmem_ld32(tmem, a);
  tc::tmem_ld_wait();
#pragma unroll
  for (int u = 0; u < 8; ++u)
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(word(lane, u)), "f"(a[4 * u]), "f"(a[4 * u + 1]),
                 "f"(a[4 * u + 2]), "f"(a[4 * u + 3]));
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t from = kUnit == 4 ? word(4 * i + (lane >> 3), lane & 7) : word(8 * (i >> 1) + (lane >> 2), 2 * (lane & 3) + (i & 1));
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[i].x), "=f"(v[i].y), "=f"(v[i].z), "=f"(v[i].w) : "r"(from));
  }
}

// The first `left` < 8 values of 8.
__device__ __forceinline__ uint4 load_tail(const uint16_t* p, int left) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < left) w[i >> 1] |= static_cast<uint32_t>(p[i]) << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_tail(uint16_t* p, const uint4& v, int left) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < left) p[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
}

struct StoreEpilogue {
  template <int kCols, class... Rest>
  static __device__ __forceinline__ void prepare(const Rest&...) {}
  using Params = StoreParams;
  using Table = Nothing;
  // Rows that are not on 16 bytes (a caller's matrix: not symmetric, no diagonal).
  template <int kCols>
  static __device__ __forceinline__ void turned(const Params& e, const Shape& s, const Tile& t, int row, int col0, uint32_t tmem,
                                                uint32_t turn) {
    const bool bf16 = e.bf16 != 0;
    const float alpha = e.scale ? e.alpha * *e.scale : e.alpha;
    const int row0 = row & ~31, lane = row & 31, rows = s.m - row0;
    const int64_t first = t.batch * e.batch_stride + static_cast<int64_t>(row0) * e.ld + col0 + lane;
#pragma unroll 1
    for (int g = 0; g < kCols / 32; ++g) {
      if (col0 + 32 * g >= s.n) break;
      const bool inside = col0 + 32 * g + lane < s.n;
      const int64_t at = first + 32 * g;
      uint16_t old[32];
      if (e.c) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (inside && i < rows) old[i] = static_cast<const uint16_t*>(e.c)[at + i * e.ld];
      }
      float v[32];
      load_turned(tmem + 32 * g, turn, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (inside && i < rows) {
          float y = v[i] * alpha;
          if (e.c) y = __fmaf_rn(e.beta, unpack16(old[i], bf16), y);
          static_cast<uint16_t*>(e.out)[at + i * e.ld] = static_cast<uint16_t>(pack16(y, 0.0f, bf16));
        }
      }
    }
  }
  template <int kCols, bool kOnlyBf16 = false, class Release>
  static __device__ __forceinline__ void run(const Params& e, const Table&, const Shape& s, const Tile& t, int row,
                                             int col0, uint32_t tmem, uint32_t turn, Release release) {
    if (e.vec < 16) {
      turned<kCols>(e, s, t, row, col0, tmem, turn);
      __syncwarp();
      release();
      return;
    }
    // 64 columns at a time through the warp's words, row by row in, four whole
    // 128-byte rows an instruction out: a lane per row would touch 32 lines with
    // every store (five symmetric products of 2048: 41.2 us that way, 36.6 so).
    const bool bf16 = kOnlyBf16 || e.bf16 != 0;
    const float alpha = e.scale ? e.alpha * *e.scale : e.alpha;
    constexpr int kAcross = kGemmTile / (2 * kCols);  // tiles of a diagonal block are formed whole
    const bool mirror = s.symmetric && t.tn >= kAcross * (t.tm + 1);
    const int lane = row & 31, row0 = row & ~31, rows = s.m - row0;
    const int64_t matrix = t.batch * e.batch_stride;
    uint16_t* const out = static_cast<uint16_t*>(e.out) + matrix;
    const uint16_t* const c = e.c ? static_cast<const uint16_t*>(e.c) + matrix : nullptr;
    const int unit = lane & 7;                              // 8 columns, of rows 4 i + lane / 8
    auto word = [&](int r, int u) { return turn + r * 128 + ((u ^ (r & 7)) << 4); };
#pragma unroll 1
    for (int h = 0; h < kCols / 64; ++h) {
      const int col = col0 + 64 * h, left = s.n - col;
      if (left <= 0) break;
      __syncwarp();
      if (c) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3);
          const uint16_t* p = c + static_cast<int64_t>(row0 + r) * e.ld + col + 8 * unit;
          w[i] = make_uint4(0, 0, 0, 0);
          if (r < rows && 8 * unit + 8 <= left)
            w[i] = *reinterpret_cast<const uint4*>(p);
          else if (r < rows && 8 * unit < left)
            w[i] = load_tail(p, left - 8 * unit);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t a = word(4 * i + (lane >> 3), unit);
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(w[i].x), "r"(w[i].y), "r"(w[i].z), "r"(w[i].w));
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
        float v[16];
        __syncwarp();
        tc::tmem_ld16(tmem + 64 * h + 16 * g, v);
        const uint32_t a0 = word(lane, 2 * g), a1 = word(lane, 2 * g + 1);
        uint32_t w[8];
        if (c) {
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a0));
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7]) : "r"(a1));
        }
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = v[i] * alpha;
        if (c) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            v[i] = __fmaf_rn(e.beta, unpack16(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))), bf16), v[i]);
        }
        const int diag = row - col - 16 * g;
        if (e.diag != 0.0f && diag >= 0 && diag < 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] += i == diag ? e.diag : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = pack16(v[2 * i], v[2 * i + 1], bf16);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a0), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]));
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a1), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]));
        if (mirror && lane < rows) {
          uint16_t* across = out + static_cast<int64_t>(col + 16 * g) * e.ld + row;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (16 * g + i < left) across[static_cast<int64_t>(i) * e.ld] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
      }
      __syncwarp();
      uint16_t* p = out + static_cast<int64_t>(row0 + (lane >> 3)) * e.ld + col + 8 * unit;
#pragma unroll
      for (int i = 0; i < 8; ++i, p += 4 * e.ld) {
        const int r = 4 * i + (lane >> 3);
        uint4 w;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(word(r, unit)));
        if (r < rows && 8 * unit + 8 <= left)
          *reinterpret_cast<uint4*>(p) = w;
        else if (r < rows && 8 * unit < left)
          store_tail(p, w, left - 8 * unit);
      }
    }
    __syncwarp();
    release();
  }
};

// The Muon update of the weights by a tile of the orthogonalised matrix.
struct UpdateEpilogue {
  using Params = UpdateParams;
  using Table = UpdateTable;
  // The tile's weights to L2 while its main loop runs, a row's columns in one request.
  template <int kCols>
  static __device__ __forceinline__ void prepare(const Params& e, const Table& table, const Shape& s, const Tile& t, int row,
                                                 int col0) {
    if (row >= s.m || col0 >= s.n || e.vec < 16) return;
    const int size = e.format == LST_L12_BF16 ? 2 : 4, bytes = (min(kCols, s.n - col0) * size) & ~15;
    const char* w = static_cast<const char*>(table.w[e.first + t.batch]) + (static_cast<int64_t>(row) * e.ld + col0) * size;
    if (bytes > 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(w), "r"(bytes) : "memory");
  }
  // Rows on 16 bytes: 32 columns of 32 rows at a time, 16 bytes a lane, whole rows
  // (128 bytes of fp32, 64 of bf16) an instruction. The last
  // product of a TinyLlama layer (mixed layout, 97 us of MMA): 136 us; with a row per
  // lane, 64 bytes at a time, 190; with 4 bytes a lane along the columns, 205.
  template <bool kBf16, int kCols>
  static __device__ __forceinline__ void units(const Params& e, float step, char* w, uint16_t* w16, int rows, int left,
                                               uint32_t tmem, uint32_t turn) {
    constexpr int kUnit = kBf16 ? 8 : 4, kAcross = 32 / kUnit, kDown = 32 / kAcross, kLoads = 32 / kDown;
    constexpr int kSize = kBf16 ? 2 : 4, kAhead = kBf16 ? 2 : 1, kGroups = kCols / 32;
    const int lane = threadIdx.x & 31, r0 = lane / kAcross, c0 = kUnit * (lane % kAcross);
    const int64_t at = r0 * e.ld + c0, down = kDown * e.ld;  // elements
    uint4 next[kAhead][kLoads];
    auto fetch = [&](uint4 (&x)[kLoads], int g) {
      if (g >= kGroups || 32 * g + c0 >= left) return;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if (kDown * i + r0 < rows) x[i] = __ldcg(reinterpret_cast<const uint4*>(w + (at + i * down + 32 * g) * kSize));
    };
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(next[k], k);
#pragma unroll 1
    for (int g = 0; g < kGroups; ++g) {
      if (32 * g >= left) break;
      uint4 x[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        x[i] = next[0][i];
        if (kAhead == 2) next[0][i] = next[kAhead - 1][i];
      }
      fetch(next[kAhead - 1], g + kAhead);
      float4 v[8];
      load_units<kUnit>(tmem + 32 * g, turn, v);
      auto updated = [&](float old, float o) { return __fsub_rn(__fmul_rn(old, e.decay), __fmul_rn(step, o)); };
      if (32 * g + c0 >= left) continue;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (kDown * i + r0 >= rows) break;
        const int64_t p = at + i * down + 32 * g;
        if (kBf16) {
          const uint32_t o[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          const float4 lo = v[(2 * i) & 7], hi = v[(2 * i + 1) & 7];
          const float d[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          uint32_t n[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            n[j] = pack16(updated(__uint_as_float(o[j] << 16), d[2 * j]), updated(__uint_as_float(o[j] & 0xffff0000u), d[2 * j + 1]), true);
          *reinterpret_cast<uint4*>(w + p * kSize) = make_uint4(n[0], n[1], n[2], n[3]);
        } else {
          const float4 d = v[i];
          const float4 n = make_float4(updated(__uint_as_float(x[i].x), d.x), updated(__uint_as_float(x[i].y), d.y),
                                       updated(__uint_as_float(x[i].z), d.z), updated(__uint_as_float(x[i].w), d.w));
          *reinterpret_cast<float4*>(w + p * kSize) = n;
          if (e.format == LST_L16_MIXED)
            *reinterpret_cast<uint2*>(w16 + p) = make_uint2(pack16(n.x, n.y, true), pack16(n.z, n.w, true));
        }
      }
    }
  }
  template <int kCols, class Release>
  static __device__ __forceinline__ void run(const Params& e, const Table& table, const Shape& s, const Tile& t, int row,
                                             int col0, uint32_t tmem, uint32_t turn, Release release) {
    const bool bf16 = e.format == LST_L12_BF16;
    const float step = table.step[e.first + t.batch];
    const int row0 = row & ~31, lane = row & 31, rows = s.m - row0;
    const int64_t first = static_cast<int64_t>(row0) * e.ld + col0 + lane;
    char* const weights = static_cast<char*>(table.w[e.first + t.batch]);
    uint16_t* const w16 = bf16 ? reinterpret_cast<uint16_t*>(weights) : table.w16[e.first + t.batch];
    if (e.vec >= 16) {
      const int64_t at = static_cast<int64_t>(row0) * e.ld + col0;
      if (bf16)
        units<true, kCols>(e, step, weights + at * 2, w16, rows, s.n - col0, tmem, turn);
      else
        units<false, kCols>(e, step, weights + at * 4, w16 + at, rows, s.n - col0, tmem, turn);
      __syncwarp();
      release();
      return;
    }
    float next[32];
    auto fetch = [&](int g) {
      const int64_t at = first + 32 * g;
      const bool inside = col0 + 32 * g + lane < s.n;
      if (bf16) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (inside && i < rows) next[i] = __uint_as_float(__ldcg(reinterpret_cast<const uint16_t*>(weights) + at + i * e.ld));
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (inside && i < rows) next[i] = __ldcg(reinterpret_cast<const float*>(weights) + at + i * e.ld);
      }
    };
    fetch(0);
#pragma unroll 1
    for (int g = 0; g < kCols / 32; ++g) {
      if (col0 + 32 * g >= s.n) break;
      const bool inside = col0 + 32 * g + lane < s.n;
      const int64_t at = first + 32 * g;
      float v[32], x[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = next[i];
      if (g + 1 < kCols / 32) fetch(g + 1);
      load_turned(tmem + 32 * g, turn, v);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (inside && i < rows) {
          if (bf16) x[i] = unpack16(static_cast<uint16_t>(__float_as_uint(x[i])), true);
          const float y = __fsub_rn(__fmul_rn(x[i], e.decay), __fmul_rn(step, v[i]));
          if (!bf16) reinterpret_cast<float*>(weights)[at + i * e.ld] = y;
          if (e.format != LST_L16_FP32)
            reinterpret_cast<__nv_bfloat16*>(w16)[at + i * e.ld] = __float2bfloat16_rn(y);
        }
      }
    }
    __syncwarp();
    release();
  }
};

struct PartialEpilogue {
  using Params = PartialParams;
  using Table = Nothing;
  // Rows of `out` hold whole units of 4 columns: ld is a multiple of 4.
  template <int kCols, class Release>
  static __device__ __forceinline__ void run(const Params& e, const Table&, const Shape& s, const Tile& t, int row,
                                             int col0, uint32_t tmem, uint32_t turn, Release release) {
    const int lane = row & 31, row0 = row & ~31, rows = s.m - row0, r0 = lane >> 3, c0 = 4 * (lane & 7);
    float* const out = e.out + t.split * e.split_stride + static_cast<int64_t>(row0 + r0) * e.ld + col0 + c0;
#pragma unroll 1
    for (int g = 0; g < kCols / 32; ++g) {
      if (col0 + 32 * g >= s.n) break;
      const bool inside = col0 + 32 * g + c0 < s.n;
      float4 old[8] = {}, v[8];
      if (e.accumulate) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (inside && 4 * i + r0 < rows) old[i] = *reinterpret_cast<const float4*>(out + 4 * i * e.ld + 32 * g);
      }
      load_units<4>(tmem + 32 * g, turn, v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (inside && 4 * i + r0 < rows)
          *reinterpret_cast<float4*>(out + 4 * i * e.ld + 32 * g) =
              make_float4(old[i].x + v[i].x, old[i].y + v[i].y, old[i].z + v[i].z, old[i].w + v[i].w);
    }
    __syncwarp();
    release();
  }
};

struct GradParams {
  StoreParams store;
  PartialParams partial;
};
struct GradEpilogue {
  template <int kCols, class... Rest>
  static __device__ __forceinline__ void prepare(const Rest&...) {}
  using Params = GradParams;
  using Table = Nothing;
  template <int kCols, class Release>
  static __device__ __forceinline__ void run(const Params& e, const Table& table, const Shape& s, const Tile& t, int row,
                                             int col0, uint32_t tmem, uint32_t turn, Release release) {
    if (e.partial.out)
      PartialEpilogue::run<kCols>(e.partial, table, s, t, row, col0, tmem, turn, release);
    else
      StoreEpilogue::run<kCols, true>(e.store, table, s, t, row, col0, tmem, turn, release);
  }
};

// A weight gradient: the sums times a weight per column, written or added.
struct WgradEpilogue {
  using Params = WgradParams;
  using Table = Nothing;
  // What the gradient holds comes to L2 while the main loop runs.
  template <int kCols>
  static __device__ __forceinline__ void prepare(const Params& e, const Table&, const Shape& s, const Tile&, int row, int col0) {
    if (!e.accumulate || e.partial.out || row >= s.m || col0 >= s.n || e.vec < 16) return;
    const int size = e.f32 ? 4 : 2, bytes = (min(kCols, s.n - col0) * size) & ~15;
    const char* p = static_cast<const char*>(e.out) + (static_cast<int64_t>(row) * e.ld + col0) * size;
    if (bytes > 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
  }
  static __device__ __forceinline__ float weight_of(const Params& e, int col) {
    return e.weight_f32 ? static_cast<const float*>(e.weight)[col] : __bfloat162float(static_cast<const __nv_bfloat16*>(e.weight)[col]);
  }
  // Rows on 16 bytes: 32 columns of 32 rows at a time, 16 bytes a lane.
  template <bool kBf16, int kCols>
  static __device__ __forceinline__ void units(const Params& e, char* out, int rows, int col0, int left, uint32_t tmem, uint32_t turn) {
    constexpr int kUnit = kBf16 ? 8 : 4, kAcross = 32 / kUnit, kDown = 32 / kAcross, kLoads = 32 / kDown, kSize = kBf16 ? 2 : 4;
    const int lane = threadIdx.x & 31, r0 = lane / kAcross, c0 = kUnit * (lane % kAcross);
#pragma unroll 1
    for (int g = 0; g < kCols / 32; ++g) {
      const int mine = left - 32 * g - c0;  // columns from this lane's first on
      if (32 * g >= left) break;
      char* const p0 = out + (r0 * e.ld + 32 * g + c0) * kSize;
      uint4 old[kLoads];
      if (e.accumulate) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          if (mine >= kUnit && kDown * i + r0 < rows) old[i] = __ldcg(reinterpret_cast<const uint4*>(p0 + kDown * i * e.ld * kSize));
      }
      float w[kUnit];
#pragma unroll
      for (int j = 0; j < kUnit; ++j) w[j] = e.weight && j < mine ? weight_of(e, col0 + 32 * g + c0 + j) : 1.0f;
      float4 v[8];
      load_units<kUnit>(tmem + 32 * g, turn, v);
      if (mine <= 0) continue;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (kDown * i + r0 >= rows) break;
        char* const p = p0 + kDown * i * e.ld * kSize;
        float d[kUnit];
        if (kBf16) {
          const float4 lo = v[(2 * i) & 7], hi = v[(2 * i + 1) & 7];
          const float t[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int j = 0; j < kUnit; ++j) d[j] = t[j] * w[j];
        } else {
          const float t[4] = {v[i & 7].x, v[i & 7].y, v[i & 7].z, v[i & 7].w};
#pragma unroll
          for (int j = 0; j < kUnit; ++j) d[j] = t[j & 3] * w[j];
        }
        if (mine >= kUnit) {
          const uint32_t o[4] = {old[i].x, old[i].y, old[i].z, old[i].w};
          uint4 n;
          if (kBf16) {
            if (e.accumulate) {
#pragma unroll
              for (int j = 0; j < kUnit; ++j) d[j] += __uint_as_float(j & 1 ? o[(j >> 1) & 3] & 0xffff0000u : o[(j >> 1) & 3] << 16);
            }
            n = make_uint4(pack16(d[0], d[1], true), pack16(d[2], d[3], true), pack16(d[4 % kUnit], d[5 % kUnit], true),
                           pack16(d[6 % kUnit], d[7 % kUnit], true));
          } else {
            if (e.accumulate) {
#pragma unroll
              for (int j = 0; j < kUnit; ++j) d[j] += __uint_as_float(o[j & 3]);
            }
            n = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
          }
          *reinterpret_cast<uint4*>(p) = n;
        } else {
#pragma unroll
          for (int j = 0; j < kUnit; ++j)
            if (j < mine) put(e, p + j * kSize, d[j]);
        }
      }
    }
  }
  // Rows on any alignment: a column a lane.
  template <class T, int kCols>
  static __device__ __forceinline__ void turned(const Params& e, char* out, int rows, int col0, int left, uint32_t tmem, uint32_t turn) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int g = 0; g < kCols / 32; ++g) {
      if (32 * g >= left) break;
      const bool inside = 32 * g + lane < left;
      const float w = e.weight && inside ? weight_of(e, col0 + 32 * g + lane) : 1.0f;
      T* const first = reinterpret_cast<T*>(out) + 32 * g + lane;
      float v[32];
      if (e.accumulate) {
        T old[32];
        const T* p = first;
#pragma unroll
        for (int i = 0; i < 32; ++i, p += e.ld)
          if (inside && i < rows) old[i] = *p;
        load_turned(tmem + 32 * g, turn, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = static_cast<float>(old[i]) + v[i] * w;
      } else {
        load_turned(tmem + 32 * g, turn, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = v[i] * w;
      }
      T* p = first;
      if (inside && rows >= 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i, p += e.ld) *p = static_cast<T>(v[i]);
      } else if (inside) {
#pragma unroll
        for (int i = 0; i < 32; ++i, p += e.ld)
          if (i < rows) *p = static_cast<T>(v[i]);
      }
    }
  }
  static __device__ __forceinline__ void put(const Params& e, char* p, float v) {
    if (e.f32) {
      float* q = reinterpret_cast<float*>(p);
      *q = e.accumulate ? *q + v : v;
    } else {
      __nv_bfloat16* q = reinterpret_cast<__nv_bfloat16*>(p);
      *q = __float2bfloat16_rn(e.accumulate ? __bfloat162float(*q) + v : v);
    }
  }
  template <int kCols, class Release>
  static __device__ __forceinline__ void run(const Params& e, const Table& table, const Shape& s, const Tile& t, int row,
                                             int col0, uint32_t tmem, uint32_t turn, Release release) {
    if (e.partial.out) {
      PartialEpilogue::run<kCols>(e.partial, table, s, t, row, col0, tmem, turn, release);
      return;
    }
    const int row0 = row & ~31, lane = row & 31, rows = s.m - row0, left = s.n - col0, size = e.f32 ? 4 : 2;
    char* const out = static_cast<char*>(e.out) + (static_cast<int64_t>(row0) * e.ld + col0) * size;
    if (e.vec >= 16) {
      if (e.f32)
        units<false, kCols>(e, out, rows, col0, left, tmem, turn);
      else
        units<true, kCols>(e, out, rows, col0, left, tmem, turn);
    } else {
      if (e.f32)
        turned<float, kCols>(e, out, rows, col0, left, tmem, turn);
      else
        turned<__nv_bfloat16, kCols>(e, out, rows, col0, left, tmem, turn);
    }
    __syncwarp();
    release();
  }
};

// One row's logits of 128 vocabulary entries: their maximum M, the sum of
// exp(l - M), the target's logit where it is among them, and (for the
// gradient) q = (M - l) * 2^11 in 16 bits. q keeps l to 2^-12 over the 32
// below M, where rounding l itself to bf16 would keep a logit of 16 only to
// 2^-5; an entry further below (a probability under 1e-14 of its group's
// largest, or zero at a logit of -inf) saturates and counts as zero.
struct XentEpilogue {
  template <int kCols, class... Rest>
  static __device__ __forceinline__ void prepare(const Rest&...) {}
  using Params = XentParams;
  using Table = Nothing;
  template <int kCols, class Release>
  static __device__ __forceinline__ void run(const Params& e, const Table& table, const Shape& s, const Tile& t, int row,
                                             int col0, uint32_t tmem, uint32_t turn, Release release) {
    static_assert(kCols == 128, "statistics are per 128 columns");
    if (col0 >= s.n) {
      release();
      return;
    }
    const int left = min(s.n - col0, 128);
    const float ninf = __int_as_float(0xff800000);
    float top = ninf;
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      float v[16];
      __syncwarp();
      tc::tmem_ld16(tmem + 16 * g, v);
      tc::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * g + i < left) top = fmaxf(top, v[i]);
    }
    const bool inside = row < s.m;
    int target = -1;
    if (inside) {
      int64_t t64 = e.index_bytes == 8 ? static_cast<const int64_t*>(e.targets)[row] : static_cast<const int32_t*>(e.targets)[row];
      t64 -= e.first_column + col0;
      if (t64 >= 0 && t64 < left) target = static_cast<int>(t64);
    }
    // all -inf: the sum is 0, or NaN where a logit is (max passes over NaN)
    const float base = top == ninf ? 0.0f : top;
    float sum0 = 0.0f, sum1 = 0.0f, at_target = 0.0f;
    uint16_t* const out = e.q && inside ? e.q + static_cast<int64_t>(row) * e.q_ld + col0 : nullptr;
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      float v[16];
      __syncwarp();
      tc::tmem_ld16(tmem + 16 * g, v);
      tc::tmem_ld_wait();
      if (16 * g + 16 > left) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (16 * g + i >= left) v[i] = ninf;
      }
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        sum0 += tc::exp2_approx((v[i] - base) * 1.4426950408889634f);
        sum1 += tc::exp2_approx((v[i + 1] - base) * 1.4426950408889634f);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) at_target = 16 * g + i == target ? v[i] : at_target;
      if (out) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = fminf((top - v[2 * i]) * 2048.0f, 65535.0f);
          const float hi = fminf((top - v[2 * i + 1]) * 2048.0f, 65535.0f);
          w[i] = __float2uint_rn(lo) | (__float2uint_rn(hi) << 16);
        }
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + 16 * g), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");  // q_ld is a multiple of 256
      }
    }
    __syncwarp();
    release();
    if (inside) {
      e.stats[row * e.stat_ld + e.first_group + (col0 >> 7)] = make_float2(top, sum0 + sum1);
      if (target >= 0) e.target_logit[row] = at_target;
    }
  }
};

// The same for few tokens, with the vocabulary in the rows and the tokens in the
// columns: a tile is 256 x 32 or 256 x 64, so that the MMAs of 16 tokens take an
// eighth of the time and the launch is bound by reading w. Per token and 32
// vocabulary entries, 16 tokens at a time: a lane takes 16 entries of a token, the
// other 16 are its partner's (lane ^ 16).
struct XentFewEpilogue {
  template <int kCols, class... Rest>
  static __device__ __forceinline__ void prepare(const Rest&...) {}
  using Params = XentParams;
  using Table = Nothing;
  template <int kCols, class Release>
  static __device__ __forceinline__ void run(const Params& e, const Table& table, const Shape& s, const Tile& t, int row,
                                             int col0, uint32_t tmem, uint32_t turn, Release release) {
    const int lane = row & 31, row0 = row & ~31, left = s.m - row0, first = lane & 16;
    if (left <= 0 || col0 >= s.n) {
      release();
      return;
    }
    const float ninf = __int_as_float(0xff800000);
#pragma unroll 1
    for (int c = 0; c < kCols; c += 16) {
      float v[16];
      __syncwarp();
      tc::tmem_ld16(tmem + c, v);
      tc::tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) asm volatile("st.shared.f32 [%0], %1;" ::"r"(turn + (lane * 17 + i) * 4), "f"(v[i]));
      __syncwarp();
      if (c + 16 == kCols) release();
      const int token = col0 + c + (lane & 15);
      float top = ninf;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[i]) : "r"(turn + ((first + i) * 17 + (lane & 15)) * 4));
        if (first + i >= left) v[i] = ninf;
        top = fmaxf(top, v[i]);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float base = top == ninf ? 0.0f : top;  // as above
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += tc::exp2_approx((v[i] - base) * 1.4426950408889634f);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (token >= s.n) continue;
      if (e.q) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float lo = fminf((top - v[2 * i]) * 2048.0f, 65535.0f);
          const float hi = fminf((top - v[2 * i + 1]) * 2048.0f, 65535.0f);
          w[i] = __float2uint_rn(lo) | (__float2uint_rn(hi) << 16);
        }
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(e.q + token * e.q_ld + row0 + first), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
      }
      if (first == 0) e.stats[token * e.stat_ld + e.first_group + (row0 >> 5)] = make_float2(top, sum);
      int64_t at = e.index_bytes == 8 ? static_cast<const int64_t*>(e.targets)[token] : static_cast<const int32_t*>(e.targets)[token];
      at -= e.first_column + row0 + first;
      if (at >= 0 && at < 16 && at < left - first) {
        float logit = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) logit = i == static_cast<int>(at) ? v[i] : logit;
        e.target_logit[token] = logit;
      }
    }
  }
};

// ---- the kernel ----------------------------------------------------------------
template <class Epi, bool kBf16, int kTileN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ Args<Epi> g) {
  constexpr int kBBytes = b_bytes(kTileN), kStageBytes = kABytes + kBBytes;
  constexpr bool kParts = std::is_same<Epi, WgradEpilogue>::value;  // only weight gradients have B in parts
  constexpr uint32_t kTmemColumns = 2 * kTileN;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (tc::smem_addr(smem_raw) + 1023) & ~1023u;
  const uint32_t bars = base + kStages * kStageBytes;
  const uint32_t full = bars, empty = bars + 8 * kStages, tfull = bars + 16 * kStages, tempty = tfull + 16;
  const uint32_t tmem_slot = tempty + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;

  let_next_start();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(full + 8 * i, 1);
      tc::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tfull + 8 * i, 1);
      tc::mbar_init(tempty + 8 * i, 2 * kEpiWarps);
    }
    tc::mbar_init_fence();
  }
  if (warp == 1) {
    __syncwarp();
    tc::tmem_alloc_pair(tmem_slot, kTmemColumns);
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
  // while the launch before runs on: the first tile's parameters and tensor maps,
  // whose first reads take about 0.5 us
  const Tile first = decode<kTileN>(g, cluster);
  if (warp == 0 && lane == 0) {
    tc::prefetch_map(&g.a[first.problem]);
    tc::prefetch_map(&g.b[first.problem]);
  }
  const int32_t* words = reinterpret_cast<const int32_t*>(&g.epi[first.problem]);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(typename Epi::Params) / 4); i += 8) asm volatile("" ::"r"(words[i]));
  wait_for_previous();
  bool ok = true;
  // tile of this pair in wave w: with sums of different lengths the waves go back and
  // forth over the pairs, so that pairs with a longer sum in one wave have a shorter
  // one in the next. (A LLaMA-7B layer by Muon: 9140 us without, 9080 with.)
  auto tile_at = [&](int w) { return w * clusters + ((w & 1) && g.mixed ? clusters - 1 - cluster : cluster); };
  if (warp == 0) {
    if (tc::elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      for (int w = 0, t = cluster; t < g.total_tiles && ok; t = tile_at(++w)) {
        const Tile tile = t == cluster ? first : decode<kTileN>(g, t);
        const CUtensorMap* ma = &g.a[tile.problem];
        const CUtensorMap* mb = &g.b[tile.problem];
        const int m0 = tile.tm * kGemmTile + 128 * static_cast<int>(rank);
        const bool half = tile.half >= 0;
        const int n0 = tile.tn * kTileN + (half ? kTileN / 2 * tile.half + kTileN / 4 * static_cast<int>(rank) : kTileN / 2 * static_cast<int>(rank));
        const uint32_t bytes = 2 * (half ? kStageBytes - kBBytes / 2 : kStageBytes);
        if (half) mb = &g.b_half[tile.problem];
        const bool a_mn = g.shape[tile.problem].a_mn, b_mn = g.shape[tile.problem].b_mn;
        for (int k = tile.kb0; k < tile.kb1; ++k) {
          int kb = k, of_b = tile.batch;  // K block of both, and matrix of B
          if (kParts)
            for (; kb >= g.shape[tile.problem].part_blocks; kb -= g.shape[tile.problem].part_blocks) ++of_b;
          ok = tc::mbar_wait(empty + 8 * stage, phase ^ 1);
          if (!ok) break;
          const uint32_t sa = base + stage * kStageBytes, sb = sa + kABytes;
          if (rank == 0) tc::mbar_expect_tx(full + 8 * stage, bytes);
          const uint32_t bar = tc::map_to_rank(full + 8 * stage, 0);
          if (a_mn) {
            tc::tma_load_3d_pair(sa, ma, bar, m0, kb * kTileK, tile.batch);
            tc::tma_load_3d_pair(sa + kABytes / 2, ma, bar, m0 + 64, kb * kTileK, tile.batch);
          } else {
            tc::tma_load_3d_pair(sa, ma, bar, kb * kTileK, m0, tile.batch);
          }
          if (b_mn) {
            tc::tma_load_3d_pair(sb, mb, bar, n0, kb * kTileK, of_b);
            if (kTileN == 256 && !half) tc::tma_load_3d_pair(sb + kBBytes / 2, mb, bar, n0 + 64, kb * kTileK, of_b);
          } else {
            tc::tma_load_3d_pair(sb, mb, bar, kb * kTileK, n0, of_b);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0 && tc::elect_one()) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      for (int w = 0, t = cluster; t < g.total_tiles && ok; t = tile_at(++w)) {
        const Tile tile = t == cluster ? first : decode<kTileN>(g, t);
        ok = tc::mbar_wait(tempty + 8 * buf, tphase ^ 1);
        if (!ok) break;
        tc::fence_after();
        const uint32_t d = tmem + kTileN * buf;
        const bool a_mn = g.shape[tile.problem].a_mn, b_mn = g.shape[tile.problem].b_mn;
        const uint32_t idesc = tc::instr_desc(kGemmTile, tile.half < 0 ? kTileN : kTileN / 2, kBf16, a_mn, b_mn);
        // one MMA is 16 deep in K: 32 bytes along a K-major row, 16 rows of 128
        // bytes in the MN-major order (descriptor units of 16 bytes)
        const uint64_t step_a = a_mn ? 128 : 2, step_b = b_mn ? 128 : 2;
        for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
          ok = tc::mbar_wait(full + 8 * stage, phase);
          if (!ok) break;
          tc::fence_after();
          const uint32_t sa = base + stage * kStageBytes;
          const uint64_t da = tc::smem_desc(sa, a_mn), db = tc::smem_desc(sa + kABytes, b_mn);
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k)
            tc::mma_f16_pair(d, da + step_a * k, db + step_b * k, idesc, kb != tile.kb0 || k != 0);
          tc::mma_commit_pair(empty + 8 * stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (ok) tc::mma_commit_pair(tfull + 8 * buf);
        buf ^= 1;
        if (buf == 0) tphase ^= 1;
      }
    }
  } else {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    int buf = 0;
    uint32_t tphase = 0;
    for (int w = 0, t = cluster; t < g.total_tiles; t = tile_at(++w)) {
      const Tile tile = t == cluster ? first : decode<kTileN>(g, t);
      const bool idle = tile.half >= 0 && half == 1;  // four warps take half a tile
      const int row = tile.tm * kGemmTile + 128 * static_cast<int>(rank) + 32 * quad + lane;
      const int col0 = tile.tn * kTileN + kTileN / 2 * (tile.half >= 0 ? tile.half : half);
      if (!idle) Epi::template prepare<kTileN / 2>(g.epi[tile.problem], g.table, g.shape[tile.problem], tile, row, col0);
      ok = __all_sync(0xffffffffu, tc::mbar_wait(tfull + 8 * buf, tphase));
      if (!ok) break;
      tc::fence_after();
      const uint32_t addr = tmem + (static_cast<uint32_t>(32 * quad) << 16) + kTileN * buf + kTileN / 2 * half;
      const uint32_t bar = tempty + 8 * buf;
      const uint32_t turn = tmem_slot + 16 + (warp - 2) * kTurnBytes;
      auto release = [&]() {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster_relaxed(tc::map_to_rank(bar, 0));
      };
      if (idle)
        release();
      else
        Epi::template run<kTileN / 2>(g.epi[tile.problem], g.table, g.shape[tile.problem], tile, row, col0, addr, turn, release);
      buf ^= 1;
      if (buf == 0) tphase ^= 1;
    }
  }
  if (!ok) {
    // a wait ran out: loads and MMAs in flight get time to land before the CTA ends
    atomicExch(&g_gemm_error, 1);
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  tc::fence_before();
  __syncthreads();
  tc::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc::tmem_free_pair(tmem, kTmemColumns);
  }
}

// ---- host ------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// Tile of 64 contiguous elements x `rows` rows (K-major: 64 deep in K) or x 64
// rows (MN-major: 64 wide, 64 deep in K).
bool make_map(CUtensorMap* map, const GemmOperand& o, bool bf16, int rows) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.inner), static_cast<cuuint64_t>(o.outer),
                              static_cast<cuuint64_t>(o.batch)};
  const cuuint64_t pitch = static_cast<cuuint64_t>(o.pitch) * 2;
  const cuuint64_t strides[2] = {pitch, o.batch > 1 ? static_cast<cuuint64_t>(o.batch_pitch) * 2 : pitch};
  const cuuint32_t box[3] = {64u, o.transposed ? 64u : static_cast<cuuint32_t>(rows), 1u};
  const cuuint32_t one[3] = {1u, 1u, 1u};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void*>(o.ptr), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTA pairs of this kernel that can be resident at once; 0 when the query fails.
template <class Epi, bool kBf16, int kTileN>
int resident_pairs() {
  auto kernel = gemm_kernel<Epi, kBf16, kTileN>;
  constexpr int kSmemBytes = smem_bytes(kTileN);
  constexpr int kMaxDevices = 16;
  static std::mutex mu;
  static int cached[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev]) return cached[dev];
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) return 0;
  int sms = 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {2, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int pairs = 0;
  if (cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg) != cudaSuccess) return 0;
  return cached[dev] = pairs;
}

void set_params(StoreParams* e, Nothing*, const GemmProblem& p, const UpdateTable*) { *e = p.store; }
void set_params(GradParams* e, Nothing*, const GemmProblem& p, const UpdateTable*) { *e = {p.store, p.partial}; }
void set_params(XentParams* e, Nothing*, const GemmProblem& p, const UpdateTable*) { *e = p.xent; }
void set_params(WgradParams* e, Nothing*, const GemmProblem& p, const UpdateTable*) { *e = p.wgrad; }
void set_params(UpdateParams* e, UpdateTable* t, const GemmProblem& p, const UpdateTable* updates) {
  *e = p.update;
  for (int64_t i = p.update.first; i < p.update.first + p.batch; ++i) {
    t->w[i] = updates->w[i];
    t->w16[i] = updates->w16[i];
    t->step[i] = updates->step[i];
  }
}

template <class Epi, bool kBf16, int kTileN>
cudaError_t launch(const GemmProblem* problems, int count, cudaStream_t stream, const UpdateTable* updates) {
  auto kernel = gemm_kernel<Epi, kBf16, kTileN>;
  const int pairs = resident_pairs<Epi, kBf16, kTileN>();
  if (pairs <= 0) {
    const cudaError_t err = cudaGetLastError();
    return err != cudaSuccess ? err : cudaErrorInvalidDevice;
  }
  Args<Epi> g;
  int64_t total = 0;
  int used = 0;
  for (int i = 0; i < count; ++i) {
    const GemmProblem& p = problems[i];
    if (p.m <= 0 || p.n <= 0 || p.k <= 0 || p.batch <= 0) continue;
    Shape& s = g.shape[used];
    s.m = static_cast<int32_t>(p.m);
    s.n = static_cast<int32_t>(p.n);
    s.k_blocks = static_cast<int32_t>(ceil_div(p.k, kTileK));
    s.k_per_split = static_cast<int32_t>(ceil_div(s.k_blocks, p.splits));
    s.splits = static_cast<int32_t>(ceil_div(s.k_blocks, s.k_per_split));
    s.part_blocks = s.k_blocks / p.parts;
    s.tiles_m = static_cast<int32_t>(ceil_div(p.m, kGemmTile));
    s.tiles_n = static_cast<int32_t>(ceil_div(p.n, kTileN));
    s.symmetric = p.symmetric;
    s.a_mn = p.a.transposed;
    s.b_mn = p.b.transposed;
    s.tiles = s.tiles_m * s.tiles_n;
    if (p.symmetric) {
      s.tiles = 0;
      for (int i = 0; i < s.tiles_m; ++i) s.tiles += s.tiles_n - kGemmTile / kTileN * i;
    }
    s.first_tile = static_cast<int32_t>(total);
    total += static_cast<int64_t>(s.tiles) * s.splits * p.batch;
    if (total > INT32_MAX / 2) return cudaErrorInvalidValue;
    if (!make_map(&g.a[used], p.a, kBf16, 128) || !make_map(&g.b[used], p.b, kBf16, kTileN / 2) ||
        (kTileN == kGemmTile && !make_map(&g.b_half[used], p.b, kBf16, kTileN / 4)))
      return cudaErrorInvalidPitchValue;
    set_params(&g.epi[used], &g.table, p, updates);
    ++used;
  }
  if (used == 0) return cudaSuccess;
  g.count = used;
  g.mixed = 0;
  for (int i = 1; i < used; ++i) g.mixed |= g.shape[i].k_per_split != g.shape[0].k_per_split;
  const unsigned grid = 2u * static_cast<unsigned>(total < pairs ? total : pairs);
  // A last wave that leaves half of the pairs or more without a tile is formed of
  // half tiles: five symmetric products of 2048 x 2048 (2.4 waves) take 34.5 us so
  // and 38.3 with whole tiles. With more tiles left their halves would take two rounds.
  const int64_t left = total % pairs;
  const bool halves = kTileN == kGemmTile && total > pairs && 2 * left <= pairs;
  g.whole_tiles = static_cast<int32_t>(halves ? total - left : total);
  g.total_tiles = static_cast<int32_t>(halves ? total + left : total);
  return launch_chained(kernel, dim3(grid), dim3(kThreads), smem_bytes(kTileN), stream, g);
}

// Fewer 256 x 256 tiles than pairs: half as wide (see the top of the file).
template <class Epi, bool kBf16>
cudaError_t launch_fit(const GemmProblem* problems, int count, cudaStream_t stream, const UpdateTable* updates) {
  int64_t tiles = 0;
  for (int i = 0; i < count; ++i) {
    const GemmProblem& p = problems[i];
    const int64_t tm = ceil_div(p.m, kGemmTile), tn = ceil_div(p.n, kGemmTile);
    tiles += (p.symmetric ? tn * (tn + 1) / 2 : tm * tn) * p.batch * p.splits;
  }
  return tiles < 76 ? launch<Epi, kBf16, 128>(problems, count, stream, updates)
                    : launch<Epi, kBf16, 256>(problems, count, stream, updates);
}

}  // namespace

cudaError_t launch_gemm(GemmKind kind, const GemmProblem* p, int count, cudaStream_t stream, const UpdateTable* updates) {
  if (count > kGemmMaxProblems) return cudaErrorInvalidValue;
  switch (kind) {
    case GEMM_F16: return launch_fit<StoreEpilogue, false>(p, count, stream, nullptr);
    case GEMM_F16_UPDATE: return launch_fit<UpdateEpilogue, false>(p, count, stream, updates);
    case GEMM_BF16: return launch_fit<GradEpilogue, true>(p, count, stream, nullptr);
    // split sums fill the pairs with tiles of 128 columns (see lst_checkpoint.cu)
    case GEMM_BF16_WGRAD:
      return p->splits > 1 ? launch<WgradEpilogue, true, 128>(p, count, stream, nullptr)
                           : launch_fit<WgradEpilogue, true>(p, count, stream, nullptr);
    case GEMM_BF16_XENT: return launch<XentEpilogue, true, 256>(p, count, stream, nullptr);
    case GEMM_BF16_XENT_FEW:
      return p->n <= 32 ? launch<XentFewEpilogue, true, 32>(p, count, stream, nullptr)
                        : launch<XentFewEpilogue, true, 64>(p, count, stream, nullptr);
  }
  return cudaErrorInvalidValue;
}

// A split costs a partial sum to write and to read, and a whole sum on one pair
// may outlast everything else in the launch. Taken: the fewest splits with which
// a tile takes no more than half of a pair's share of the work (76 pairs).
int gemm_splits(int64_t tiles, int64_t k, int64_t others) {
  const int64_t blocks = ceil_div(k, kTileK), share = (tiles * blocks + others) / 76;
  int64_t s = 1;
  while (s < 32 && ceil_div(blocks, s) > std::max<int64_t>(share / 2, 8)) ++s;
  return static_cast<int>(ceil_div(blocks, ceil_div(blocks, s)));
}

cudaError_t gemm_take_error(int* out) {
  cudaError_t err = cudaMemcpyFromSymbol(out, g_gemm_error, sizeof(int));
  if (err != cudaSuccess || *out == 0) return err;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_gemm_error, &zero, sizeof(int));
}

}  // namespace lst
