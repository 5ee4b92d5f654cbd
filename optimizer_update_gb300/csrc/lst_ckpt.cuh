// Device side of 8-bit activation checkpoints and of rows held by a group of
// threads, shared by the residual-norm and checkpoint kernels.
//
// A checkpoint keeps a row in blocks of 32 values. A block has a scale 2^k, the
// smallest with max|x| <= M 2^k (M the largest stored magnitude: 127 for signed
// integers, 448 for e4m3), kept as the byte k + 127, and its values are
// x 2^-k rounded to nearest, ties to even. Powers of two make the division exact
// and the result independent of the order of operations: a restored value is off
// by half a step of the stored type and nothing else (integers: 2^-8 of the
// block's largest magnitude at most; e4m3: 2^-4 of the value). Integers are 2 to 3
// times nearer for values of one size (block RMS error of normal values 0.7 %
// against 2.3 %), e4m3 keeps the small values beside large ones.
// A block with an infinity or NaN has the byte 255 and restores as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "lst_ops.h"

namespace lst {

constexpr int kCkptBlock = 32;

// Scale byte of a block whose largest magnitude has the bits `most`: the exponent
// is that of `most` less M's, one more where its fraction is above M's. Blocks below
// 127 or 448 times 2^-127 take the smallest scale.
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t most, bool e4m3) {
  if (most >= 0x7f800000u) return 255u;
  const uint32_t up = e4m3 ? 0x7fffffu - 0x600000u : 0x7fffffu - 0x7e0000u;
  return static_cast<uint32_t>(max(static_cast<int>((most + up) >> 23) - (e4m3 ? 8 : 6), 0));
}
// 2^-k (k >= -127, so never subnormal); 0 for the byte 255, whose values are stored as 0.
__device__ __forceinline__ float ckpt_inverse(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^k; NaN for the byte 255.
__device__ __forceinline__ float ckpt_step(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}

// The integer nearest to v (|v| < 2^22, ties to even) in the low bits of the sum.
__device__ __forceinline__ uint32_t ckpt_round_i8(float v) { return __float_as_uint(v + 12582912.0f); }

// Four values divided by their step, as bytes.
__device__ __forceinline__ uint32_t ckpt_encode4(float a, float b, float c, float d, bool e4m3) {
  if (e4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    return lo | static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  const uint32_t lo = __byte_perm(ckpt_round_i8(a), ckpt_round_i8(b), 0x0040);
  const uint32_t hi = __byte_perm(ckpt_round_i8(c), ckpt_round_i8(d), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ void ckpt_decode4(uint32_t w, bool e4m3, float& a, float& b, float& c, float& d) {
  if (e4m3) {
    const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3)));
    const float2 hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3)));
    a = lo.x, b = lo.y, c = hi.x, d = hi.y;
    return;
  }
  // byte + 128 in the mantissa of 2^23
  w ^= 0x80808080u;
  a = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)) - 8388736.0f;
  b = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441)) - 8388736.0f;
  c = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)) - 8388736.0f;
  d = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443)) - 8388736.0f;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) { return __bfloat162float(__float2bfloat16_rn(v)); }

// A row of `cols` values held by `threads` threads (a multiple of 32), 8 K each. On the
// vector path (rows on 16 bytes, a multiple of 8 columns) a thread has K groups of 8
// consecutive columns, otherwise every `threads`-th column, so that a warp's
// accesses stay consecutive. Either way a checkpoint's block of 32 lies inside one
// warp: in 4 neighbouring lanes, or in all 32. Columns behind the last read as zero.
template <bool VEC, int K>
struct Cols {
  int tid, threads, cols;
  __device__ __forceinline__ int at(int k, int i) const {
    return VEC ? (tid + k * threads) * 8 + i : tid + (8 * k + i) * threads;
  }
  __device__ __forceinline__ bool in(int k, int i) const { return at(k, VEC ? 0 : i) < cols; }

  __device__ __forceinline__ void load(const float* p, float (&v)[K][8]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC) {
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (in(k, 0)) {
          a = *reinterpret_cast<const float4*>(p + at(k, 0));
          b = *reinterpret_cast<const float4*>(p + at(k, 4));
        }
        v[k][0] = a.x, v[k][1] = a.y, v[k][2] = a.z, v[k][3] = a.w, v[k][4] = b.x, v[k][5] = b.y, v[k][6] = b.z, v[k][7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = in(k, i) ? p[at(k, i)] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[K][8]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (in(k, 0)) a = *reinterpret_cast<const uint4*>(p + at(k, 0));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[k][2 * i] = __uint_as_float(w[i] << 16);
          v[k][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = in(k, i) ? __bfloat162float(p[at(k, i)]) : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void store(float* p, const float (&v)[K][8]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC) {
        if (in(k, 0)) {
          *reinterpret_cast<float4*>(p + at(k, 0)) = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
          *reinterpret_cast<float4*>(p + at(k, 4)) = make_float4(v[k][4], v[k][5], v[k][6], v[k][7]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (in(k, i)) p[at(k, i)] = v[k][i];
      }
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[K][8]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC) {
        if (in(k, 0))
          *reinterpret_cast<uint4*>(p + at(k, 0)) = make_uint4(pack_bf16(v[k][0], v[k][1]), pack_bf16(v[k][2], v[k][3]),
                                                               pack_bf16(v[k][4], v[k][5]), pack_bf16(v[k][6], v[k][7]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (in(k, i)) p[at(k, i)] = __float2bfloat16_rn(v[k][i]);
      }
    }
  }
  // A row of weights of either type, on any alignment.
  __device__ __forceinline__ void load_any(const void* p, bool f32, float (&v)[K][8]) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[k][i] = !in(k, i) ? 0.0f
                  : f32     ? static_cast<const float*>(p)[at(k, i)]
                            : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at(k, i)]);
  }

  // All threads of the warps call these two.
  __device__ __forceinline__ void save(const float (&v)[K][8], uint8_t* data, uint8_t* scales, bool e4m3) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[k][i]) & 0x7fffffffu);
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        const uint32_t byte = ckpt_scale_byte(most, e4m3);
        const float r = ckpt_inverse(byte);
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = byte == 255u ? 0.0f : v[k][i] * r;
        if (in(k, 0)) {
          *reinterpret_cast<uint2*>(data + at(k, 0)) =
              make_uint2(ckpt_encode4(q[0], q[1], q[2], q[3], e4m3), ckpt_encode4(q[4], q[5], q[6], q[7], e4m3));
          if ((tid & 3) == 0) scales[at(k, 0) / kCkptBlock] = static_cast<uint8_t>(byte);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(v[k][i]) & 0x7fffffffu);
          const uint32_t byte = ckpt_scale_byte(most, e4m3);
          const float q = byte == 255u ? 0.0f : v[k][i] * ckpt_inverse(byte);
          if (in(k, i)) {
            data[at(k, i)] = static_cast<uint8_t>(ckpt_encode4(q, 0.0f, 0.0f, 0.0f, e4m3));
            if ((tid & 31) == 0) scales[at(k, i) / kCkptBlock] = static_cast<uint8_t>(byte);
          }
        }
      }
    }
  }
  __device__ __forceinline__ void restore(const uint8_t* data, const uint8_t* scales, bool e4m3, float (&v)[K][8]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (VEC) {
        uint2 w = make_uint2(0, 0);
        float step = 0.0f;
        if (in(k, 0)) {
          w = *reinterpret_cast<const uint2*>(data + at(k, 0));
          step = ckpt_step(scales[at(k, 0) / kCkptBlock]);
        }
        ckpt_decode4(w.x, e4m3, v[k][0], v[k][1], v[k][2], v[k][3]);
        ckpt_decode4(w.y, e4m3, v[k][4], v[k][5], v[k][6], v[k][7]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * step;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[k][i] = 0.0f;
          if (in(k, i)) {
            float b, c, d;
            ckpt_decode4(data[at(k, i)], e4m3, v[k][i], b, c, d);
            v[k][i] = v[k][i] * ckpt_step(scales[at(k, i) / kCkptBlock]);
          }
        }
      }
    }
  }
};

}  // namespace lst
