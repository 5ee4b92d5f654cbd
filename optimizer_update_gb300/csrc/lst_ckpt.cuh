// Device side of 8-bit activation checkpoints and of rows held by a group of
// threads, shared by the residual-norm and checkpoint kernels.
//
// A checkpoint keeps a row in blocks of 32 values. A block has a scale 2^k, the
// smallest with max|x| <= M 2^k (M the largest stored magnitude: 127 for signed
// integers, 448 for e4m3), kept as the byte k + 127, and its values are
// x 2^-k rounded to nearest, ties to even. Powers of two make the division exact
// and the result independent of the order of operations: a restored value is off
// by half a step of the stored type and nothing else (integers: 2^-7 of the
// block's largest magnitude at most; e4m3: 2^-4 of the value). Integers are 3
// times nearer for values of one size (RMS error of normal values 0.8 % against
// 2.7 %), e4m3 keeps the small values beside large ones.
// A block with an infinity or NaN has the byte 255 and restores as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "lst_ops.h"

namespace lst {

constexpr int kCkptBlock = 32;

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Scale byte of a block whose largest magnitude has the bits `most`: the exponent
// is that of `most` less M's, one more where its fraction is above M's. Blocks below
// 127 or 448 times 2^-127 take the smallest scale.
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t most, bool e4m3) {
  if (most >= 0x7f800000u) return 255u;
  const uint32_t up = e4m3 ? 0x7fffffu - 0x600000u : 0x7fffffu - 0x7e0000u;
  return static_cast<uint32_t>(max(static_cast<int>((most + up) >> 23) - (e4m3 ? 8 : 6), 0));
}
// 2^-k (k >= -127, so never subnormal) for a byte below 255.
__device__ __forceinline__ float ckpt_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
// 2^k; NaN for the byte 255.
__device__ __forceinline__ float ckpt_step(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7fffffffu : byte << 23);
}

// The integer nearest to v (|v| < 2^22, ties to even) in the low bits of the sum.
__device__ __forceinline__ uint32_t ckpt_round_i8(float v) { return __float_as_uint(v + 12582912.0f); }

// Four values divided by their step, as bytes.
__device__ __forceinline__ uint32_t ckpt_encode4(float2 a, float2 b, bool e4m3) {
  if (e4m3) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    return lo | static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  const uint32_t lo = __byte_perm(ckpt_round_i8(a.x), ckpt_round_i8(a.y), 0x0040);
  const uint32_t hi = __byte_perm(ckpt_round_i8(b.x), ckpt_round_i8(b.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ void ckpt_decode4(uint32_t w, bool e4m3, float2& a, float2& b) {
  if (e4m3) {
    a = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3)));
    b = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3)));
    return;
  }
  // byte + 128 in the mantissa of 2^23
  w ^= 0x80808080u;
  const float2 off = both(-8388736.0f);
  a = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)), __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))), off);
  b = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)), __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443))), off);
}

__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ float2 round_to(float2 v, const float*) { return v; }
__device__ __forceinline__ float2 round_to(float2 v, const __nv_bfloat16*) { return unpack_bf16(pack_bf16(v)); }

// Values of a row in a thread: a unit of eight, or half of one.
template <int P>
struct Part {
  float2 v[P];
  __device__ __forceinline__ float& at(int i) { return i & 1 ? v[i >> 1].y : v[i >> 1].x; }
  __device__ __forceinline__ float at(int i) const { return i & 1 ? v[i >> 1].y : v[i >> 1].x; }
  __device__ __forceinline__ void fill(float s) {
#pragma unroll
    for (int j = 0; j < P; ++j) v[j] = both(s);
  }
};
using Unit = Part<4>;
using Half = Part<2>;

// A row of `cols` values held in units by `threads` threads (a multiple of 32). On the
// vector path (rows on 16 bytes, a multiple of 8 columns) a unit is 8 consecutive
// columns, otherwise every `threads`-th one, so that a warp's accesses stay
// consecutive. Either way a checkpoint's block of 32 lies inside one warp: in 4
// neighbouring lanes, or in all 32. Columns behind the last read as zero, but on the
// vector path units are whole or not there at all: callers pass over those (`has`).
template <bool VEC>
struct Cols {
  uint32_t tid, threads, cols;
  __device__ __forceinline__ uint32_t at(int k, int i) const {
    return VEC ? (tid + k * threads) * 8 + i : tid + (8 * k + i) * threads;
  }
  __device__ __forceinline__ bool in(int k, int i) const { return at(k, VEC ? 0 : i) < cols; }
  __device__ __forceinline__ bool has(int k) const { return !VEC || at(k, 0) < cols; }

  // f(i, column, inside the row) for the values of a part
  template <int P, class F>
  __device__ __forceinline__ void each(int k, int i0, F f) const {
    uint32_t e = at(k, i0);
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) {
      f(i, e, e < cols);
      e += VEC ? 1u : threads;
    }
  }
  // Unit k, or the half of it from its value `i0` on.
  template <int P>
  __device__ __forceinline__ void load(const float* p, int k, Part<P>& u, int i0 = 0) const {
    if (VEC) {
#pragma unroll
      for (int j = 0; j < P; j += 2) {
        const float4 a = *reinterpret_cast<const float4*>(p + at(k, i0 + 2 * j));
        u.v[j] = make_float2(a.x, a.y), u.v[j + 1] = make_float2(a.z, a.w);
      }
    } else {
      each<P>(k, i0, [&](int i, uint32_t e, bool inside) { u.at(i) = inside ? p[e] : 0.0f; });
    }
  }
  template <int P>
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int k, Part<P>& u, int i0 = 0) const {
    if (VEC && P == 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(p + at(k, 0));
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int j = 0; j < P; ++j) u.v[j] = unpack_bf16(w[j & 3]);
    } else if (VEC) {
      const uint2 a = *reinterpret_cast<const uint2*>(p + at(k, i0));
      u.v[0] = unpack_bf16(a.x), u.v[1] = unpack_bf16(a.y);
    } else {
      each<P>(k, i0, [&](int i, uint32_t e, bool inside) { u.at(i) = inside ? __bfloat162float(p[e]) : 0.0f; });
    }
  }
  template <int P>
  __device__ __forceinline__ void store(float* p, int k, const Part<P>& u, int i0 = 0) const {
    if (VEC) {
#pragma unroll
      for (int j = 0; j < P; j += 2)
        *reinterpret_cast<float4*>(p + at(k, i0 + 2 * j)) = make_float4(u.v[j].x, u.v[j].y, u.v[j + 1].x, u.v[j + 1].y);
    } else {
      each<P>(k, i0, [&](int i, uint32_t e, bool inside) {
        if (inside) p[e] = u.at(i);
      });
    }
  }
  template <int P>
  __device__ __forceinline__ void store(__nv_bfloat16* p, int k, const Part<P>& u, int i0 = 0) const {
    if (VEC && P == 4) {
      *reinterpret_cast<uint4*>(p + at(k, 0)) =
          make_uint4(pack_bf16(u.v[0]), pack_bf16(u.v[1]), pack_bf16(u.v[2 % P]), pack_bf16(u.v[3 % P]));
    } else if (VEC) {
      *reinterpret_cast<uint2*>(p + at(k, i0)) = make_uint2(pack_bf16(u.v[0]), pack_bf16(u.v[1]));
    } else {
      each<P>(k, i0, [&](int i, uint32_t e, bool inside) {
        if (inside) p[e] = __float2bfloat16_rn(u.at(i));
      });
    }
  }
  // Weights of either type, on any alignment.
  template <class T, int P>
  __device__ __forceinline__ void load_weights(const T* p, int k, Part<P>& u, int i0) const {
    if (VEC && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
      load(p, k, u, i0);
    } else {
      each<P>(k, i0, [&](int i, uint32_t e, bool inside) { u.at(i) = inside ? static_cast<float>(p[e]) : 0.0f; });
    }
  }
  template <int P>
  __device__ __forceinline__ void load_any(const void* p, bool f32, int k, Part<P>& u, int i0 = 0) const {
    if (f32)
      load_weights(static_cast<const float*>(p), k, u, i0);
    else
      load_weights(static_cast<const __nv_bfloat16*>(p), k, u, i0);
  }

  // Unit k to and from a checkpoint's row. All threads of a warp save together, units that
  // are not there holding zeros.
  __device__ __forceinline__ void save(const Unit& u, int k, uint8_t* data, uint8_t* scales, bool e4m3) const {
    if (VEC) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(u.at(i)) & 0x7fffffffu);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const uint32_t byte = ckpt_scale_byte(most, e4m3);
      const float2 r = both(ckpt_inverse(min(byte, 254u)));
      uint2 w;
      if (e4m3)
        w = make_uint2(ckpt_encode4(mul2(u.v[0], r), mul2(u.v[1], r), true), ckpt_encode4(mul2(u.v[2], r), mul2(u.v[3], r), true));
      else
        w = make_uint2(ckpt_encode4(mul2(u.v[0], r), mul2(u.v[1], r), false), ckpt_encode4(mul2(u.v[2], r), mul2(u.v[3], r), false));
      if (byte == 255u) w = make_uint2(0, 0);
      if (in(k, 0)) {
        *reinterpret_cast<uint2*>(data + at(k, 0)) = w;
        if ((tid & 3) == 0) scales[at(k, 0) / kCkptBlock] = static_cast<uint8_t>(byte);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(u.at(i)) & 0x7fffffffu);
        const uint32_t byte = ckpt_scale_byte(most, e4m3);
        const float q = byte == 255u ? 0.0f : u.at(i) * ckpt_inverse(byte);
        if (in(k, i)) {
          data[at(k, i)] = static_cast<uint8_t>(ckpt_encode4(both(q), both(q), e4m3));
          if ((tid & 31) == 0) scales[at(k, i) / kCkptBlock] = static_cast<uint8_t>(byte);
        }
      }
    }
  }
  template <int P>
  __device__ __forceinline__ void restore(const uint8_t* data, const uint8_t* scales, bool e4m3, int k, Part<P>& u, int i0 = 0) const {
    if (VEC) {
      uint32_t w[2];
      if (P == 4) {
        const uint2 q = *reinterpret_cast<const uint2*>(data + at(k, 0));
        w[0] = q.x, w[1] = q.y;
      } else {
        w[0] = w[1] = *reinterpret_cast<const uint32_t*>(data + at(k, i0));
      }
      const bool there = has(k);  // bytes behind the row may be anything
      const float step = there ? ckpt_step(scales[at(k, 0) / kCkptBlock]) : 0.0f;
      w[0] = there ? w[0] : 0u, w[1] = there ? w[1] : 0u;
#pragma unroll
      for (int j = 0; j < P; j += 2) ckpt_decode4(w[j >> 1], e4m3, u.v[j], u.v[j + 1]);
#pragma unroll
      for (int j = 0; j < P; ++j) u.v[j] = mul2(u.v[j], both(step));
    } else {
      each<P>(k, i0, [&](int i, uint32_t e, bool inside) {
        float2 a = both(0.0f), b;
        float step = 0.0f;
        if (inside) {
          ckpt_decode4(data[e], e4m3, a, b);
          step = ckpt_step(scales[e / kCkptBlock]);
        }
        u.at(i) = a.x * step;
      });
    }
  }
};

}  // namespace lst
