// qg_blocks.cuh -- eight neighbouring elements of a row: loads, stores, and Q8_0 blocks made of f32 values (the rotary and
// cache calls, qg_rope.cu; normed rows, qg_norm.cu; looked-up rows, qg_embed.cu).
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

#include "qg_common.cuh"

namespace qg {

// Eight consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// The larger or smaller of two numbers, the largest magnitude, number or smallest number of three; a NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float abs_max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// x / d as the division rounds it, d an f16, inv 1 / d to 2^-23: a quotient and what it leaves. The remainder is exact (its multiples of
// 2^-35 of x reach 2^-22), the corrected quotient off by less than 2^-44 before it is rounded; and no f32 over an 11-bit d lies
// closer than 2^-36 to the middle between two f32.
__device__ __forceinline__ float2 quotients(float2 x, float d, float inv) {
  const float2 q = mul2(x, make_float2(inv, inv));
  return fma2(fma2(q, make_float2(-d, -d), x), make_float2(inv, inv), q);
}

// Eight elements of a block of 32, which lie on four neighbouring lanes that call together: the bytes q + BIAS (128, or 0: signed)
// in w, the scale's bits returned.
//
// The scale is the smallest f16 h with 127 h >= the block's largest magnitude. The product with R, a little
// above 1/127, rounded up is that h or the f16 behind it, and 127 h is exact in f32 (18 bits), so one comparison
// decides. 1.5 2^23 + BIAS + q, q rounded to the nearest integer as it is added, has q + BIAS as its low byte.
// (With two IEEE divisions a block, a clamp and a test an element, key and value rows took most of the append kernel's issue
// slots: a prompt of 16,382 tokens, appended and read back, 142 us instead of 135.)
//
// TAME: of blocks whose largest magnitude, returned in top, is not above Q8_TOP (others come out wrong, and are made again), without
// branches, so that several blocks' instructions mix.
constexpr float Q8_TOP = 127.f * 65504.f;
template <int BIAS, bool TAME>
__device__ __forceinline__ uint32_t q8_block(const float (&y)[8], uint32_t (&w)[2], float& top) {
  // (an infinity or a NaN stays one)
  top = abs_max_nan(abs_max_nan(y[0], y[1], y[2]), abs_max_nan(y[3], y[4], y[5]), abs_max_nan(y[6], y[7], y[7]));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
  constexpr float R = 0x1.02040cp-7f;
  uint32_t bits = __half_as_ushort(__float2half_ru(top * R));
  if (127.f * __half2float(__ushort_as_half(bits - 1)) >= top) --bits;  // (false for 0 - 1, a NaN)
  const bool bad = !TAME && !(top <= 3.402823466e38f), high = !TAME && bits > 0x7BFF;
  if (high) bits = 0x7BFF;
  if (bad) bits = 0x7FFF;
  w[0] = w[1] = BIAS * 0x01010101u;
  if (TAME || (!bad && bits != 0)) {
    const float ds = __half2float(__ushort_as_half(bits)), magic = 12582912.f + (float)BIAS;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(TAME ? fmaxf(ds, 0x1p-24f) : ds));
    float b[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 m = sub2(quotients(make_float2(y[e], y[e + 1]), ds, inv), make_float2(-magic, -magic));
      b[e] = m.x;
      b[e + 1] = m.y;
    }
    if (high)
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = fminf(fmaxf(__fdiv_rn(y[e], ds), -127.f), 127.f) + magic;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = __byte_perm(__byte_perm(__float_as_uint(b[4 * h]), __float_as_uint(b[4 * h + 1]), 0x0040),
                         __byte_perm(__float_as_uint(b[4 * h + 2]), __float_as_uint(b[4 * h + 3]), 0x0040), 0x5410);
  }
  return bits;
}

}  // namespace qg
