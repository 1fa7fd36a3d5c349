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

// The larger of two magnitudes; a NaN if either is one.
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

// Eight elements of a block of 32, which lie on four neighbouring lanes that call together: the bytes q + 128 in w, the scale's
// bits returned.
//
// The scale is the smallest f16 h with 127 h >= the block's largest magnitude. The product with R, a little
// above 1/127, rounded up is that h or the f16 behind it, and 127 h is exact in f32 (18 bits), so one comparison
// decides. x / h by an approximate reciprocal is off by at most 127 (2^-23 + 2^-24) < 2.3e-5; only next to a half is the
// division needed to know the nearest integer q. 1.5 2^23 + 128 + q has q + 128 as its low byte.
// (With two IEEE divisions a block, a clamp and a test an element, key and value rows took most of the append kernel's issue
// slots: a prompt of 16,382 tokens, appended and read back, 142 us instead of 135.)
__device__ __forceinline__ uint32_t q8_block(const float (&y)[8], uint32_t (&w)[2]) {
  float top = fabsf(y[0]);  // an infinity or a NaN stays one
#pragma unroll
  for (int e = 1; e < 8; ++e) top = max_nan(top, fabsf(y[e]));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
  constexpr float R = 0x1.02040cp-7f;
  uint32_t bits = __half_as_ushort(__float2half_ru(top * R));
  if (127.f * __half2float(__ushort_as_half(bits - 1)) >= top) --bits;  // (false for 0 - 1, a NaN)
  const bool bad = !(top <= 3.402823466e38f), high = bits > 0x7BFF;
  if (high) bits = 0x7BFF;
  if (bad) bits = 0x7FFF;
  w[0] = w[1] = 0x80808080u;
  if (!bad && bits != 0) {
    const float ds = __half2float(__ushort_as_half(bits)), magic = 12582912.f + 128.f;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(ds));
    float b[8], off = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 q = mul2(make_float2(y[e], y[e + 1]), make_float2(inv, inv));
      const float2 m = sub2(q, make_float2(-magic, -magic));
      const float2 r = sub2(q, sub2(m, make_float2(magic, magic)));
      off = fmaxf(off, fmaxf(fabsf(r.x), fabsf(r.y)));
      b[e] = m.x;
      b[e + 1] = m.y;
    }
    if (off > 0.49996f || high)
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
