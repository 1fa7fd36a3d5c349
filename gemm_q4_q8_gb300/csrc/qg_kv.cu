// qg_kv.cu -- the paged key/value cache read back (qkv_read): a warp owns a
// token, eight consecutive elements a lane as in qg_rope.cu, and walks over the
// key rows, then the value rows. A Q8_0 element is (quant - 128) * scale, exact
// in f32 (an 8-bit integer times an 11-bit significand), rounded once for f16. A Q4_1
// element is quant * d + m, rounded once.
//
// Bound by memory: 2 (f16) or 17/16 (Q8_0) bytes read an element, 2 or 4 written.
// 32,767 f16 tokens of 8 heads of 128 (268 MB moved): 44.5 us, 6.0 TB/s. Q4_1 to f16 by its instructions, 70% of the issue slots
// used: 16,382 tokens (88 MB) in 20.1 us; six or eight rows in flight 22.7 to 28.9.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_kv.cuh"

namespace qg {

namespace {

// 32,767 f16 tokens of 8 heads of 128: 44.5 us with blocks of four warps, 44.9 with eight. 47.4 with eight rows in flight, 50
// with two, 49 with two warps a token. Warps that take several tokens in turn and look the next page up ahead: 43.2, but
// 9,800 tokens 16.9 instead of 16.2 and 3,000 6.45 instead of 6.1.
constexpr int RD_THREADS = 128;
constexpr int RD_WARPS = RD_THREADS / 32;
constexpr int RD_UNROLL = 4;  // rows that a lane has in flight

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void write8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void write8(__half* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(half2_bits(v[0], v[1]), half2_bits(v[2], v[3]),
                                            half2_bits(v[4], v[5]), half2_bits(v[6], v[7]));
}

template <int TYPE, class TO>
__global__ void __launch_bounds__(RD_THREADS)
    kv_read_kernel(const __grid_constant__ qg_kvcache c, const int32_t* seqs, const int32_t* poss,
                   int ntok, int per_seq, TO* k_out, TO* v_out, int32_t* err, int parts) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * RD_WARPS + (threadIdx.x >> 5);
  const int64_t tok = w / parts;
  if (tok >= ntok) return;
  const int part = (int)(w - tok * parts);
  const int d = c.head_dim, lanes = d >> 3, at_once = 32 / lanes;
  const int d0 = (lane & (lanes - 1)) * 8, first = lane / lanes;
  const int groups = c.page_size / KV_GROUP, head_bytes = groups * kv_record_bytes(TYPE, d);
  const int pos = poss[tok];
  const uint8_t* place = nullptr;
  if (pos >= 0) {
    int bits = 0;
    const int seq = seqs ? seqs[tok] : (int)(tok / per_seq);
    const int page = kv_page_of(c, seq, pos, &bits);
    const int slot = pos & (c.page_size - 1);
    if (page >= 0)
      place = static_cast<const uint8_t*>(c.pool) + (size_t)page * c.n_kv_heads * head_bytes +
              slot / KV_GROUP * kv_record_bytes(TYPE, d);
    else if (part == 0 && lane == 0 && err)
      atomicOr(err, bits);
  }
  // this lane's eight elements of a half record, and their scale
  const int i = pos & (KV_GROUP - 1), blk = d0 >> 5;
  const int at = (blk * (KV_GROUP * 32) + i * 32 + (d0 & 31)) * (TYPE == QG_F16 ? 4 : TYPE == QG_Q8_0 ? 2 : 1) / 2;
  const int scale_at = KV_GROUP * d + (blk * KV_GROUP + kv_scale_place(i)) * 2;
  const int kv = c.n_kv_heads, kg = (kv + at_once - 1) / at_once;  // row groups: keys, then values
  TO* const ko = k_out ? k_out + tok * kv * d + d0 : nullptr;
  TO* const vo = v_out ? v_out + tok * kv * d + d0 : nullptr;
  for (int n = part; n < 2 * kg; n += RD_UNROLL * parts) {
    uint4 q[RD_UNROLL];
    uint16_t sc[RD_UNROLL];
    TO* to[RD_UNROLL];
#pragma unroll
    for (int j = 0; j < RD_UNROLL; ++j) {
      const int m = n + j * parts;
      const bool is_v = m >= kg;
      const int r = (is_v ? m - kg : m) * at_once + first;
      TO* const out = is_v ? vo : ko;
      to[j] = m < 2 * kg && r < kv && out ? out + r * d : nullptr;
      q[j] = TYPE == QG_Q8_0 ? make_uint4(0x80808080u, 0x80808080u, 0, 0) : make_uint4(0, 0, 0, 0);
      sc[j] = 0;
      if (place && to[j]) {
        const uint8_t* half = place + (size_t)((uint32_t)r * (uint32_t)head_bytes + (is_v ? kv_half_bytes(TYPE, d) : 0));
        if constexpr (TYPE == QG_F16) {
          q[j] = *reinterpret_cast<const uint4*>(half + at);
        } else if constexpr (TYPE == QG_Q4_1) {
          const uint8_t* const d_at = half + 8 * d + 2 * kv_q4_place(is_v, d, blk, i);
          q[j].x = *reinterpret_cast<const uint32_t*>(half + at);
          sc[j] = *reinterpret_cast<const uint16_t*>(d_at);
          q[j].y = *reinterpret_cast<const uint16_t*>(d_at + d);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(half + at);
          q[j].x = x.x;
          q[j].y = x.y;
          sc[j] = *reinterpret_cast<const uint16_t*>(half + scale_at);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RD_UNROLL; ++j) {
      if (!to[j]) continue;
      if constexpr (TYPE == QG_F16 && sizeof(TO) == 2) {
        *reinterpret_cast<uint4*>(to[j]) = q[j];
        continue;
      }
      if constexpr (TYPE == QG_Q8_0 && sizeof(TO) == 2) {
        // f16 1024 + u, less 1152, is the integer q exactly, and q * d is rounded once: the same as through f32
        const __half2 s = __half2half2(__ushort_as_half(sc[j]));
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const uint32_t u = __byte_perm(h < 2 ? q[j].x : q[j].y, 0x64646464u, h & 1 ? 0x4342 : 0x4140);
          const __half2 v = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480))), s);
          w[h] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(to[j]) = make_uint4(w[0], w[1], w[2], w[3]);
        continue;
      }
      if constexpr (TYPE == QG_Q4_1) {
        // pairs of quants as f16 1024 + q, less 1024; quant * d + m has one rounding
        __half2 h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t u = ((k & 2 ? q[j].x >> 4 : q[j].x) >> (k & 1 ? 8 : 0) & 0x000F000Fu) | 0x64006400u;
          h[k] = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6400)));
        }
        if constexpr (sizeof(TO) == 2) {
          const __half2 s = __half2half2(__ushort_as_half(sc[j])), m = __half2half2(__ushort_as_half((uint16_t)q[j].y));
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = __hfma2(h[k], s, m);
          *reinterpret_cast<uint4*>(to[j]) = *reinterpret_cast<const uint4*>(h);
        } else {
          const float s = h2f(sc[j]), m = h2f((uint16_t)q[j].y);
          float y[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(h[k]);
            y[2 * k] = fmaf(f.x, s, m);
            y[2 * k + 1] = fmaf(f.y, s, m);
          }
          write8(to[j], y);
        }
        continue;
      }
      float y[8];
      if constexpr (TYPE == QG_F16) {
        const uint32_t u[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
          y[2 * e] = f.x;
          y[2 * e + 1] = f.y;
        }
      } else {
        // u = q + 128 as the low byte of the float 2^23 + u, exact
        const float s = h2f(sc[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          y[e] = (u2f(__byte_perm(e < 4 ? q[j].x : q[j].y, MAGIC_2P23, 0x7440 + (e & 3))) - (F_2P23 + 128.f)) * s;
      }
      write8(to[j], y);
    }
  }
}

template <int TYPE, class TO>
cudaError_t read_typed(const qg_kvcache& c, const int32_t* seq, const int32_t* pos, int ntok,
                       void* k_out, void* v_out, int32_t* err, cudaStream_t s) {
  const int at_once = 256 / c.head_dim;
  const int groups = 2 * ((c.n_kv_heads + at_once - 1) / at_once);
  // a token's rows are spread over several warps while there are fewer tokens than fill the machine
  int parts = (152 * 40 + ntok - 1) / ntok;
  if (parts > groups) parts = groups;
  const int64_t warps = (int64_t)ntok * parts;
  return launch_pdl(kv_read_kernel<TYPE, TO>, dim3((unsigned)((warps + RD_WARPS - 1) / RD_WARPS)),
                    dim3(RD_THREADS), 0, s, 0, LC_L1, c, seq, pos, ntok, seq ? 1 : ntok / c.n_seq,
                    static_cast<TO*>(k_out), static_cast<TO*>(v_out), err, parts);
}

}  // namespace

cudaError_t kv_read_launch(const qg_kvcache& c, const int32_t* seq, const int32_t* pos, int ntok,
                           int yt, void* k_out, void* v_out, int32_t* err, cudaStream_t s) {
  if (c.type == QG_F16)
    return yt == QG_F32 ? read_typed<QG_F16, float>(c, seq, pos, ntok, k_out, v_out, err, s)
                        : read_typed<QG_F16, __half>(c, seq, pos, ntok, k_out, v_out, err, s);
  if (c.type == QG_Q4_1)
    return yt == QG_F32 ? read_typed<QG_Q4_1, float>(c, seq, pos, ntok, k_out, v_out, err, s)
                        : read_typed<QG_Q4_1, __half>(c, seq, pos, ntok, k_out, v_out, err, s);
  return yt == QG_F32 ? read_typed<QG_Q8_0, float>(c, seq, pos, ntok, k_out, v_out, err, s)
                      : read_typed<QG_Q8_0, __half>(c, seq, pos, ntok, k_out, v_out, err, s);
}

}  // namespace qg
