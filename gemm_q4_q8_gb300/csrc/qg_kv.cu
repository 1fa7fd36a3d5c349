// qg_kv.cu -- the paged key/value cache read back (qkv_read): a warp owns a
// token, eight consecutive elements a lane as in qg_rope.cu, and walks over the
// key rows, then the value rows. A Q8_0 element is (quant - 128) * scale, exact
// in f32 (an 8-bit integer times an 11-bit significand), rounded once for f16.
//
// Bound by memory: 2 (f16) or 17/16 (Q8_0) bytes read an element, 2 or 4 written.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_kv.cuh"

namespace qg {

namespace {

constexpr int RD_THREADS = 256;
constexpr int RD_WARPS = RD_THREADS / 32;

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
                   int ntok, int per_seq, TO* k_out, TO* v_out, int32_t* err, int parts, int per_part) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * RD_WARPS + (threadIdx.x >> 5);
  const int64_t tok = w / parts;
  if (tok >= ntok) return;
  const int part = (int)(w - tok * parts);
  const int d = c.head_dim, lanes = d >> 3, at_once = 32 / lanes;
  const int d0 = (lane & (lanes - 1)) * 8;
  const int groups = c.page_size / KV_GROUP, rec = kv_record_bytes(TYPE, d);
  const int pos = poss[tok];
  const uint8_t* place = nullptr;
  if (pos >= 0) {
    int bits = 0;
    const int seq = seqs ? seqs[tok] : (int)(tok / per_seq);
    const int page = kv_page_of(c, seq, pos, &bits);
    const int slot = pos & (c.page_size - 1);
    if (page >= 0)
      place = static_cast<const uint8_t*>(c.pool) +
              ((size_t)page * c.n_kv_heads * groups + slot / KV_GROUP) * rec;
    else if (part == 0 && lane == 0 && err)
      atomicOr(err, bits);
  }
  const int i = pos & (KV_GROUP - 1);
  const int kv = c.n_kv_heads;
  const int r0 = part * per_part * at_once + lane / lanes;
#pragma unroll 4
  for (int n = 0; n < per_part; ++n) {
    const int r = r0 + n * at_once;
    if (r >= 2 * kv) break;
    const bool is_k = r < kv;
    const int head = is_k ? r : r - kv;
    TO* out = is_k ? k_out : v_out;
    if (!out) continue;
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (place) {
      const uint8_t* half = place + (size_t)head * groups * rec + (is_k ? 0 : kv_half_bytes(TYPE, d));
      const int blk = d0 >> 5, at = blk * (KV_GROUP * 32) + i * 32 + (d0 & 31);
      if constexpr (TYPE == QG_F16) {
        const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const __half*>(half) + at);
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
          y[2 * e] = f.x;
          y[2 * e + 1] = f.y;
        }
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(half + at);
        const float s = h2f(reinterpret_cast<const uint16_t*>(half + KV_GROUP * d)[blk * KV_GROUP + kv_scale_place(i)]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t b = ((e < 4 ? q.x : q.y) >> (8 * (e & 3))) & 0xffu;
          y[e] = (float)((int)b - 128) * s;
        }
      }
    }
    write8(out + (tok * kv + head) * (int64_t)d + d0, y);
  }
}

template <int TYPE, class TO>
cudaError_t read_typed(const qg_kvcache& c, const int32_t* seq, const int32_t* pos, int ntok,
                       void* k_out, void* v_out, int32_t* err, cudaStream_t s) {
  const int at_once = 256 / c.head_dim;
  const int groups = (2 * c.n_kv_heads + at_once - 1) / at_once;
  int parts = (152 * 32 + ntok - 1) / ntok;  // as in qg_rope.cu: rows spread over warps for few tokens
  if (parts > groups) parts = groups;
  const int per_part = (groups + parts - 1) / parts;
  parts = (groups + per_part - 1) / per_part;
  const int64_t warps = (int64_t)ntok * parts;
  return launch_pdl(kv_read_kernel<TYPE, TO>, dim3((unsigned)((warps + RD_WARPS - 1) / RD_WARPS)),
                    dim3(RD_THREADS), 0, s, 0, LC_L1, c, seq, pos, ntok, seq ? 1 : ntok / c.n_seq,
                    static_cast<TO*>(k_out), static_cast<TO*>(v_out), err, parts, per_part);
}

}  // namespace

cudaError_t kv_read_launch(const qg_kvcache& c, const int32_t* seq, const int32_t* pos, int ntok,
                           int yt, void* k_out, void* v_out, int32_t* err, cudaStream_t s) {
  if (c.type == QG_F16)
    return yt == QG_F32 ? read_typed<QG_F16, float>(c, seq, pos, ntok, k_out, v_out, err, s)
                        : read_typed<QG_F16, __half>(c, seq, pos, ntok, k_out, v_out, err, s);
  return yt == QG_F32 ? read_typed<QG_Q8_0, float>(c, seq, pos, ntok, k_out, v_out, err, s)
                      : read_typed<QG_Q8_0, __half>(c, seq, pos, ntok, k_out, v_out, err, s);
}

}  // namespace qg
