// qg_attn.cu -- attention of new tokens over the paged key/value cache
// (qattn_paged): one CTA for a (sequence, column, head), its warps striding over
// the tokens with a running maximum and sum, joined through shared memory.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_kv.cuh"

namespace qg {

namespace {

constexpr int AT_WARPS = 8;

template <int TYPE>
__device__ __forceinline__ float kv_elem(const uint8_t* half, int d, int blk, int i, int lane) {
  const int at = blk * (KV_GROUP * 32) + i * 32 + lane;
  if constexpr (TYPE == QG_F16) {
    return __half2float(reinterpret_cast<const __half*>(half)[at]);
  } else {
    return ((float)half[at] - 128.f) *
           h2f(reinterpret_cast<const uint16_t*>(half + KV_GROUP * d)[blk * KV_GROUP + kv_scale_place(i)]);
  }
}

template <int TYPE, int D>
__global__ void __launch_bounds__(AT_WARPS * 32) attn_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int NB = D / 32;
  __shared__ float s_m[AT_WARPS], s_l[AT_WARPS], s_o[AT_WARPS][D];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x, col = blockIdx.y, seq = blockIdx.z;
  const int kv = a.c.n_kv_heads, head = h / (a.n_heads / kv);
  const int groups = a.c.page_size / KV_GROUP, rec = kv_record_bytes(TYPE, D);
  const int64_t len = a.lens[seq], cap = (int64_t)a.c.max_pages * a.c.page_size;
  if ((len < 0 || len > cap) && a.err && threadIdx.x == 0) atomicOr(a.err, QG_KV_BAD_POS);
  const int64_t p = (len < 0 ? 0 : len) - a.ncols + col;
  const int64_t lo = a.window > 0 && p - a.window + 1 > 0 ? p - a.window + 1 : 0;
  const int64_t hi = p + 1 < cap ? p + 1 : cap;
  const size_t row = (((size_t)seq * a.ncols + col) * a.n_heads + h) * D;
  float q[NB], o[NB], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    q[b] = h2f(a.q[row + b * 32 + lane]) * a.scale;
    o[b] = 0.f;
  }
  for (int64_t j = lo + warp; j < hi; j += AT_WARPS) {
    int bits = 0;
    const int page = kv_page_of(a.c, seq, (int)j, &bits);
    if (page < 0) {
      if (a.err && lane == 0) atomicOr(a.err, bits);
      continue;
    }
    const int slot = (int)j & (a.c.page_size - 1), i = slot & (KV_GROUP - 1);
    const uint8_t* r = static_cast<const uint8_t*>(a.c.pool) +
                       (((size_t)page * kv + head) * groups + slot / KV_GROUP) * rec;
    float s = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) s += q[b] * kv_elem<TYPE>(r, D, b, i, lane);
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float m2 = fmaxf(m, s);
    const float base = m2 == -INFINITY ? 0.f : m2;
    const float f = expf(m - base), w = expf(s - base);
    l = l * f + w;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      o[b] = o[b] * f + w * kv_elem<TYPE>(r + kv_half_bytes(TYPE, D), D, b, i, lane);
    m = m2;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) s_o[warp][b * 32 + lane] = o[b];
  __syncthreads();
  float top = -INFINITY;
  for (int w = 0; w < AT_WARPS; ++w) top = fmaxf(top, s_m[w]);
  if (top == -INFINITY) top = 0.f;
  float total = 0.f;
  for (int w = 0; w < AT_WARPS; ++w) total += s_l[w] * expf(s_m[w] - top);
  for (int e = threadIdx.x; e < D; e += AT_WARPS * 32) {
    float y = 0.f;
    for (int w = 0; w < AT_WARPS; ++w) y += s_o[w][e] * expf(s_m[w] - top);
    y = total == 0.f ? 0.f : y / total;
    a.y[row + e] = __half_as_ushort(__float2half_rn(y));
  }
}

template <int TYPE, int D>
cudaError_t attn_typed(const AttnArgs& a, cudaStream_t s) {
  return launch_pdl(attn_kernel<TYPE, D>, dim3(a.n_heads, a.ncols, a.c.n_seq), dim3(AT_WARPS * 32), 0, s, 0,
                    LC_L1, a);
}

}  // namespace

bool attn_shape_ok(int n_seq, int n_heads, int n_kv_heads, int head_dim, int ncols) {
  return n_seq >= 1 && n_seq <= QG_KV_MAX_SEQ && n_kv_heads >= 1 && n_kv_heads <= 256 && n_heads >= n_kv_heads &&
         n_heads % n_kv_heads == 0 && n_heads / n_kv_heads <= QG_ATTN_MAX_GROUP &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && ncols >= 1 && ncols <= QG_ATTN_MAX_COLS;
}

size_t attn_ws_bytes(int, int, int, int, int) { return 16; }

cudaError_t attn_launch(const AttnArgs& a, cudaStream_t s) {
  if (a.c.type == QG_F16) {
    if (a.c.head_dim == 64) return attn_typed<QG_F16, 64>(a, s);
    if (a.c.head_dim == 128) return attn_typed<QG_F16, 128>(a, s);
    return attn_typed<QG_F16, 256>(a, s);
  }
  if (a.c.head_dim == 64) return attn_typed<QG_Q8_0, 64>(a, s);
  if (a.c.head_dim == 128) return attn_typed<QG_Q8_0, 128>(a, s);
  return attn_typed<QG_Q8_0, 256>(a, s);
}

}  // namespace qg
