// qg_embed.cu -- embedding lookup: rows of a matrix in the library's layout by token id, times a scale (qembed). A lane makes
// units of neighbouring elements that it stores in one access, 4 f32 or 8 f16. For Q8_0 and Q4_0 it reads the 8 or 16 stored
// bytes that hold them and takes every second one, as the halves of a group lie byte by byte; a weight, an integer times its
// f16 scale, is exact in f32, then multiplied by the call's scale and rounded.
//
// Bound by memory where there are many rows: 20,011 of 2,048 from Q8_0, 208 MB, to f32 32.0 us, 96% of the rate of a large copy; to f16 21.0, 88%.
// 4,095 rows, 42 MB that stay in L2: 8.6 us, issue slots 66% used (the floor of a copy is 6.3). One row: 1.5 us, the launch and
// two loads, the second at the first one's place.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_blocks.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {

namespace {

constexpr int EM_WARPS = 4;

__device__ __forceinline__ void store_unit(float* p, const float (&v)[4]) { *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]); }
__device__ __forceinline__ void store_unit(__half* p, const float (&v)[8]) { store8(p, v); }

// U: units of a lane, whose loads are in flight together. A warp makes 32 U units of a token's row.
template <int QT, class TO, int U>
__global__ void __launch_bounds__(EM_WARPS * 32)
    embed_kernel(const void* q, const uint16_t* scl, int rows, int k, const int32_t* ids, int64_t pieces, int per_tok, float scale, TO* y,
                 int64_t ys, int32_t* err) {
  constexpr int E = 16 / sizeof(TO);  // elements of a unit; twice as many bytes hold them
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t piece = (int64_t)blockIdx.x * EM_WARPS + (threadIdx.x >> 5);
  if (piece >= pieces) return;
  const int64_t tok = per_tok == 1 ? piece : piece / per_tok;
  const int part = (int)(piece - tok * per_tok), id = ids[tok];
  const bool bad = id < 0 || id >= rows;
  if (bad && err && part == 0 && lane == 0) atomicOr(err, QG_EMBED_BAD_ID);
  TO* const out = y + tok * ys;
  const int first = part * (32 * U) + lane, units = k / E;
  uint32_t b[U][E / 2];
  uint16_t d[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int i = first + 32 * j, e = E * i;  // its first element
#pragma unroll
    for (int x = 0; x < E / 2; ++x) b[j][x] = 0;
    d[j] = 0;
    if (bad || i >= units) continue;
    const size_t at = QT == QG_F16    ? ((size_t)id * k + e) * 2
                      : QT == QG_Q8_0 ? (size_t)id * k + (e & ~15) + 2 * (e & 7)
                                      : (size_t)id * (k / 2) + e / 32 * 16 + 2 * (e & 7);
    const uint8_t* const p = static_cast<const uint8_t*>(q) + at;
    if constexpr (E == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      b[j][0] = x.x; b[j][1] = x.y; b[j][2] = x.z; b[j][3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      b[j][0] = x.x; b[j][1] = x.y;
    }
    if constexpr (QT != QG_F16) d[j] = scl[(size_t)id * (k / 32) + e / 32];
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int i = first + 32 * j, e = E * i;
    if (i >= units) continue;
    float v[E];
    if constexpr (QT == QG_F16) {
#pragma unroll
      for (int x = 0; x < E / 2; ++x) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&b[j][x]));
        v[2 * x] = f.x * scale;
        v[2 * x + 1] = f.y * scale;
      }
    } else {
      const float f = h2f(d[j]);
      const int shift = (e & 8) + (QT == QG_Q8_0 ? 0 : (e & 16) / 4);  // the half of the group; of Q4_0 its low or high bits
#pragma unroll
      for (int x = 0; x < E; ++x) {
        const uint32_t u = b[j][x >> 1] >> (shift + 16 * (x & 1));
        const int n = QT == QG_Q8_0 ? (int)(int8_t)(u & 0xff) : (int)(u & 15) - 8;
        v[x] = bad ? 0.f : (float)n * f * scale;
      }
    }
    store_unit(out + e, v);
  }
}

template <int QT, class TO, int U>
cudaError_t embed_u(const EmbedArgs& a, cudaStream_t s) {
  const int64_t units = (int64_t)a.k * sizeof(TO) / 16;
  const int per_tok = (int)((units + 32 * U - 1) / (32 * U));
  const int64_t pieces = (int64_t)a.ntok * per_tok;
  return launch_pdl(embed_kernel<QT, TO, U>, dim3((unsigned)((pieces + EM_WARPS - 1) / EM_WARPS)), dim3(EM_WARPS * 32), 0, s, 0, LC_L1, a.q,
                    a.scl, a.rows, a.k, a.ids, pieces, per_tok, a.scale, static_cast<TO*>(a.y), a.ys, a.err);
}

template <int QT, class TO>
cudaError_t embed_go(const EmbedArgs& a, cudaStream_t s) {
  // one unit a lane where that makes no more warps than the machine holds at a time; else four (one row of 5,120: 1.5 us, with four 1.65;
  // 150 rows of 2,048 1.73 and 1.79; 1,000 4.5 and 3.1; 4,095 17.4 and 8.5, 9.8 where a lane's elements are 16 neighbours)
  return (int64_t)a.ntok * a.k * sizeof(TO) <= (int64_t)152 * 64 * 512 ? embed_u<QT, TO, 1>(a, s) : embed_u<QT, TO, 4>(a, s);
}

template <class TO>
cudaError_t embed_to(const EmbedArgs& a, cudaStream_t s) {
  return a.qt == QG_Q4_0 ? embed_go<QG_Q4_0, TO>(a, s) : a.qt == QG_Q8_0 ? embed_go<QG_Q8_0, TO>(a, s) : embed_go<QG_F16, TO>(a, s);
}

}  // namespace

cudaError_t embed_launch(const EmbedArgs& a, cudaStream_t s) {
  return a.yt == QG_F32 ? embed_to<float>(a, s) : embed_to<__half>(a, s);
}

}  // namespace qg
