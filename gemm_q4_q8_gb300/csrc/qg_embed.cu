// qg_embed.cu -- embedding lookup: rows of a matrix in the library's layout by token id, times a scale (qembed). A thread
// makes eight neighbouring elements at a time. For Q8_0 and Q4_0 it reads the 16 stored bytes that hold them (its neighbours
// read the same ones) and takes every second byte, as the halves of a group lie byte by byte; a weight, an integer times its
// f16 scale, is exact in f32, then multiplied by the call's scale and rounded.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_blocks.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {

namespace {

constexpr int EM_THREADS = 128;

template <int QT, class TO>
__global__ void __launch_bounds__(EM_THREADS)
    embed_kernel(const void* q, const uint16_t* scl, int rows, int k, const int32_t* ids, float scale, TO* y, int64_t ys,
                 int32_t* err) {
  pdl_trigger();
  pdl_wait();
  const int tok = blockIdx.x, id = ids[tok];
  const bool bad = id < 0 || id >= rows;
  if (bad && err && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(err, QG_EMBED_BAD_ID);
  TO* const out = y + tok * ys;
  for (int i = blockIdx.y * EM_THREADS + threadIdx.x; i < k / 8; i += gridDim.y * EM_THREADS) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (!bad) {
      if constexpr (QT == QG_F16) {
        load8(static_cast<const __half*>(q) + (size_t)id * k + 8 * i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
      } else {
        // eighth i of the row: of Q8_0 half i % 2 of group i / 2; of Q4_0 half i % 2 of block i / 4, its low or high bits
        const uint4 b = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(q) +
                                                        (QT == QG_Q8_0 ? (size_t)id * k + 16 * (i / 2) : (size_t)id * (k / 2) + 16 * (i / 4)));
        const float d = h2f(scl[(size_t)id * (k / 32) + i / 4]);
        const uint32_t w[4] = {b.x, b.y, b.z, b.w};
        const int shift = 8 * (i & 1) + (QT == QG_Q8_0 ? 0 : 4 * ((i >> 1) & 1));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t u = w[e >> 1] >> (shift + 16 * (e & 1));
          const int n = QT == QG_Q8_0 ? (int)(int8_t)(u & 0xff) : (int)(u & 15) - 8;
          v[e] = (float)n * d * scale;
        }
      }
    }
    store8(out + 8 * i, v);
  }
}

template <int QT, class TO>
cudaError_t embed_go(const EmbedArgs& a, cudaStream_t s) {
  const int parts = (a.k / 8 + EM_THREADS - 1) / EM_THREADS;
  return launch_pdl(embed_kernel<QT, TO>, dim3((unsigned)a.ntok, (unsigned)parts), dim3(EM_THREADS), 0, s, 0, LC_L1, a.q, a.scl, a.rows, a.k,
                    a.ids, a.scale, static_cast<TO*>(a.y), a.ys, a.err);
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
