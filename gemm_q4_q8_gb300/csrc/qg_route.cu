// qg_route.cu -- routing to experts from logits (qmoe_route): a warp a token (qg_route.cuh).
//
// Bound by instructions: 808 a token of 256 experts in 8 groups, 70% of the issue slots used: 16,383 tokens in 18.0 us, where
// their 18 MB would take 2.6 (18.4 with one expert shut out by -1e9, or by -infinity). Without bias and groups 11.1 us, 512 experts
// 31.5, 1,000 tokens 6.5; all of them in 64 bits, as a bias of NaN has it, 581. Eight or sixteen lanes a token instead of a
// warp: 22.6 and 25.2 us, as the k best one after the other then are a chain for few tokens at a time; the next token's logits
// loaded ahead: no gain.
#include <cuda_runtime.h>

#include <cmath>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_route.cuh"

namespace qg {

namespace {

constexpr int RO_WARPS = 4;
// Blocks of an SM (up to 8 experts a lane), which leave a thread 80 registers, and so many in all: with more tokens than warps, each
// takes several in turn. 16,383 tokens of 256 experts: 18.0 us; 19.5 with 8 blocks of 64 registers (which spill), 18.5 with twice as many in
// all.
constexpr int RO_PER_SM = 6, RO_BLOCKS = 152 * RO_PER_SM;

// NE: experts of a lane, at most; 0: all in 64 bits. WIDE: every lane has NE, and their logits are aligned to 16 bytes.
template <int NE, bool WIDE>
__global__ void __launch_bounds__(RO_WARPS * 32, NE <= 8 ? RO_PER_SM : 1)
    route_kernel(const __grid_constant__ qg_route r, const float* logits, int64_t stride, const float* bias, int ntok, int E,
                 int topk, int32_t* ids, float* rw) {
  extern __shared__ double s_c[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  double* const c = s_c + warp * E;
  const int64_t step = (int64_t)gridDim.x * RO_WARPS;
  int64_t tok = (int64_t)blockIdx.x * RO_WARPS + warp;
  if constexpr (NE == 0) {
    for (; tok < ntok; tok += step) route_exact(r, logits + tok * stride, bias, E, topk, c, ids + tok * topk, rw + tok * topk);
  } else {
    __shared__ RouteSlot slots[RO_WARPS][RO_SLOTS];
    const RouteDeal deal = route_deal(r, E);
    int first, mine;
    route_share(deal, E, first, mine);
    float b[NE], l[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) b[i] = bias && (WIDE || i < mine) ? bias[first + i] : 0.f;
    for (; tok < ntok; tok += step) {
      const float* const row = logits + tok * stride;
      if constexpr (WIDE) {
#pragma unroll
        for (int i = 0; i < NE; i += 4) {
          const float4 x = *reinterpret_cast<const float4*>(row + first + i);
          l[i] = x.x; l[i + 1] = x.y; l[i + 2] = x.z; l[i + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) l[i] = i < mine ? row[first + i] : -INFINITY;
      }
      if (!route_fast<NE, WIDE>(r, deal, l, b, row, bias, first, mine, topk, slots[warp], ids + tok * topk, rw + tok * topk))
        route_exact(r, row, bias, E, topk, c, ids + tok * topk, rw + tok * topk);
      __syncwarp();  // the slots have been read
    }
  }
}

}  // namespace

bool route_plan_ok(const qg_route& r) {
  return (r.score == QG_SCORE_SOFTMAX || r.score == QG_SCORE_SIGMOID) && r.n_group >= 1 && r.n_group <= RO_MAXG && r.top_group >= 1 &&
         r.top_group <= r.n_group && (r.group_top == 1 || r.group_top == 2) && std::isfinite(r.scale);
}
bool route_shape_ok(const qg_route& r, int E, int topk) {
  if (E < 1 || E > RO_MAXE || topk < 1 || topk > RO_MAXK || E % r.n_group) return false;
  const int size = E / r.n_group;
  return topk <= r.top_group * size && (r.top_group == r.n_group || r.group_top <= size);
}

cudaError_t route_launch(const qg_route& r, const float* logits, int64_t stride, const float* bias, int ntok, int E, int topk,
                         int32_t* ids, float* rw, cudaStream_t s) {
  const RouteDeal deal = route_deal(r, E);
  const int per = deal.per;
  // (16,383 tokens of 256 experts 17.9 us, 19.1 without; 128 15.5 and 16.0; 512 33.6 and 35.7; 1,024 64.6 and 90.6)
  const bool wide = E == 32 * per && per % 4 == 0 && (reinterpret_cast<uintptr_t>(logits) & 15) == 0 && (ntok == 1 || stride % 4 == 0);
  const auto kern = wide && per == 4    ? route_kernel<4, true>
                    : wide && per == 8  ? route_kernel<8, true>
                    : wide && per == 16 ? route_kernel<16, true>
                    : wide && per == 32 ? route_kernel<32, true>
                    : per <= 1          ? route_kernel<1, false>
                    : per <= 2          ? route_kernel<2, false>
                    : per <= 4          ? route_kernel<4, false>
                    : per <= 8          ? route_kernel<8, false>
                    : per <= 16         ? route_kernel<16, false>
                    : per <= 32         ? route_kernel<32, false>
                                        : route_kernel<0, false>;
  const int64_t blocks = ((int64_t)ntok + RO_WARPS - 1) / RO_WARPS;
  return launch_pdl(kern, dim3((unsigned)(blocks < RO_BLOCKS ? blocks : RO_BLOCKS)), dim3(RO_WARPS * 32),
                    (size_t)RO_WARPS * E * sizeof(double), s, 0, LC_L1, r, logits, stride, bias, ntok, E, topk, ids, rw);
}

}  // namespace qg
