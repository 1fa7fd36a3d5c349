// qg_route.cu -- routing to experts from logits (qmoe_route): a warp a token (qg_route.cuh).
#include <cuda_runtime.h>

#include <cmath>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_route.cuh"

namespace qg {

namespace {

constexpr int RO_WARPS = 4;
constexpr int RO_BLOCKS = 152 * 12;  // with more tokens than warps of these, each takes several in turn

// One lane's experts of a row.
template <int NE>
__device__ __forceinline__ void load_row(const float* row, int first, int mine, float (&v)[NE]) {
#pragma unroll
  for (int i = 0; i < NE; ++i) v[i] = i < mine ? row[first + i] : 0.f;
}

// NE: experts of a lane, at most; 0: all in 64 bits
template <int NE>
__global__ void __launch_bounds__(RO_WARPS * 32, NE <= 8 ? 8 : 1)
    route_kernel(const __grid_constant__ qg_route r, const float* logits, int64_t stride, const float* bias, int ntok, int E,
                 int topk, int32_t* ids, float* rw) {
  extern __shared__ double s_c[];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  double* const c = s_c + warp * E;
  const int64_t step = (int64_t)gridDim.x * RO_WARPS;
  int64_t tok = (int64_t)blockIdx.x * RO_WARPS + warp;
  if constexpr (NE == 0) {
    for (; tok < ntok; tok += step) route_exact(r, logits + tok * stride, bias, E, topk, c, ids + tok * topk, rw + tok * topk);
  } else {
    __shared__ RouteSlot slots[RO_WARPS][RO_SLOTS];
    const RouteDeal deal = route_deal(r, E);
    const int group = lane / deal.lanes, from = (lane & (deal.lanes - 1)) * deal.per;
    const int first = group * deal.size + from;
    const int mine = first < E ? max(0, min(deal.per, deal.size - from)) : 0;
    float b[NE], l[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i) b[i] = 0.f;
    if (bias) load_row(bias, first, mine, b);
    for (; tok < ntok; tok += step) {
      load_row(logits + tok * stride, first, mine, l);
      if (!route_fast(r, deal, l, b, bias, first, mine, topk, slots[warp], ids + tok * topk, rw + tok * topk))
        route_exact(r, logits + tok * stride, bias, E, topk, c, ids + tok * topk, rw + tok * topk);
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
  const int per = route_deal(r, E).per;
  const auto kern = per <= 1    ? route_kernel<1>
                    : per <= 2  ? route_kernel<2>
                    : per <= 4  ? route_kernel<4>
                    : per <= 8  ? route_kernel<8>
                    : per <= 16 ? route_kernel<16>
                    : per <= 32 ? route_kernel<32>
                                : route_kernel<0>;
  const int64_t blocks = ((int64_t)ntok + RO_WARPS - 1) / RO_WARPS;
  return launch_pdl(kern, dim3((unsigned)(blocks < RO_BLOCKS ? blocks : RO_BLOCKS)), dim3(RO_WARPS * 32),
                    (size_t)RO_WARPS * E * sizeof(double), s, 0, LC_L1, r, logits, stride, bias, ntok, E, topk, ids, rw);
}

}  // namespace qg
