// qg_route.cu -- routing to experts from logits (qmoe_route): a warp a token (qg_route.cuh).
#include <cuda_runtime.h>

#include <cmath>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_route.cuh"

namespace qg {

namespace {

constexpr int RO_WARPS = 4;

__global__ void __launch_bounds__(RO_WARPS * 32)
    route_kernel(const __grid_constant__ qg_route r, const float* logits, int64_t stride, const float* bias, int ntok, int E,
                 int topk, int32_t* ids, float* rw) {
  extern __shared__ double s_c[];
  pdl_trigger();
  pdl_wait();
  const int64_t tok = (int64_t)blockIdx.x * RO_WARPS + (threadIdx.x >> 5);
  if (tok >= ntok) return;
  route_token(r, logits + tok * stride, bias, E, topk, s_c + (threadIdx.x >> 5) * E, ids + tok * topk, rw + tok * topk);
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
  return launch_pdl(route_kernel, dim3((unsigned)((ntok + (int64_t)RO_WARPS - 1) / RO_WARPS)), dim3(RO_WARPS * 32),
                    (size_t)RO_WARPS * E * sizeof(double), s, 0, LC_L1, r, logits, stride, bias, ntok, E, topk, ids, rw);
}

}  // namespace qg
