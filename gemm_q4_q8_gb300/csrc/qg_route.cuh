// qg_route.cuh -- a token's experts by a warp, from its logits: scores, bias, groups, top k, weights (qmoe_route, and
// qmoe_router_planned on the logits that it has made).
//
// p_e = softmax or sigmoid of the logits, c_e = p_e + bias_e (p_e without a bias); the order is that of c, in 64 bits, and
// without a bias that of the logits; lowest id on ties, NaN behind everything. With groups, a group's value is the sum of its
// one or two largest c.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "qgemm.h"

namespace qg {

constexpr int RO_MAXE = 1024, RO_MAXK = 32, RO_MAXG = 32;

// A key whose order is that of the numbers, +0 and -0 alike; 1: NaN; 0: nothing there.
__device__ __forceinline__ uint64_t ro_key(double v) {
  if (v != v) return 1;
  const uint64_t b = (uint64_t)__double_as_longlong(v == 0. ? 0. : v);
  return b >> 63 ? ~b : b | (1ull << 63);
}
// The largest key of a warp and the lowest index that has it.
__device__ __forceinline__ void ro_best(uint64_t& key, int& idx) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
  const uint64_t best = (uint64_t)hi << 32 | lo;
  idx = __reduce_min_sync(0xffffffffu, key == best ? idx : 0x7fffffff);
  key = best;
}
__device__ __forceinline__ double ro_warp_sum(double v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// By a whole warp. c: shared, a double for each expert; done with when the call returns.
__device__ __forceinline__ void route_token(const qg_route& r, const float* logits, const float* bias, int E, int topk, double* c,
                                            int32_t* ids, float* rw) {
  const int lane = threadIdx.x & 31;
  // softmax: the largest logit and the sum, NaN left out
  double top = -INFINITY, sum = 1.;
  if (r.score == QG_SCORE_SOFTMAX) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, logits[e]);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    top = m;
    sum = 0.;
  }
  auto score = [&](float l) {  // over the sum
    if (r.score == QG_SCORE_SIGMOID) return 1. / (1. + exp(-(double)l));
    return l == top ? 1. : exp((double)l - top);  // (infinite ones are alike)
  };
  if (r.score == QG_SCORE_SOFTMAX) {
    for (int e = lane; e < E; e += 32)
      if (logits[e] == logits[e]) sum += score(logits[e]);
    sum = ro_warp_sum(sum);
  }
  for (int e = lane; e < E; e += 32) c[e] = score(logits[e]) / sum + (bias ? (double)bias[e] : 0.);
  __syncwarp();
  uint32_t open = 0xffffffffu;  // groups
  const int size = E / r.n_group;
  if (r.top_group < r.n_group) {
    uint64_t key = 0;
    if (lane < r.n_group) {
      uint64_t k0 = 0, k1 = 0;
      double v0 = 0., v1 = 0.;
      for (int e = lane * size; e < (lane + 1) * size; ++e) {
        const double v = c[e];
        const uint64_t k = ro_key(v);
        if (k > k0) {
          k1 = k0; v1 = v0;
          k0 = k; v0 = v;
        } else if (k > k1) {
          k1 = k; v1 = v;
        }
      }
      key = ro_key(r.group_top == 2 ? v0 + v1 : v0);
    }
    open = 0;
    for (int i = 0; i < r.top_group; ++i) {
      uint64_t k = key;
      int g = lane;
      ro_best(k, g);
      open |= 1u << g;
      if (lane == g) key = 0;
    }
  }
  // each lane's best expert still there; the ones taken are marked
  uint32_t taken = 0;  // lane's experts, lane + 32 i
  int mine = -1;       // the lane's choice of the token
  for (int n = 0; n < topk; ++n) {
    uint64_t best = 0;
    int at = 0x7fffffff;
    for (int e = lane, i = 0; e < E; e += 32, ++i) {
      if ((taken >> i & 1) || !(open >> (r.n_group > 1 ? e / size : 0) & 1)) continue;
      const uint64_t k = ro_key(bias ? c[e] : (double)logits[e]);
      if (k > best) {
        best = k;
        at = e;
      }
    }
    ro_best(best, at);
    if ((at & 31) == lane) taken |= 1u << (at >> 5);
    if (n == lane) mine = at;
  }
  // weights, without the bias
  double w = 0.;
  if (mine >= 0) w = score(logits[mine]) / sum;
  if (r.renorm) {
    double all = 0.;
    for (int n = 0; n < topk; ++n) all += __shfl_sync(0xffffffffu, w, n);
    w = all == 0. ? 0. : w / all;
  }
  if (lane < topk) {
    ids[lane] = mine;
    rw[lane] = (float)(w * (double)r.scale);
  }
  __syncwarp();
}

}  // namespace qg
