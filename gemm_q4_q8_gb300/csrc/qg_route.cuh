// qg_route.cuh -- a token's experts by a warp, from its logits: scores, bias, groups, top k, weights (qmoe_route, and
// qmoe_router_planned on the logits that it has made).
//
// p_e = softmax or sigmoid of the logits, c_e = p_e + bias_e (p_e without a bias); the order is that of c, in 64 bits, and
// without a bias that of the logits; lowest id on ties, NaN behind everything. With groups, a group's value is the sum of its
// one or two largest c.
//
// Nearly always f32 decides: with a bound on the error of every c at hand, two that lie further apart than their bounds are in
// the order that 64 bits find. So a token is routed in f32 (route_fast); where two of the k best and their next, or two groups at
// the border, are too near, these few are compared in 64 bits, and where more than 64 experts may be among the k best, a logit or a
// bias is NaN or +infinity, one of -infinity is chosen, or a weight is next to nothing, all of it is done again in 64 bits
// (route_exact).
//
// A bound is `off`, the largest that a p may be off by, and 2^-24 of c itself for the addition of the bias. So experts that are shut out by
// biases or logits far below the others' are off by much themselves and blur no others. (16,383 tokens of 256 experts in 8 groups, logits
// from memory, a bias of -1e9 on one of them: 19.3 us, 19.2 without it; with one bound for all c, from the largest bias, 931.)
//
// route_fast. The lanes of a warp are dealt to the groups, and a group's experts in runs to its lanes, in registers. The k-th
// largest of the lanes' maxima is a bound below which no expert can be among the k best; what is above it, a few more than
// k, goes to shared memory, one or two for each lane, which counts how many are ahead.
//
// The numbers of route_fast stay within f32's, or are -infinity where 64 bits have next to nothing or less than f32 holds: a group's
// worth is halved, as the sum of two c may leave it.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "qgemm.h"

namespace qg {

constexpr int RO_MAXE = 1024, RO_MAXK = 32, RO_MAXG = 32;
constexpr int RO_SLOTS = 64;  // experts that may be among the k best: two a lane
constexpr int RO_NONE = 1 << 20;  // a rank behind all

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
static __device__ __noinline__ void route_exact(const qg_route& r, const float* logits, const float* bias, int E, int topk, double* c,
                                            int32_t* ids, float* rw) {
  __syncwarp();  // (functions that are called: their lanes come together first)
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

// How the experts are dealt to the lanes: a group's to `lanes` of them (a power of two), `per` neighbours each.
struct RouteDeal {
  int lanes, per, size;
};
__host__ __device__ inline RouteDeal route_deal(const qg_route& r, int E) {
  RouteDeal d;
  const int groups = r.top_group < r.n_group ? r.n_group : 1;
  d.size = E / groups;
  d.lanes = 32;
  while (d.lanes * groups > 32) d.lanes /= 2;
  d.per = (d.size + d.lanes - 1) / d.lanes;
  return d;
}

// A lane's: `mine` experts from id `first`.
__device__ __forceinline__ void route_share(const RouteDeal& d, int E, int& first, int& mine) {
  const int lane = threadIdx.x & 31, from = (lane & (d.lanes - 1)) * d.per;
  first = lane / d.lanes * d.size + from;
  mine = first < E ? max(0, min(d.per, d.size - from)) : 0;
}

__device__ __forceinline__ float ro_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float ro_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Order of finite f32 as unsigned numbers above 0.
__device__ __forceinline__ uint32_t ro_key32(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float ro_warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// An expert that may be among the k best: its c in 32 or in 64 bits.
struct RouteSlot {
  union {
    float c;
    double exact;
  };
  int id;
};
// A number of a key.
__device__ __forceinline__ float ro_value(uint32_t key) { return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key); }

// exp(x - y), with what rounding the difference leaves (half a step of 32 to 64 is 2^-19).
__device__ __forceinline__ float ro_exp_diff(float x, float y) {
  const float d = x - y, v = d - x, left = (x - (d - v)) - (y + v), e = expf(d);
  return fmaf(e, left, e);
}

// Scores in 64 bits (softmax: over the sum), of finite logits.
static __device__ __noinline__ double ro_score(bool soft, float l, float top) {
  const double e = exp(soft ? (double)l - (double)top : -(double)l);
  return soft ? e : 1. / (1. + e);
}
static __device__ __noinline__ double ro_sum64(const float* row, int first, int mine, float top) {
  double all = 0.;
  for (int i = 0; i < mine; ++i) all += ro_score(true, row[first + i], top);
  __syncwarp();
  return ro_warp_sum(all);
}

// The experts of this lane: `mine` of them from id `first`, their logits l and biases b in registers (where there are fewer than NE:
// -infinity and 0; FULL: there are not), the logits of all at `row`. False: not decided.
template <int NE, bool FULL>
__device__ __forceinline__ bool route_fast(const qg_route& r, const RouteDeal& deal, const float (&l)[NE], const float (&b)[NE],
                                           const float* row, const float* bias, int first, int mine, int topk, RouteSlot* slots,
                                           int32_t* ids, float* rw) {
  __syncwarp();
  const int lane = threadIdx.x & 31;
  const bool grouped = r.top_group < r.n_group, soft = r.score == QG_SCORE_SOFTMAX;
  auto here = [&](int i) { return FULL || i < mine; };
  // the largest of the logits
  float most = -INFINITY;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    most = fmaxf(most, l[i]);
    odd |= here(i) && !(l[i] + b[i] < INFINITY);
  }
  if (__any_sync(0xffffffffu, odd)) return false;
  float top = 0.f, sum = 1.f;
  if (soft) {
    top = ro_value(__reduce_max_sync(0xffffffffu, ro_key32(most)));
    if (top == -INFINITY) return false;  // (all of them)
    if (bias || grouped || !r.renorm) {    // (else only ratios are wanted)
      float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NE; ++i) part[i & 3] += expf(l[i] - top);
      sum = ro_warp_sum((part[0] + part[1]) + (part[2] + part[3]));
    }
  }
  // c, and a bound on the errors of all p. Sigmoid: the exponent is off by |l| 2^-23.4 (its factor and product), ex2, sum and reciprocal
  // by less than 2^-21 together. Softmax: the exponent by |l - top| 2^-24 more, expf by 2^-22, and the sum by its additions, at most
  // 15 2^-24, the same 2^-22 and the exponents' mean error, below 7 2^-24 (an entropy). The bounds are twice that and more.
  float c[NE], off = 0.f;
  if (bias || grouped) {
    const float inv = ro_rcp(sum);
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const float x = soft ? l[i] - top : l[i];
      const float p = soft ? ro_ex2(x * 1.44269504f) * inv : ro_rcp(1.f + ro_ex2(x * -1.44269504f));
      off = fmaxf(off, p * fmaf(fabsf(x), 0x1p-21f, soft ? 0x1p-18f : 0x1p-20f));  // (0 times infinity, a NaN, is passed over)
      c[i] = here(i) ? p + b[i] : -INFINITY;
    }
    off = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(off))) + 0x1p-120f;  // (p below f32's normals are 0)
  }
  bool open = true;
  if (grouped) {
    // the group's two largest, by its lanes
    float v0 = -INFINITY, v1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      v1 = fmaxf(v1, fminf(v0, c[i]));
      v0 = fmaxf(v0, c[i]);
    }
    for (int x = deal.lanes >> 1; x >= 1; x >>= 1) {
      const float u0 = __shfl_xor_sync(0xffffffffu, v0, x), u1 = __shfl_xor_sync(0xffffffffu, v1, x);
      v1 = fmaxf(fminf(v0, u0), fmaxf(v1, u1));
      v0 = fmaxf(v0, u0);
    }
    // half the sum, and how far that may be off: two p, two additions and its own. (-infinity: not at all)
    const float v_last = r.group_top == 2 ? v1 : v0, worth = 0.5f * v0 + 0.5f * v_last, f32_least = -3.402823466e38f;
    const float err = fmaf(fabsf(fmaxf(v0, f32_least)), 0x1p-22f, fmaf(fabsf(fmaxf(v_last, f32_least)), 0x1p-22f, off));
    const float lo = worth - err, hi = worth + err;
    int ahead = 0;
#pragma unroll 4
    for (int h = 0; h < r.n_group; ++h) ahead += __shfl_sync(0xffffffffu, worth, h * deal.lanes) > worth;
    const bool there = lane < r.n_group * deal.lanes;
    open = ahead < r.top_group;
    // every group that stays surely above every other?
    const int n_in = __popc(__ballot_sync(0xffffffffu, there && open));
    const float last = ro_value(__reduce_min_sync(0xffffffffu, there && open ? ro_key32(lo) : 0xffffffffu));
    const uint32_t out = __reduce_max_sync(0xffffffffu, there && !open ? ro_key32(hi) : 0u);
    if (n_in > r.top_group * deal.lanes || !(last > ro_value(out))) {  // (groups equal at the border are all open)
      if (last == -INFINITY) return false;
      // Surely above the last one that stays and all others: stays. Surely below all that stay: does not. Those between in 64 bits, of
      // each the experts that may be its largest.
      const float edge = ro_value(__reduce_min_sync(0xffffffffu, there && open ? ro_key32(worth) : 0xffffffffu));
      const float next = ro_value(__reduce_max_sync(0xffffffffu, there && worth <= edge ? ro_key32(hi) : 0u));
      const bool above = there && lo > next, close = there && !above && hi >= last;
      const float from = fmaf(-0x1p-20f, fabsf(v_last), fmaf(-2.f, off, v_last));
      const double all = soft ? ro_sum64(row, first, mine, top) : 1.;
      double t0 = -INFINITY, t1 = -INFINITY;
      uint32_t todo = 0;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (close && here(i) && c[i] >= from) todo |= 1u << i;
      for (; todo; todo &= todo - 1) {
        const int e = first + __ffs(todo) - 1;
        const double v = ro_score(soft, row[e], top) / all + (bias ? (double)bias[e] : 0.);
        if (v > t0) {
          t1 = t0;
          t0 = v;
        } else if (v > t1) {
          t1 = v;
        }
      }
      __syncwarp();
      for (int x = deal.lanes >> 1; x >= 1; x >>= 1) {
        const double u0 = __shfl_xor_sync(0xffffffffu, t0, x), u1 = __shfl_xor_sync(0xffffffffu, t1, x);
        t1 = t0 > u0 ? (u0 > t1 ? u0 : t1) : (t0 > u1 ? t0 : u1);
        t0 = t0 > u0 ? t0 : u0;
      }
      const double exact = r.group_top == 2 ? t0 + t1 : t0;
      const uint32_t all_close = __ballot_sync(0xffffffffu, close);
      int left = r.top_group - __popc(__ballot_sync(0xffffffffu, above)) / deal.lanes;
      const int g = lane / deal.lanes;
      for (int h = 0; h < r.n_group; ++h) {
        const double its = __shfl_sync(0xffffffffu, exact, h * deal.lanes);
        if (all_close >> (h * deal.lanes) & 1) left -= its > exact || (its == exact && h < g);
      }
      open = above || (close && left > 0);
    }
  }
  if (!bias) {
    off = 0.f;
#pragma unroll
    for (int i = 0; i < NE; ++i) c[i] = l[i];
  } else {
    most = -INFINITY;
#pragma unroll
    for (int i = 0; i < NE; ++i) most = fmaxf(most, c[i]);
  }
  // the k-th largest of the lanes' maxima, less what it may be off and what one below it may be: off each, and 2^-24 of itself each, of
  // which that of the lower one follows the other's (less than 2^-20 of the k-th in all)
  const float rel = bias ? 0x1p-20f : 0.f;
  uint32_t key = open && most > -INFINITY ? ro_key32(most) : 0u, bound = 0;
  for (int n = 0; n < topk; ++n) {
    bound = __reduce_max_sync(0xffffffffu, key);
    if (key == bound) key = 0;  // (with every lane that has it: the bound is then lower than need be)
  }
  const float its = ro_value(bound);
  // (not below f32's least number: -infinity would let in experts that are not there)
  const float least = open ? (bound ? fmaxf(fmaf(-rel, fabsf(its), fmaf(-2.f, off, its)), -3.402823466e38f) : -3.402823466e38f) : INFINITY;
  uint32_t in = 0;
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (c[i] >= least) in |= 1u << i;
  int at = __popc(in);
  const int own = at;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, at, x);
    if (lane >= x) at += up;
  }
  const int n = __shfl_sync(0xffffffffu, at, 31);
  if (n > RO_SLOTS || n < topk) return false;  // (nothing is left unwritten)
  RouteSlot* to = slots + (at - own);
#pragma unroll
  for (int i = 0; i < NE; ++i)
    if (in >> i & 1) {
      to->c = c[i];
      to->id = first + i;
      ++to;
    }
  __syncwarp();
  // each lane's one or two: how many are ahead, and whether another is too near to tell
  int rank[2] = {RO_NONE, RO_NONE}, id[2] = {0, 0};
  bool near = false;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    if (j * 32 >= n) break;
    const bool one = j * 32 + lane < n;
    const float mine_c = one ? slots[j * 32 + lane].c : INFINITY;
    id[j] = one ? slots[j * 32 + lane].id : 0;
    const float reach = fmaf(rel, fabsf(mine_c), 2.f * off);
    int ahead = 0, close = 0;
#pragma unroll 4
    for (int m = 0; m < n; ++m) {
      const float d = slots[m].c - mine_c;
      ahead += d > 0.f;
      close += fabsf(d) <= reach;
    }
    if (one) rank[j] = ahead;
    near |= one && close > 1 && ahead < topk;
  }
  if (__any_sync(0xffffffffu, near)) {  // these few in 64 bits (without a bias: equal ones by their ids)
    const double all = soft && bias ? ro_sum64(row, first, mine, top) : 1.;
    double v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (rank[j] != RO_NONE) v[j] = bias ? ro_score(soft, row[id[j]], top) / all + (double)bias[id[j]] : (double)row[id[j]];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (rank[j] != RO_NONE) slots[j * 32 + lane].exact = v[j];
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (rank[j] != RO_NONE) {
        rank[j] = 0;
        for (int m = 0; m < n; ++m) rank[j] += slots[m].exact > v[j] || (slots[m].exact == v[j] && slots[m].id < id[j]);
      }
  }
  // (the weights' errors: expf 2^-22, the sums and the reciprocals below 2^-22 each; in the softmax's sum the differences' roundings
  // count by their terms)
  float w[2] = {0.f, 0.f}, all = 0.f;
  const float inv = soft ? ro_rcp(sum) : 1.f;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (rank[j] < topk) {
      const float x = row[id[j]];
      w[j] = soft ? ro_exp_diff(x, top) * inv : ro_rcp(1.f + expf(-x));
    }
  all = ro_warp_sum(w[0] + w[1]);
  const float by = r.renorm ? ro_rcp(all) : 1.f;
  // weights that f32 holds badly, or their reciprocal's
  const bool small = (rank[0] < topk && !(w[0] >= 0x1p-100f)) || (rank[1] < topk && !(w[1] >= 0x1p-100f));  // (NaN: of a difference)
  if (__any_sync(0xffffffffu, small)) return false;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (rank[j] < topk) {
      ids[rank[j]] = id[j];
      rw[rank[j]] = w[j] * by * r.scale;
    }
  __syncwarp();
  return true;
}

}  // namespace qg
