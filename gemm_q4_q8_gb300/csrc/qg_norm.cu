// qg_norm.cu -- root-mean-square norm of rows with the residual's addition (qrms_norm), to f32, f16 or Q8_0 rows.
//
// s = x + add (rounded to x's type where that is f16: the sum that is stored is the one that is normed),
// y = s (w + w_add) / sqrt(mean s^2 + eps). A row stays in registers: its elements are read once, their squares summed in f32,
// and normed where they are. Rows of up to 1,024 elements are a warp's (or 8 or 16 lanes' of one), longer ones a block's.
//
// Squares that leave the range of f32 (elements beyond 10^18, or all below 10^-17 with an eps as small) are summed again in
// 64 bits: a row that needs it shows by its sum.
//
// Bound by memory: 8,191 rows of 5,120 f32 with the residual, to f16 and f32: 84.6 us, 587 MB, the rate of a large copy; without it 38.6 us,
// 252 MB, 96% of it. To Q8_0 by its instructions, 140 for eight elements of a lane: 20,011 rows of 2,048 f16 in 28.5 us, where the bytes
// take 18.5, with 28 warps an SM and two thirds of the issue slots used (read back in the rest of 48.7; groups of eight a thread: two
// 54.4, eight, whose registers halve the warps, 67.3). One row of 5,120: 2.5 us, the launch, two trips to memory and one barrier.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "qg_blocks.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {

namespace {

constexpr int NM_WARP_THREADS = 128;

template <class TI>
struct NormParams {
  const TI *x, *add;
  TI* sum;
  const float* w;
  void* y;
  uint16_t* scl;
  int64_t xs, as, ss, ys;
  float w_add, eps, inv_n;
  uint32_t heads, rows;
  int n;
};

template <class T>
__device__ __forceinline__ float round_to(float v);
template <>
__device__ __forceinline__ float round_to<float>(float v) { return v; }
template <>
__device__ __forceinline__ float round_to<__half>(float v) { return __half2float(__float2half_rn(v)); }
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }

// Sum over the group of a row: `lanes` lanes of a warp, or (BLOCK) all warps, in one order for everybody.
template <bool BLOCK, class A>
__device__ __forceinline__ A row_sum(A v, int lanes, A* part) {
  for (int off = BLOCK ? 16 : lanes >> 1; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if constexpr (BLOCK) {
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) v += part[i];
  }
  return v;
}

// YT: the type of y. ROWS: SINGLE, any rows, element by element; EIGHTS, in groups of eight elements, 16-byte aligned; FULL, and
// every thread of a block has U such groups.
enum { SINGLE, EIGHTS, FULL };
template <class TI, int YT, int ROWS, int U, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : NM_WARP_THREADS) norm_kernel(const __grid_constant__ NormParams<TI> p, int lanes) {
  constexpr bool VEC = ROWS != SINGLE;
  __shared__ float part[BLOCK ? 32 : 1];
  __shared__ double part64[BLOCK ? 32 : 1];
  pdl_trigger();
  pdl_wait();
  const int width = BLOCK ? blockDim.x : lanes;
  const int t = BLOCK ? threadIdx.x : threadIdx.x & (lanes - 1);
  const uint32_t row = BLOCK ? blockIdx.x : blockIdx.x * (NM_WARP_THREADS / lanes) + threadIdx.x / lanes;  // (below 2^31 + 32)
  const bool live = BLOCK || row < p.rows;
  const uint32_t of = !live ? 0 : p.heads == 1 ? row : row / p.heads;
  const int64_t tok = of, head = live ? row - of * p.heads : 0;
  const TI* const x = p.x + tok * p.xs + head * p.n;
  const TI* const add = p.add ? p.add + tok * p.as + head * p.n : nullptr;
  TI* const sum = p.sum ? p.sum + tok * p.ss + head * p.n : nullptr;
  // element e of the thread's group c; ok: is it one
  auto at = [&](int c, int e) { return VEC ? (c * width + t) * 8 + e : (c * 8 + e) * width + t; };
  auto ok = [&](int i) { return ROWS == FULL || (live && i < p.n); };

  float v[U][8];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    if constexpr (VEC) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = 0.f;
      if (ok(at(c, 0))) load8(x + at(c, 0), v[c]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = ok(at(c, e)) ? as_f32(x[at(c, e)]) : 0.f;
    }
  }
  if (add) {
#pragma unroll
    for (int c = 0; c < U; ++c) {
      float a[8];
      if constexpr (VEC) {
        if (!ok(at(c, 0))) continue;
        load8(add + at(c, 0), a);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = ok(at(c, e)) ? as_f32(add[at(c, e)]) : 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = round_to<TI>(v[c][e] + a[e]);
    }
  }
  if (sum) {
#pragma unroll
    for (int c = 0; c < U; ++c) {
      if constexpr (VEC) {
        if (ok(at(c, 0))) store8(sum + at(c, 0), v[c]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (ok(at(c, e))) put(sum + at(c, e), v[c][e]);
      }
    }
  }
  float2 sq = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < U; ++c)
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 x = make_float2(v[c][e], v[c][e + 1]);
      sq = fma2(x, x, sq);
    }
  const float ss = row_sum<BLOCK>(sq.x + sq.y, lanes, part);
  const float mean = fmaf(ss, p.inv_n, p.eps);
  float r = rsqrtf(mean);  // (off by 2 steps at most)
  const bool wide = live && !(ss <= 0x1p120f && mean >= 0x1p-100f);  // (NaN, too)
  if (__builtin_expect(BLOCK ? wide : __any_sync(0xffffffffu, wide), 0)) {
    double s = 0;
#pragma unroll
    for (int c = 0; c < U; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fma((double)v[c][e], (double)v[c][e], s);
    s = 1. / sqrt(row_sum<BLOCK>(s, lanes, part64) / p.n + (double)p.eps);
    // an element times s is at most sqrt n; s alone may leave the range of f32
    if (wide) {
#pragma unroll
      for (int c = 0; c < U; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = (float)(v[c][e] * s);
      r = 1.f;
    }
  }
  // group c's normed elements (VEC)
  auto normed = [&](int c, float (&y)[8]) {
    const int i = at(c, 0);
    float g[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (p.w && ok(i)) load8(p.w + i, g);
    if (p.w_add != 0.f)
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] += p.w_add;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float2 x = mul2(mul2(make_float2(v[c][e], v[c][e + 1]), make_float2(r, r)), make_float2(g[e], g[e + 1]));
      y[e] = x.x;
      y[e + 1] = x.y;
    }
  };
  if constexpr (YT == QG_Q8_0) {
    auto blocks = [&](auto tame) {  // the largest magnitude
      float most = 0.f;
#pragma unroll
      for (int c = 0; c < U; ++c) {
        const int i = at(c, 0);
        float y[8], top;
        uint32_t q[2];
        normed(c, y);
        const uint32_t bits = q8_block<0, decltype(tame)::value>(y, q, top);
        most = max_nan(most, top);
        // stored order: of each 16 bytes the two halves byte by byte, a half a lane
        const bool second = t & 1;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, second ? q[0] : q[1], 1);
        const uint32_t a = second ? got : q[0], b = second ? q[1] : got;
        if (ok(i)) {
          reinterpret_cast<uint2*>(static_cast<int8_t*>(p.y) + (int64_t)row * p.n)[i >> 3] =
              make_uint2(__byte_perm(a, b, 0x5140), __byte_perm(a, b, 0x7362));
          if ((t & 3) == 0) p.scl[(int64_t)row * (p.n >> 5) + (i >> 5)] = (uint16_t)bits;
        }
      }
      return most;
    };
    const float most = blocks(std::true_type());
    if (__builtin_expect(__any_sync(0xffffffffu, !(most <= Q8_TOP)), 0)) blocks(std::false_type());
    return;
  }
#pragma unroll
  for (int c = 0; c < U; ++c) {
    float y[8];
    if constexpr (VEC) {
      const int i = at(c, 0);
      normed(c, y);
      if (ok(i)) {
        if constexpr (YT == QG_F16) store8(static_cast<__half*>(p.y) + tok * p.ys + head * p.n + i, y);
        if constexpr (YT == QG_F32) store8(static_cast<float*>(p.y) + tok * p.ys + head * p.n + i, y);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = at(c, e);
        if (!ok(i)) continue;
        const float o = v[c][e] * r * ((p.w ? p.w[i] : 1.f) + p.w_add);
        if constexpr (YT == QG_F16) put(static_cast<__half*>(p.y) + tok * p.ys + head * p.n + i, o);
        if constexpr (YT == QG_F32) put(static_cast<float*>(p.y) + tok * p.ys + head * p.n + i, o);
      }
    }
  }
}

template <class TI, int YT, int ROWS, int U>
cudaError_t norm_u(const NormParams<TI>& p, cudaStream_t s) {
  const int eights = (p.n + 7) / 8, need = (eights + U - 1) / U;
  if (need <= 32) {
    int lanes = 4;
    while (lanes < need) lanes *= 2;
    const int per = NM_WARP_THREADS / lanes;
    return launch_pdl(norm_kernel<TI, YT, ROWS, U, false>, dim3((p.rows + per - 1) / per), dim3(NM_WARP_THREADS), 0, s, 0,
                      LC_L1, p, lanes);
  }
  // (without the tests 20,011 rows of 2,048 made Q8_0 and read back took 52.9 us instead of 54.0, one token of 5,120 2.5 instead of 2.7)
  const auto kern = ROWS == EIGHTS && p.n % (8 * 32 * U) == 0 ? norm_kernel<TI, YT, FULL, U, true> : norm_kernel<TI, YT, ROWS, U, true>;
  return launch_pdl(kern, dim3(p.rows), dim3((need + 31) / 32 * 32), 0, s, 0, LC_L1, p, 0);
}

// Groups of eight a thread. Few rows, 1,280 threads an SM at most: one, the shortest way through a row (5,120 f32 elements with add: 150
// rows 3.5 us, with two groups 3.8; 300: 3.8 and 4.5; 400, above the bound, 5.7 and 4.8). Many: as many as keep the loads of other rows
// in flight behind a row's sums, four, or two where add is read, too (8,191 rows, to f16: 38.5 us with four, 45.2 with two, 61.1
// with one; with add 88.3, 84.8 and 90.0); of rows of 64 elements or fewer two, as four leave lanes without any (240,000 rows of
// 64: 17.1 us, 21.1 with four; of 96: 28.0, 24.7). Rows read element by element: one (108.7 us for rows of 5,119 with add, 115 and
// 176).
template <class TI, int YT, int ROWS>
cudaError_t norm_rows(const NormParams<TI>& p, cudaStream_t s) {
  const int eights = (p.n + 7) / 8;
  if (eights <= 1024 && (ROWS == SINGLE || (int64_t)p.rows * eights <= 152 * 1280)) return norm_u<TI, YT, ROWS, 1>(p, s);
  if (eights <= 2048 && (ROWS == SINGLE || p.add || eights <= 8)) return norm_u<TI, YT, ROWS, 2>(p, s);
  return norm_u<TI, YT, ROWS, 4>(p, s);
}

template <class TI>
cudaError_t norm_typed(const NormArgs& a, cudaStream_t s) {
  NormParams<TI> p;
  p.x = static_cast<const TI*>(a.x);
  p.add = static_cast<const TI*>(a.add);
  p.sum = static_cast<TI*>(a.sum);
  p.w = a.w;
  p.y = a.y;
  p.scl = a.scl;
  p.xs = a.xs; p.as = a.as; p.ss = a.ss; p.ys = a.ys;
  p.w_add = a.w_add; p.eps = a.eps; p.inv_n = (float)(1. / a.n);
  p.heads = a.heads; p.n = a.n;
  p.rows = (uint32_t)a.ntok * a.heads;
  if (a.yt == QG_Q8_0) return norm_rows<TI, QG_Q8_0, EIGHTS>(p, s);
  if (a.vec) return a.yt == QG_F16 ? norm_rows<TI, QG_F16, EIGHTS>(p, s) : norm_rows<TI, QG_F32, EIGHTS>(p, s);
  return a.yt == QG_F16 ? norm_rows<TI, QG_F16, SINGLE>(p, s) : norm_rows<TI, QG_F32, SINGLE>(p, s);
}

}  // namespace

cudaError_t norm_launch(const NormArgs& a, cudaStream_t s) {
  return a.xt == QG_F32 ? norm_typed<float>(a, s) : norm_typed<__half>(a, s);
}

}  // namespace qg
