// qg_rope.cu -- rotary positions, alone (qrope) and fused with the write of the
// paged key/value cache (qkv_append).
//
// Both kernels have one shape: a warp owns a token and walks over rows (heads)
// of it. A row's D elements sit on D/8 neighbouring lanes, eight consecutive
// elements a lane, so a warp covers 256 / D heads at a time (D rounded up to a
// power of two). The angles depend on the token and the pair only, so a lane
// computes the sines and cosines of its eight elements once and keeps them over
// all heads.
//
// Angles: a pair's frequency is a 64-bit fixed-point fraction of a turn per
// position. Frequency times position modulo 2^64 is then the exact fraction of
// a turn (no large f32 angle, no f64), whose top 32 bits go to sincospif.
//
// Q8_0: the 32 elements of a block are on four lanes of the same quad of lanes,
// so the block's largest magnitude is two shuffles away.
//
// Bound by memory: 4 bytes read and 2 (f16) or 17/16 (Q8_0) written an element.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_kv.cuh"

namespace qg {

namespace {

constexpr int ROW_THREADS = 256;
constexpr int ROW_WARPS = ROW_THREADS / 32;

template <class T>
__device__ __forceinline__ float elem(const T* p);
template <>
__device__ __forceinline__ float elem<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float elem<__half>(const __half* p) { return __half2float(*p); }

// Eight consecutive elements, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __half* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// A lane's share of a token's rotation: y = x * c + partner * s, element by
// element, s carrying the sign. Elements past rot_dim get c = 1, s = 0.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ void make_turn(const qg_rope& plan, const uint64_t* steps, int pos, int d0,
                                          Turn& t) {
  const int h = plan.rot_dim >> 1;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = d0 + e;
    t.c[e] = 1.f;
    t.s[e] = 0.f;
    if (d < plan.rot_dim) {
      const bool second = plan.interleaved ? (e & 1) : d >= h;
      if (plan.interleaved && second) {  // the pair's angle is already there
        t.c[e] = t.c[e - 1];
        t.s[e] = -t.s[e - 1];
        continue;
      }
      const int pair = plan.interleaved ? d >> 1 : (second ? d - h : d);
      const uint64_t phase = steps[pair] * (uint64_t)(int64_t)pos;
      // the turn's fraction, signed, in half turns
      const float half_turns = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31
      float sn, cs;
      sincospif(half_turns, &sn, &cs);
      t.c[e] = cs * plan.mscale;
      t.s[e] = (second ? sn : -sn) * plan.mscale;
    }
  }
}

// The rotated values of a lane's eight elements; `row` points at the head.
// Every element of the head is read before the caller's __syncwarp, so y may
// overwrite x after it.
template <class T>
__device__ __forceinline__ void rotate8(const qg_rope& plan, const T* row, int d0, const Turn& t,
                                        float (&y)[8]) {
  float x[8];
  load8(row + d0, x);
  const int h = plan.rot_dim >> 1;
  if (d0 >= plan.rot_dim) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e];
    return;
  }
  float o[8];
  if (plan.interleaved) {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = x[e ^ 1];
  } else if ((h & 7) == 0) {
    load8(row + (d0 < h ? d0 + h : d0 - h), o);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      o[e] = d < plan.rot_dim ? elem(row + (d < h ? d + h : d - h)) : 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool in = d0 + e < plan.rot_dim;
    y[e] = in ? fmaf(x[e], t.c[e], o[e] * t.s[e]) : x[e];
  }
}

// Lanes of a row: D/8 rounded up to a power of two.
__host__ __device__ inline int row_lanes(int d) {
  int l = 1;
  while (l * 8 < d) l *= 2;
  return l;
}

struct RowSplit {
  int parts;      // warps of a token
  int per_part;   // row groups (of 32 / row_lanes rows) of each
};
// A token's rows are spread over several warps while there are fewer tokens
// than warps that fill the machine (152 SMs x 32 warps).
RowSplit split_rows(int ntok, int rows, int rows_at_once) {
  const int groups = (rows + rows_at_once - 1) / rows_at_once;
  int parts = (152 * 32 + ntok - 1) / ntok;
  if (parts > groups) parts = groups;
  if (parts < 1) parts = 1;
  RowSplit s;
  s.per_part = (groups + parts - 1) / parts;
  s.parts = (groups + s.per_part - 1) / s.per_part;
  return s;
}

// ------------------------------------------------------------------- qrope
template <class TI, class TO>
__global__ void __launch_bounds__(ROW_THREADS) rope_kernel(
    const __grid_constant__ qg_rope plan, const TI* x, int64_t xs, const int32_t* pos, int ntok,
    int n_heads, int d, TO* y, int64_t ys, int parts, int per_part) {
  __shared__ uint64_t steps[QG_ROPE_MAX_DIM / 2];
  pdl_trigger();
  if (threadIdx.x < plan.rot_dim / 2) steps[threadIdx.x] = plan.step[threadIdx.x];
  __syncthreads();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  const int64_t tok = w / parts;
  if (tok >= ntok) return;
  const int part = (int)(w - tok * parts);
  const int lanes = row_lanes(d), at_once = 32 / lanes;
  const int d0 = (lane & (lanes - 1)) * 8;
  const bool on = d0 < d;
  Turn t;
  make_turn(plan, steps, pos[tok], d0, t);
  const int r0 = part * per_part * at_once + lane / lanes;
  for (int i = 0; i < per_part; ++i) {
    const int r = r0 + i * at_once;
    const bool live = on && r < n_heads;
    float v[8];
    if (live) rotate8(plan, x + tok * xs + (int64_t)r * d, d0, t, v);
    __syncwarp();
    if (live) store8(y + tok * ys + (int64_t)r * d + d0, v);
  }
}

// -------------------------------------------------------------- qkv_append
template <class T>
struct AppendParams {
  qg_kvcache c;
  const T *q, *k, *v;
  int64_t qs, ks, vs;
  int n_q;
  __half* q_out;
  const int32_t *seq, *pos;
  int ntok, per_seq;  // per_seq: tokens of a sequence when seq is NULL
  int32_t* err;
  int parts, per_part;
  int rotate;
};

// Eight elements of a row into the record of (token slot, head).
template <int TYPE>
__device__ __forceinline__ void put8(uint8_t* half, int d0, int d, int i, float (&y)[8], bool live) {
  if constexpr (TYPE == QG_F16) {
    if (live)
      store8(reinterpret_cast<__half*>(half) + (d0 >> 5) * (KV_GROUP * 32) + i * 32 + (d0 & 31), y);
  } else {
    // largest magnitude of the block; a NaN or an infinity makes it infinite
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float a = fabsf(y[e]);
      top = fmaxf(top, a <= 3.402823466e38f ? a : __int_as_float(0x7f800000));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const bool bad = top > 3.402823466e38f;
    // rounded up, so that no quant of the block passes 127
    uint16_t bits = __half_as_ushort(__float2half_ru(__fdiv_rn(top, 127.f)));
    if (bits > 0x7BFF) bits = 0x7BFF;
    if (bad) bits = 0x7FFF;
    const float ds = __half2float(__ushort_as_half(bits));
    uint32_t w[2] = {0x80808080u, 0x80808080u};
    if (!bad && bits != 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float r = fminf(fmaxf(rintf(__fdiv_rn(y[e], ds)), -127.f), 127.f);
        const uint32_t b = (uint32_t)((int)r + 128);
        w[e >> 2] = (w[e >> 2] & ~(0xffu << (8 * (e & 3)))) | (b << (8 * (e & 3)));
      }
    }
    if (live) {
      const int blk = d0 >> 5;
      *reinterpret_cast<uint2*>(half + blk * (KV_GROUP * 32) + i * 32 + (d0 & 31)) = make_uint2(w[0], w[1]);
      if ((d0 & 31) == 0)
        reinterpret_cast<uint16_t*>(half + KV_GROUP * d)[blk * KV_GROUP + kv_scale_place(i)] = bits;
    }
  }
}

template <class T, int TYPE>
__global__ void __launch_bounds__(ROW_THREADS)
    append_kernel(const __grid_constant__ qg_rope plan, const __grid_constant__ AppendParams<T> a) {
  __shared__ uint64_t steps[QG_ROPE_MAX_DIM / 2];
  pdl_trigger();
  if (threadIdx.x < plan.rot_dim / 2) steps[threadIdx.x] = plan.step[threadIdx.x];
  __syncthreads();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * ROW_WARPS + (threadIdx.x >> 5);
  const int64_t tok = w / a.parts;
  if (tok >= a.ntok) return;
  const int part = (int)(w - tok * a.parts);
  const int d = a.c.head_dim;
  const int lanes = d >> 3, at_once = 32 / lanes;
  const int d0 = (lane & (lanes - 1)) * 8;
  const int pos = a.pos[tok];
  Turn t;
  if (a.rotate) make_turn(plan, steps, pos, d0, t);

  // the token's place in the cache (NULL: nowhere)
  uint8_t* place = nullptr;
  const int groups = a.c.page_size / KV_GROUP, rec = kv_record_bytes(TYPE, d);
  if (pos >= 0) {
    int bits = 0;
    const int seq = a.seq ? a.seq[tok] : (int)(tok / a.per_seq);
    const int page = kv_page_of(a.c, seq, pos, &bits);
    const int slot = pos & (a.c.page_size - 1);
    if (page >= 0)
      place = static_cast<uint8_t*>(a.c.pool) +
              ((size_t)page * a.c.n_kv_heads * groups + slot / KV_GROUP) * rec;
    else if (part == 0 && lane == 0 && a.err)
      atomicOr(a.err, bits);
  }
  const int in_group = pos & (KV_GROUP - 1);
  const int kv = a.c.n_kv_heads, rows = a.n_q + 2 * kv;
  const int r0 = part * a.per_part * at_once + lane / lanes;
  for (int i = 0; i < a.per_part; ++i) {
    const int r = r0 + i * at_once;
    if (r - lane / lanes >= rows) break;  // the whole warp is past the end
    const bool in = r < rows;
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const bool is_q = r < a.n_q, is_k = !is_q && r < a.n_q + kv;
    const int head = is_q ? r : is_k ? r - a.n_q : r - a.n_q - kv;
    if (in) {
      const T* row = is_q ? a.q + tok * a.qs : is_k ? a.k + tok * a.ks : a.v + tok * a.vs;
      row += (int64_t)head * d;
      if (a.rotate && (is_q || is_k))
        rotate8(plan, row, d0, t, y);
      else
        load8(row + d0, y);
    }
    if (in && is_q) store8(a.q_out + (tok * a.n_q + head) * (int64_t)d + d0, y);
    uint8_t* half = place + (size_t)head * groups * rec + (is_k ? 0 : kv_half_bytes(TYPE, d));
    put8<TYPE>(half, d0, d, in_group, y, in && !is_q && place != nullptr);
  }
}

template <class T, int TYPE>
cudaError_t append_typed(const KvAppendArgs& a, cudaStream_t s) {
  AppendParams<T> p;
  p.c = a.c;
  p.q = static_cast<const T*>(a.q);
  p.k = static_cast<const T*>(a.k);
  p.v = static_cast<const T*>(a.v);
  p.qs = a.qs; p.ks = a.ks; p.vs = a.vs;
  p.n_q = a.n_q;
  p.q_out = reinterpret_cast<__half*>(a.q_out);
  p.seq = a.seq; p.pos = a.pos;
  p.ntok = a.ntok;
  p.per_seq = a.seq ? 1 : a.ntok / a.c.n_seq;
  p.err = a.err;
  p.rotate = a.rope != nullptr;
  const RowSplit sp = split_rows(a.ntok, a.n_q + 2 * a.c.n_kv_heads, 256 / a.c.head_dim);
  p.parts = sp.parts;
  p.per_part = sp.per_part;
  qg_rope plan{};
  if (a.rope) plan = *a.rope;
  const int64_t warps = (int64_t)a.ntok * sp.parts;
  return launch_pdl(append_kernel<T, TYPE>, dim3((unsigned)((warps + ROW_WARPS - 1) / ROW_WARPS)),
                    dim3(ROW_THREADS), 0, s, 0, LC_L1, plan, p);
}

template <class TI, class TO>
cudaError_t rope_typed(const qg_rope& plan, const void* x, int64_t xs, const int32_t* pos, int ntok,
                       int n_heads, int d, void* y, int64_t ys, cudaStream_t s) {
  const RowSplit sp = split_rows(ntok, n_heads, 32 / row_lanes(d));
  const int64_t warps = (int64_t)ntok * sp.parts;
  return launch_pdl(rope_kernel<TI, TO>, dim3((unsigned)((warps + ROW_WARPS - 1) / ROW_WARPS)),
                    dim3(ROW_THREADS), 0, s, 0, LC_L1, plan, static_cast<const TI*>(x), xs, pos, ntok,
                    n_heads, d, static_cast<TO*>(y), ys, sp.parts, sp.per_part);
}

}  // namespace

cudaError_t rope_launch(const qg_rope& plan, int xt, const void* x, int64_t xs, const int32_t* pos,
                        int ntok, int n_heads, int head_dim, int yt, void* y, int64_t ys,
                        cudaStream_t s) {
  if (xt == QG_F32)
    return yt == QG_F32 ? rope_typed<float, float>(plan, x, xs, pos, ntok, n_heads, head_dim, y, ys, s)
                        : rope_typed<float, __half>(plan, x, xs, pos, ntok, n_heads, head_dim, y, ys, s);
  return yt == QG_F32 ? rope_typed<__half, float>(plan, x, xs, pos, ntok, n_heads, head_dim, y, ys, s)
                      : rope_typed<__half, __half>(plan, x, xs, pos, ntok, n_heads, head_dim, y, ys, s);
}

cudaError_t kv_append_launch(const KvAppendArgs& a, cudaStream_t s) {
  if (a.xt == QG_F32)
    return a.c.type == QG_F16 ? append_typed<float, QG_F16>(a, s) : append_typed<float, QG_Q8_0>(a, s);
  return a.c.type == QG_F16 ? append_typed<__half, QG_F16>(a, s) : append_typed<__half, QG_Q8_0>(a, s);
}

}  // namespace qg
