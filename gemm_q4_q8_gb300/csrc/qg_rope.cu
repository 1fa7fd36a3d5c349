// qg_rope.cu -- rotary positions, alone (qrope) and fused with the write of the
// paged key/value cache (qkv_append).
//
// Both kernels have one shape. A block of four warps takes 4 / P tokens, P warps
// each (and P x gridDim.y in all, so that few tokens still fill the machine). Its
// threads first compute the tokens' sines and cosines, one pair each, into shared
// memory; then each warp walks over rows (heads) of its token. A row's D elements
// sit on D/8 neighbouring lanes, eight consecutive elements a lane, so a warp
// covers 256 / D heads at a time (D rounded up to a power of two); a lane keeps
// the sines and cosines of its eight elements over all rows.
//
// Angles: a pair's frequency is a 64-bit fixed-point fraction of a turn per
// position. Frequency times position modulo 2^64 is then the fraction of a turn
// without rounding (no large f32 angle, no f64 here), whose top 32 bits go to
// sincospif.
//
// Q8_0: the 32 elements of a block are on four neighbouring lanes, so the
// block's largest magnitude is two shuffles away.
//
// Bound by memory: 4 bytes read and 2 (f16) or 17/16 (Q8_0) written an element.
// qrope, 8,191 tokens of 40 heads of 128, f32 to f16: 40.1 us, 6.3 TB/s. qkv_append,
// 16,382 tokens of 40 + 8 + 8 heads into Q8_0 blocks: 112 us, 5.7 TB/s, waiting for
// rows (46% of the issue slots used, 36 warps an SM).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_kv.cuh"

namespace qg {

namespace {

constexpr int ROW_THREADS = 128;
constexpr int ROW_WARPS = ROW_THREADS / 32;
// Blocks that share an SM: the rows' loads hide behind other warps (48 of them), not behind more rows a lane; 8,191 x 40
// x 128 from f32 to f16 took 40.1 us so, 42.5 with two rows and 46.6 with four rows a lane in flight. Blocks of eight warps:
// 40.8, and 145 us instead of 142 for a prompt of 16,382 tokens appended and read back.
constexpr int ROW_BLOCKS = 12;
// qkv_append's rows need more registers: that prompt takes 137 us with 10 blocks (which spill), 135 with 9, 138 with 8. The
// next key or value row in flight as well is no gain (142 with 9, 141 with 8), nor are prefetches into L2 (149).
constexpr int APPEND_BLOCKS = 9;

// How the eight elements of a lane meet their partners.
enum Layout {
  PLAIN,   // no rotation
  PAIRS,   // interleaved, rot_dim a multiple of 8: partners within the lane
  HALVES,  // half layout, rot_dim a multiple of 16: partners in one other aligned group of eight
  ANY      // everything else, element by element (8,191 x 40 x 128, 100 of them turned: 65 to 72 us instead of 40)
};
Layout layout_of(const qg_rope& p) {
  return p.interleaved ? (p.rot_dim % 8 ? ANY : PAIRS) : (p.rot_dim % 16 ? ANY : HALVES);
}

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
// Four consecutive elements, aligned to four.
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const __half* p, float (&v)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__half* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// The larger of two magnitudes; a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sines and cosines (times mscale) of the block's tokens: sc[token][pair].
__device__ __forceinline__ void make_turns(const qg_rope& plan, float2* sc, const int32_t* pos, int64_t tok0,
                                           int tokens, int64_t ntok) {
  const int half = plan.rot_dim >> 1;
  for (int i = threadIdx.x; i < tokens * half; i += ROW_THREADS) {
    const int t = i / half, pair = i - t * half;
    if (tok0 + t < ntok) {
      const uint64_t phase = plan.step[pair] * (uint64_t)(int64_t)pos[tok0 + t];
      // the turn's fraction, signed, in half turns
      const float half_turns = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31
      float sn, cs;
      sincospif(half_turns, &sn, &cs);
      sc[t * (QG_ROPE_MAX_DIM / 2) + pair] = make_float2(sn * plan.mscale, cs * plan.mscale);
    }
  }
}

// A lane's share of a token's rotation: elements d0 .. d0 + 7 of every row.
template <int LAYOUT>
struct Turn {
  float c[LAYOUT == PAIRS ? 4 : 8], s[LAYOUT == PAIRS ? 4 : 8];
  bool turned;   // the lane has elements that turn (all eight, but for ANY)
  int partner;   // HALVES: offset of the other group; its sines carry the sign
  Turn() = default;
  __device__ __forceinline__ Turn(const qg_rope& plan, const float2* sc, int d0) {
    const int rot = plan.rot_dim, h = rot >> 1;
    turned = d0 < rot;
    partner = 0;
    if (!turned) return;
    if constexpr (LAYOUT == PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = sc[(d0 >> 1) + i];
        s[i] = x.x;
        c[i] = x.y;
      }
    } else if constexpr (LAYOUT == HALVES) {
      partner = d0 < h ? h : -h;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 x = sc[(d0 < h ? d0 : d0 - h) + e];
        s[e] = d0 < h ? -x.x : x.x;
        c[e] = x.y;
      }
    } else if constexpr (LAYOUT == ANY) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = d0 + e;
        c[e] = 1.f;
        s[e] = 0.f;
        if (d < rot) {
          const bool second = plan.interleaved ? (d & 1) : d >= h;
          const float2 x = sc[plan.interleaved ? d >> 1 : second ? d - h : d];
          c[e] = x.y;
          s[e] = second ? x.x : -x.x;
        }
      }
    }
  }
  // The turned values of a lane's eight elements; `row` points at element 0 of the head. Every element of
  // the head is read before the caller's __syncwarp, so the result may overwrite it after.
  template <class T>
  __device__ __forceinline__ void apply(const qg_rope& plan, const T* row, int d0, const float (&x)[8],
                                        float (&y)[8]) const {
    if (LAYOUT == PLAIN || !turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x[e];
      return;
    }
    if constexpr (LAYOUT == PAIRS) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[2 * i] = fmaf(x[2 * i], c[i], -(x[2 * i + 1] * s[i]));
        y[2 * i + 1] = fmaf(x[2 * i + 1], c[i], x[2 * i] * s[i]);
      }
    } else if constexpr (LAYOUT == HALVES) {
      float o[8];
      load8(row + d0 + partner, o);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = fmaf(x[e], c[e], o[e] * s[e]);
    } else {
      const int rot = plan.rot_dim, h = rot >> 1;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int d = d0 + e;
        y[e] = x[e];
        if (d < rot) y[e] = fmaf(x[e], c[e], elem(row + (plan.interleaved ? d ^ 1 : d < h ? d + h : d - h)) * s[e]);
      }
    }
  }
};

// Where a row need not come out as aligned groups of eight, HALVES is done by quads: lane l < rot_dim / 8 turns the
// pairs 4l .. 4l+3, elements 4l .. and rot_dim/2 + 4l .., and every element is read once.
template <int LAYOUT>
struct RowTurn : Turn<LAYOUT> {
  __device__ __forceinline__ RowTurn(const qg_rope&, int) {}
  __device__ __forceinline__ void angles(const qg_rope& plan, const float2* sc, int d0) {
    Turn<LAYOUT>::operator=(Turn<LAYOUT>(plan, sc, d0));
  }
  // load: the lane's elements of a row; turn: the turned values of what was loaded from it; write: to where they belong.
  template <class TI>
  __device__ __forceinline__ void load(const TI* row, int d0, float (&x)[8]) const {
    load8(row + d0, x);
  }
  template <class TI>
  __device__ __forceinline__ void turn(const qg_rope& plan, const TI* row, int d0, const float (&x)[8],
                                       float (&y)[8]) const {
    this->apply(plan, row, d0, x, y);
  }
  template <class TO>
  __device__ __forceinline__ void write(TO* row, int d0, const float (&y)[8]) const {
    store8(row + d0, y);
  }
};
template <>
struct RowTurn<HALVES> {
  float c[4], s[4];
  int a, b;  // the lane's two quads
  bool turned;
  __device__ __forceinline__ RowTurn(const qg_rope& plan, int d0) {
    turned = d0 < plan.rot_dim;
    a = turned ? d0 >> 1 : d0;
    b = turned ? (plan.rot_dim + d0) >> 1 : d0 + 4;
  }
  __device__ __forceinline__ void angles(const qg_rope&, const float2* sc, int) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = turned ? sc[a + i] : make_float2(0.f, 1.f);
      s[i] = x.x;
      c[i] = x.y;
    }
  }
  template <class TI>
  __device__ __forceinline__ void load(const TI* row, int, float (&x)[8]) const {
    float u[4], v[4];
    load4(row + a, u);
    load4(row + b, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = u[i];
      x[4 + i] = v[i];
    }
  }
  template <class TI>
  __device__ __forceinline__ void turn(const qg_rope&, const TI*, int, const float (&x)[8], float (&y)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = turned ? fmaf(x[i], c[i], -(x[4 + i] * s[i])) : x[i];
      y[4 + i] = turned ? fmaf(x[4 + i], c[i], x[i] * s[i]) : x[4 + i];
    }
  }
  template <class TO>
  __device__ __forceinline__ void write(TO* row, int, const float (&y)[8]) const {
    store4(row + a, y);
    store4(row + b, y + 4);
  }
};

// Lanes of a row: D/8 rounded up to a power of two.
__host__ __device__ inline int row_lanes(int d) {
  int l = 1;
  while (l * 8 < d) l *= 2;
  return l;
}

// Warps of a token: as many as fill the machine (152 SMs x 40 warps) where there are few tokens, two at
// least, no more than it has row groups.
struct RowSplit {
  int parts;   // warps of a token in a block: 1, 2 or 4
  dim3 grid;
};
RowSplit split_rows(int ntok, int groups) {
  int want = (152 * 40 + ntok - 1) / ntok;
  if (want < 2) want = 2;
  if (want > groups) want = groups;
  RowSplit r;
  r.parts = 1;
  while (r.parts < want && r.parts < ROW_WARPS) r.parts *= 2;
  const int tokens = ROW_WARPS / r.parts;
  r.grid = dim3((unsigned)((ntok + (int64_t)tokens - 1) / tokens), (unsigned)((want + r.parts - 1) / r.parts));
  return r;
}

// ------------------------------------------------------------------- qrope
template <class TI, class TO, int LAYOUT>
__global__ void __launch_bounds__(ROW_THREADS, ROW_BLOCKS) rope_kernel(
    const __grid_constant__ qg_rope plan, const TI* x, int64_t xs, const int32_t* pos, int ntok,
    int n_heads, int d, TO* y, int64_t ys, int parts) {
  __shared__ float2 sc[ROW_WARPS * (QG_ROPE_MAX_DIM / 2)];
  pdl_trigger();
  pdl_wait();
  const int tokens = ROW_WARPS / parts;
  const int64_t tok0 = (int64_t)blockIdx.x * tokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok = tok0 + warp / parts;
  const int lanes = row_lanes(d), at_once = 32 / lanes, d0 = (lane & (lanes - 1)) * 8;
  const int step = at_once * parts * gridDim.y;
  int r = (warp % parts + parts * blockIdx.y) * at_once + lane / lanes;
  const TI* xr = x + tok * xs + (int64_t)r * d;
  TO* yr = y + tok * ys + (int64_t)r * d;
  const int64_t hop = (int64_t)step * d;
  if (d0 >= d || tok >= ntok) r = n_heads;  // no elements for this lane
  RowTurn<LAYOUT> t(plan, d0);
  float x8[8], v[8];
  if (r < n_heads) t.load(xr, d0, x8);  // the first row is on its way while the angles are found
  make_turns(plan, sc, pos, tok0, tokens, ntok);
  __syncthreads();
  t.angles(plan, sc + warp / parts * (QG_ROPE_MAX_DIM / 2), d0);
  while (__any_sync(0xffffffffu, r < n_heads)) {
    if (r < n_heads) t.turn(plan, xr, d0, x8, v);
    __syncwarp();  // in place: the row has been read
    if (r < n_heads) t.write(yr, d0, v);
    r += step;
    xr += hop;
    yr += hop;
    if (r < n_heads) t.load(xr, d0, x8);
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
  int parts;
};

// Where a lane's eight elements of a row, and their block's scale, go in a half record.
template <int TYPE>
struct Spot {
  int at, scale_at;  // bytes; scale_at < 0: another lane writes it
  __device__ __forceinline__ Spot(int d0, int d, int i) {
    const int blk = d0 >> 5;
    at = (blk * (KV_GROUP * 32) + i * 32 + (d0 & 31)) * (TYPE == QG_F16 ? 2 : 1);
    scale_at = (d0 & 31) == 0 ? KV_GROUP * d + 2 * (blk * KV_GROUP + kv_scale_place(i)) : -1;
  }
};

// Eight elements of a row into its half record (NULL: nowhere; the lanes of a block call together).
//
// Q8_0. The scale is the smallest f16 h with 127 h >= the block's largest magnitude. The product with R, a little
// above 1/127, rounded up is that h or the f16 behind it, and 127 h is exact in f32 (18 bits), so one comparison
// decides. x / h by an approximate reciprocal is off by at most 127 (2^-23 + 2^-24) < 2.3e-5; only next to a half is the
// division needed to know the nearest integer q. 1.5 2^23 + 128 + q has q + 128 as its low byte.
// (With two IEEE divisions a block, a clamp and a test an element, key and value rows took most of the kernel's issue
// slots: a prompt of 16,382 tokens, appended and read back, 142 us instead of 135.)
template <int TYPE>
__device__ __forceinline__ void put8(uint8_t* half, const Spot<TYPE>& spot, float (&y)[8]) {
  if constexpr (TYPE == QG_F16) {
    if (half) store8(reinterpret_cast<__half*>(half + spot.at), y);
  } else {
    float top = fabsf(y[0]);  // an infinity or a NaN stays one
#pragma unroll
    for (int e = 1; e < 8; ++e) top = max_nan(top, fabsf(y[e]));
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
    constexpr float R = 0x1.02040cp-7f;
    uint32_t bits = __half_as_ushort(__float2half_ru(top * R));
    if (127.f * __half2float(__ushort_as_half(bits - 1)) >= top) --bits;  // (false for 0 - 1, a NaN)
    const bool bad = !(top <= 3.402823466e38f), high = bits > 0x7BFF;
    if (high) bits = 0x7BFF;
    if (bad) bits = 0x7FFF;
    uint32_t w[2] = {0x80808080u, 0x80808080u};
    if (!bad && bits != 0) {
      const float ds = __half2float(__ushort_as_half(bits)), magic = 12582912.f + 128.f;
      float inv;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(ds));
      float b[8], off = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 q = mul2(make_float2(y[e], y[e + 1]), make_float2(inv, inv));
        const float2 m = sub2(q, make_float2(-magic, -magic));
        const float2 r = sub2(q, sub2(m, make_float2(magic, magic)));
        off = fmaxf(off, fmaxf(fabsf(r.x), fabsf(r.y)));
        b[e] = m.x;
        b[e + 1] = m.y;
      }
      if (off > 0.49996f || high)
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = fminf(fmaxf(__fdiv_rn(y[e], ds), -127.f), 127.f) + magic;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[h] = __byte_perm(__byte_perm(__float_as_uint(b[4 * h]), __float_as_uint(b[4 * h + 1]), 0x0040),
                           __byte_perm(__float_as_uint(b[4 * h + 2]), __float_as_uint(b[4 * h + 3]), 0x0040), 0x5410);
    }
    if (half) {
      *reinterpret_cast<uint2*>(half + spot.at) = make_uint2(w[0], w[1]);
      if (spot.scale_at >= 0) *reinterpret_cast<uint16_t*>(half + spot.scale_at) = (uint16_t)bits;
    }
  }
}

template <class T, int TYPE, int LAYOUT>
__global__ void __launch_bounds__(ROW_THREADS, APPEND_BLOCKS)
    append_kernel(const __grid_constant__ qg_rope plan, const __grid_constant__ AppendParams<T> a) {
  __shared__ float2 sc[ROW_WARPS * (QG_ROPE_MAX_DIM / 2)];
  pdl_trigger();
  pdl_wait();
  const int tokens = ROW_WARPS / a.parts;
  const int64_t tok0 = (int64_t)blockIdx.x * tokens;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok = tok0 + warp / a.parts;
  const int d = a.c.head_dim, lanes = d >> 3, at_once = 32 / lanes, d0 = (lane & (lanes - 1)) * 8;
  // Row groups of the token in order: queries, keys, values; the parts take them in turn. The first queries are on
  // their way while the place and the angles are found.
  const int part = warp % a.parts + a.parts * blockIdx.y, all_parts = a.parts * gridDim.y;
  const int first = lane / lanes;
  const int qg = (a.n_q + at_once - 1) / at_once, kg = (a.c.n_kv_heads + at_once - 1) / at_once;
  const T* row = a.q + tok * a.qs + (int64_t)(part * at_once + first) * d;
  float next[8];
  RowTurn<LAYOUT> tq(plan, d0);
  if (tok < a.ntok && part * at_once + first < a.n_q) tq.load(row, d0, next);
  // the token's place in the cache (NULL: nowhere)
  uint8_t* place = nullptr;
  const int groups = a.c.page_size / KV_GROUP, rec = kv_record_bytes(TYPE, d);
  int in_group = 0;
  if (tok < a.ntok) {
    const int pos = a.pos[tok];
    if (pos >= 0) {
      int bits = 0;
      const int seq = a.seq ? a.seq[tok] : (int)(tok / a.per_seq);
      const int page = kv_page_of(a.c, seq, pos, &bits);
      const int slot = pos & (a.c.page_size - 1);
      in_group = slot & (KV_GROUP - 1);
      if (page >= 0)
        place = static_cast<uint8_t*>(a.c.pool) + ((size_t)page * a.c.n_kv_heads * groups + slot / KV_GROUP) * rec;
      else if (part == 0 && lane == 0 && a.err)
        atomicOr(a.err, bits);
    }
  }
  if (LAYOUT != PLAIN) {
    make_turns(plan, sc, a.pos, tok0, tokens, a.ntok);
    __syncthreads();
  }
  if (tok >= a.ntok) return;
  const float2* const my_sc = sc + warp / a.parts * (QG_ROPE_MAX_DIM / 2);
  int n = part;
  {
    tq.angles(plan, my_sc, d0);
    const int64_t hop = (int64_t)all_parts * at_once * d;
    for (; n < qg; n += all_parts, row += hop) {
      const int r = n * at_once + first;
      float x[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = next[e];
      if (r + all_parts * at_once < a.n_q) tq.load(row + hop, d0, next);
      if (r < a.n_q) {
        tq.turn(plan, row, d0, x, y);
        tq.write(a.q_out + (tok * a.n_q + r) * (int64_t)d, d0, y);
      }
    }
  }
  const Turn<LAYOUT> t(plan, my_sc, d0);
  const Spot<TYPE> spot(d0, d, in_group);
  const uint32_t head_bytes = groups * rec;
  const int kv = a.c.n_kv_heads;
  const T* const kr = a.k + tok * a.ks;
  for (n -= qg; n < kg; n += all_parts) {
    const int r = n * at_once + first;
    float x[8], y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < kv) {
      load8(kr + r * d + d0, x);
      t.apply(plan, kr + r * d, d0, x, y);
    }
    put8<TYPE>(place && r < kv ? place + (size_t)r * head_bytes : nullptr, spot, y);
  }
  const T* const vr = a.v + tok * a.vs + d0;
  for (n -= kg; n < kg; n += all_parts) {
    const int r = n * at_once + first;
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r < kv) load8(vr + r * d, y);
    put8<TYPE>(place && r < kv ? place + (size_t)r * head_bytes + kv_half_bytes(TYPE, d) : nullptr, spot, y);
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
  const int at_once = 256 / a.c.head_dim;
  const int kg = (a.c.n_kv_heads + at_once - 1) / at_once, qg = (a.n_q + at_once - 1) / at_once;
  const RowSplit sp = split_rows(a.ntok, qg + 2 * kg);
  p.parts = sp.parts;
  qg_rope plan{};
  if (a.rope) plan = *a.rope;
  const Layout l = a.rope ? layout_of(plan) : PLAIN;
  const auto kern = l == PLAIN    ? append_kernel<T, TYPE, PLAIN>
                    : l == PAIRS  ? append_kernel<T, TYPE, PAIRS>
                    : l == HALVES ? append_kernel<T, TYPE, HALVES>
                                  : append_kernel<T, TYPE, ANY>;
  return launch_pdl(kern, sp.grid, dim3(ROW_THREADS), 0, s, 0, LC_L1, plan, p);
}

template <class TI, class TO>
cudaError_t rope_typed(const qg_rope& plan, const void* x, int64_t xs, const int32_t* pos, int ntok,
                       int n_heads, int d, void* y, int64_t ys, cudaStream_t s) {
  const int at_once = 32 / row_lanes(d);
  const RowSplit sp = split_rows(ntok, (n_heads + at_once - 1) / at_once);
  const Layout l = layout_of(plan);
  const auto kern = l == PAIRS    ? rope_kernel<TI, TO, PAIRS>
                    : l == HALVES ? rope_kernel<TI, TO, HALVES>
                                  : rope_kernel<TI, TO, ANY>;
  return launch_pdl(kern, sp.grid, dim3(ROW_THREADS), 0, s, 0, LC_L1, plan, static_cast<const TI*>(x), xs, pos, ntok,
                    n_heads, d, static_cast<TO*>(y), ys, sp.parts);
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
