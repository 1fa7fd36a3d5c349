// qg_attn.cu -- attention of new tokens over the paged key/value cache
// (qattn_paged).
//
// Mathematics. For a row (a query of one column and head) with scores s_j over
// the tokens it sees, y = sum_j 2^(s_j - m) V_j / sum_j 2^(s_j - m) for any m,
// scores in units of log 2. A run of tokens is summed with its own running
// maximum m; two runs are joined by scaling each with 2^(m_run - m_both). So the
// tokens may be cut into runs anywhere, and every byte of the cache is read once.
//
// Work. The rows of one kv head (all its query heads, all columns; 16 to a
// tile, the m of an m16n8k16 mma) share its keys and values. An item is a
// (sequence, kv head, row tile); its tokens come in units of 64 (four warps x a
// record of 16 tokens). All items' units in a row are cut into equal runs, one
// for each CTA of a grid that fills the machine once, so a batch of ragged
// lengths and one very long sequence load every SM alike. A CTA that covers an
// item whole writes y; where an item is cut, each CTA writes its sum, maximum
// and weight to the workspace, and a second kernel joins them in CTA order. The
// cuts depend on lens and the shape alone, and so do the results.
//
// Inside a CTA each warp is on its own: it has a ring of shared-memory slots,
// fetches the key half and the value half of its records with bulk copies (one
// lane for each, a slot refilled as soon as it is consumed), and keeps a
// running maximum, sum and its 16 x D accumulator in registers. The four warps
// meet only at the end of an item. Page numbers of 32 steps are loaded by the 32
// lanes at once, a batch ahead.
//
// Scores: A = Q (16 rows), B = K. The 32 dimensions of a block are given to
// the lanes of a quad as 8 neighbouring ones each, the same in A and B, so a
// lane's operands are one load. Weights: the accumulator layout of the scores
// is the A layout of the second product, with lane t of a quad holding tokens
// t, t + 4, t + 8, t + 12; V's pairs of tokens are put together by byte
// permutation after plain row loads.
//
// Q8_0: quants are stored as u = q + 128. As the low byte of an f16 u is the
// subnormal u 2^-24, exact on the tensor cores, so K needs one byte permutation
// for two elements: sum_d Q_d q_d = sum_d Q_d u_d - 128 sum_d Q_d, the last
// term being the initial accumulator. A block's sum is then multiplied by its
// scale in f32. V's u becomes the f16 integer q (exponent trick, exact), and
// the block's scale is multiplied into the f32 weight before the weight is
// rounded to f16 (so V itself is never rounded); a power of two that follows
// the largest scale seen keeps that product in the normal range of f16.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qg_async.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_kv.cuh"
#include "qg_mma.cuh"

namespace qg {

__device__ int32_t g_attn_error;

namespace {

constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = AT_WARPS * 32;
constexpr int AT_ROWS = 16;                      // rows of a tile
constexpr int AT_UNIT = AT_WARPS * KV_GROUP;     // tokens of a unit
constexpr int AT_SMS = 152;
constexpr int AT_OPITCH = 68;                    // floats of a row of 64 in the join buffer: no bank conflicts

template <int TYPE, int D>
struct AttnCfg {
  // CTAs per SM: 128 threads each; the accumulator takes D / 2 registers
  static constexpr int CPS = D == 64 ? 4 : D == 128 ? 3 : 2;
  static constexpr int GRID = AT_SMS * CPS;
  static constexpr int HALF = kv_half_bytes(TYPE, D);
  static constexpr int SLOT = (HALF + 127) / 128 * 128;
  // slots of a warp's ring: as many as leave CPS CTAs on an SM
  static constexpr int SLOTS = TYPE == QG_F16 ? (D == 64 ? 4 : D == 128 ? 3 : 2) : (D == 256 ? 4 : 6);
  static constexpr int NB = D / 32;
  static constexpr bool QSMEM = D == 256;  // Q fragments in shared memory, not registers
  static constexpr size_t ring = (size_t)AT_WARPS * SLOTS * SLOT;
  static constexpr size_t obuf = (size_t)AT_WARPS * AT_ROWS * AT_OPITCH * 4;
  static constexpr size_t stats = 2 * 2 * AT_WARPS * AT_ROWS * 4;
  static constexpr size_t qbuf = QSMEM ? (size_t)NB * 32 * 32 + NB * AT_ROWS * 4 : 0;
  static constexpr size_t bars = (size_t)AT_WARPS * SLOTS * 8;
  static size_t smem(int n_seq) {
    return ring + obuf + stats + qbuf + bars + (size_t)(n_seq + 1) * 8 + (size_t)n_seq * 4 + 16;
  }
};

// What a CTA tells the joining kernel about the item that its run starts in.
struct AttnCut {
  int32_t first;   // 1: this CTA is the second that has a part of the item (and joins for it)
  int32_t c0, c1;  // the item's CTAs
  int32_t seq, head, tile;
  int32_t pad[2];
};

struct AttnWs {
  AttnCut* cut;  // [GRID]
  float* ml;     // [GRID][2][rows][2]
  float* o;      // [GRID][2][rows][D]
};

struct AttnDev {
  AttnArgs a;
  AttnWs ws;
  int group;   // query heads of a kv head
  int tiles;   // row tiles of a kv head
  float scale; // times log2 e
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The CTA whose run holds unit u of n, run c being [c n / N, (c+1) n / N).
__device__ __forceinline__ int run_of(int64_t u, int64_t n, int64_t N) { return (int)(((u + 1) * N - 1) / n); }

// Units of the sequences: position of the first token that any row sees,
// and the number of units (at least one, so that every item is written by some CTA).
struct SeqSpan {
  int lo;   // first token that any row sees
  int hi;   // one past the last
  int unit; // first unit
  int n;    // units
};
__device__ __forceinline__ SeqSpan span_of(const AttnArgs& a, int len) {
  SeqSpan s;
  const int cap = a.c.max_pages * a.c.page_size;
  s.hi = len < cap ? len : cap;
  const int64_t lo = (int64_t)len - a.ncols - a.window + 1;
  s.lo = a.window > 0 && lo > 0 ? (int)lo : 0;
  s.unit = s.lo / AT_UNIT;
  const int end = (int)(((int64_t)s.hi + AT_UNIT - 1) / AT_UNIT);
  s.n = end - s.unit > 1 ? end - s.unit : 1;
  return s;
}

template <int TYPE, int D>
__global__ void __launch_bounds__(AT_THREADS, AttnCfg<TYPE, D>::CPS)
    attn_kernel(const __grid_constant__ AttnDev p) {
  using C = AttnCfg<TYPE, D>;
  constexpr int NB = C::NB;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* const s_ring = smem;
  float* const s_o = reinterpret_cast<float*>(smem + C::ring);
  float* const s_stat = reinterpret_cast<float*>(smem + C::ring + C::obuf);  // [parity][m | l][warp][row]
  uint8_t* const s_q = smem + C::ring + C::obuf + C::stats;
  uint64_t* const s_bar = reinterpret_cast<uint64_t*>(s_q + C::qbuf);
  int64_t* const s_first = reinterpret_cast<int64_t*>(s_bar + AT_WARPS * C::SLOTS);  // units before a sequence
  int32_t* const s_len = reinterpret_cast<int32_t*>(s_first + p.a.c.n_seq + 1);
  __shared__ int64_t s_part[AT_WARPS];

  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  pdl_trigger();
  if (tid < AT_WARPS * C::SLOTS) {
    mbar_init(s_bar + tid, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  // units of every sequence, and their running sum
  const int n_seq = a.c.n_seq;
  {
    const int per = (n_seq + AT_THREADS - 1) / AT_THREADS;
    const int b0 = tid * per, b1 = min(b0 + per, n_seq);
    const int cap = a.c.max_pages * a.c.page_size;
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) {
      int len = a.lens[b];
      if ((len < 0 || len > cap) && blockIdx.x == 0 && a.err) atomicOr(a.err, QG_KV_BAD_POS);
      len = max(len, 0);
      s_len[b] = len;
      sum += span_of(a, len).n;
    }
    int64_t run = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += up;
    }
    if (lane == 31) s_part[warp] = run;
    __syncthreads();
    int64_t before = run - sum;
    for (int w = 0; w < warp; ++w) before += s_part[w];
    for (int b = b0; b < b1; ++b) {
      s_first[b] = before;
      before += span_of(a, s_len[b]).n;
    }
    if (b1 == n_seq && b0 < n_seq) s_first[n_seq] = before;
    __syncthreads();
  }
  const int per_unit = a.c.n_kv_heads * p.tiles;  // items of a sequence
  const int64_t units = s_first[n_seq] * per_unit;
  const int64_t N = units < C::GRID ? units : C::GRID;
  const int cta = blockIdx.x;
  const int64_t u0 = cta < N ? cta * units / N : 0, u1 = cta < N ? (cta + 1) * units / N : 0;
  const int steps = (int)(u1 - u0 < 0x7fffffff ? u1 - u0 : 0x7fffffff);

  // the sequence that holds unit u: the last whose items start at or before it
  auto seq_of = [&](int64_t u) {
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_first[mid] * per_unit <= u) lo = mid; else hi = mid;
    }
    return lo;
  };

  if (tid == 0) {
    AttnCut cut{};
    if (cta < N) {
      const int b = seq_of(u0);
      const int64_t nu = s_first[b + 1] - s_first[b], rem = u0 - s_first[b] * per_unit;
      const int hr = (int)(rem / nu);
      const int64_t i0 = s_first[b] * per_unit + hr * nu;
      if (i0 < u0) {
        cut.c0 = run_of(i0, units, N);
        cut.c1 = run_of(i0 + nu - 1, units, N);
        cut.first = cta == cut.c0 + 1;
        cut.seq = b;
        cut.head = hr / p.tiles;
        cut.tile = hr % p.tiles;
      }
    }
    p.ws.cut[cta] = cut;
  }
  if (steps == 0) return;

  // ------------------------------------------------------------ the ring
  const int gpp = a.c.page_size / KV_GROUP;  // records of a page and head
  uint8_t* const ring = s_ring + (size_t)warp * C::SLOTS * C::SLOT;
  const uint32_t ring_at = smem_u32(ring), bar_at = smem_u32(s_bar + warp * C::SLOTS);
  // Page numbers: lane i looks up step base + i. Raw until the batch is entered,
  // so that the load has the whole batch before to arrive.
  int nx_page = -1, nx_off = 0;
  bool nx_in = false;
  auto look_up = [&](int base) {
    nx_in = false;
    nx_page = -1;
    if (base + lane < steps) {
      const int64_t u = u0 + base + lane;
      const int b = seq_of(u);
      const int64_t nu = s_first[b + 1] - s_first[b], rem = u - s_first[b] * per_unit;
      const int hr = (int)(rem / nu), un = (int)(rem - hr * nu);
      const SeqSpan sp = span_of(a, s_len[b]);
      const int64_t grp = (int64_t)(sp.unit + un) * AT_WARPS + warp;
      if (grp * KV_GROUP < sp.hi && grp * KV_GROUP + KV_GROUP > sp.lo) {
        nx_in = true;
        nx_page = a.c.page_table[(size_t)b * a.c.max_pages + (int)(grp / gpp)];
        nx_off = (hr / p.tiles) * gpp + (int)(grp % gpp);
      }
    }
  };
  const uint8_t* my_rec = nullptr;        // this lane's record of the batch in issue
  uint32_t valid_even = 0, valid_odd = 0;  // steps of the even / odd batches that have a record
  auto enter = [&](int step) {             // step: a multiple of 32
    my_rec = nullptr;
    if (nx_in) {
      if (nx_page >= 0 && nx_page < a.c.n_pages)
        my_rec = static_cast<const uint8_t*>(a.c.pool) +
                 ((size_t)nx_page * a.c.n_kv_heads * gpp + nx_off) * (2 * C::HALF);
      else if (a.err)
        atomicOr(a.err, QG_KV_BAD_PAGE);
    }
    const uint32_t v = __ballot_sync(0xffffffffu, my_rec != nullptr);
    if (step & 32) valid_odd = v; else valid_even = v;
    look_up(step + 32);
  };
  int is_step = 0, is_v = 0, is_slot = 0;  // the next half to fetch and its slot
  auto issue = [&]() {
    if (is_step < steps) {
      if (!is_v && (is_step & 31) == 0) enter(is_step);
      if (lane == (is_step & 31) && my_rec) {
        const uint32_t bar = bar_at + 8 * is_slot;
        mbar_expect_tx(bar, C::HALF);
        bulk_g2s(ring_at + is_slot * C::SLOT, my_rec + is_v * C::HALF, C::HALF, bar);
      }
      is_step += is_v;
      is_v ^= 1;
      is_slot = is_slot + 1 == C::SLOTS ? 0 : is_slot + 1;
    }
  };
  __syncwarp();
  look_up(0);
  for (int i = 0; i < C::SLOTS; ++i) issue();

  int co_slot = 0;        // the slot of the next half to consume
  uint32_t phases = 0;    // parity of each slot's next phase
  bool ok = true;         // false (in all lanes) once a wait gave up: no more copies, no more waits
  auto arrived = [&]() {
    if (ok)
      ok = __all_sync(0xffffffffu, mbar_wait(bar_at + 8 * co_slot, (phases >> co_slot) & 1, &g_attn_error));
    phases ^= 1u << co_slot;
    return ring_at + co_slot * C::SLOT;
  };
  // The slot's reads are over: every lane orders its own before the refill.
  auto release = [&]() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (ok) issue();
    co_slot = co_slot + 1 == C::SLOTS ? 0 : co_slot + 1;
  };

  // --------------------------------------------------------------- items
  const int rows = p.group * a.ncols;
  int parity = 0;
  int64_t u = u0;
  int step = 0;
  int b = seq_of(u0);
  while (u < u1) {
    while (s_first[b + 1] * per_unit <= u) ++b;
    const int64_t nu = s_first[b + 1] - s_first[b], base = s_first[b] * per_unit;
    const int hr = (int)((u - base) / nu);
    const int64_t i0 = base + hr * nu, i1 = i0 + nu;
    const int64_t uend = i1 < u1 ? i1 : u1;
    const int head = hr / p.tiles, tile = hr % p.tiles;
    const int len = s_len[b];
    const SeqSpan sp = span_of(a, len);

    // rows g and g + 8 of the tile: what they see, and their queries
    int row_hi[2], row_lo[2];  // tokens row_lo < j <= row_hi
    const uint16_t* row_q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = tile * AT_ROWS + g + 8 * i;
      const int col = r / p.group;
      const int64_t pos = (int64_t)len - a.ncols + col;
      row_hi[i] = r < rows ? (int)(pos < sp.hi - 1 ? pos : sp.hi - 1) : -1;
      row_lo[i] = a.window > 0 && pos - a.window > -1 ? (int)(pos - a.window) : -1;
      row_q[i] = r < rows ? a.q + (((size_t)b * a.ncols + col) * a.n_heads + head * p.group + r % p.group) * D + 8 * t
                          : nullptr;
    }
    // tokens that all rows see: no mask needed from `lo_all` up to `hi_all`
    const int hi_all = (int)min((int64_t)sp.hi - 1, (int64_t)len - a.ncols);
    const int lo_all = a.window > 0 ? (int)max((int64_t)0, (int64_t)len - a.window) : 0;

    uint32_t qf[C::QSMEM ? 1 : NB][8];
    float qc[C::QSMEM || TYPE == QG_F16 ? 1 : NB][2];  // -128 2^-24 sum of a block's queries
    auto load_q = [&](int blk, uint32_t (&w)[8], float (&c)[2]) {
      uint4 x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        x[i] = row_q[i] ? *reinterpret_cast<const uint4*>(row_q[i] + 32 * blk) : make_uint4(0, 0, 0, 0);
      w[0] = x[0].x; w[1] = x[1].x; w[2] = x[0].y; w[3] = x[1].y;  // first k-step of the block: A0..A3
      w[4] = x[0].z; w[5] = x[1].z; w[6] = x[0].w; w[7] = x[1].w;  // second
      if constexpr (TYPE == QG_Q8_0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) s += lo_f32(w[2 * k + i]) + hi_f32(w[2 * k + i]);
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          c[i] = s * -7.62939453125e-06f;  // -128 * 2^-24
        }
      }
    };
    if constexpr (C::QSMEM) {
      // in fragment order [block][lane][8 words]; the sums by row behind them
      for (int blk = warp; blk < NB; blk += AT_WARPS) {
        uint32_t w[8];
        float c[2];
        load_q(blk, w, c);
        uint4* dst = reinterpret_cast<uint4*>(s_q + blk * 1024 + lane * 16);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[32] = make_uint4(w[4], w[5], w[6], w[7]);
        if (TYPE == QG_Q8_0 && t == 0) {
          float* s = reinterpret_cast<float*>(s_q + NB * 1024) + blk * AT_ROWS;
          s[g] = c[0];
          s[g + 8] = c[1];
        }
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        float c[2] = {0.f, 0.f};
        load_q(blk, qf[blk], c);
        if constexpr (TYPE == QG_Q8_0) {
          qc[blk][0] = c[0];
          qc[blk][1] = c[1];
        }
      }
    }

    float o[NB][4][4];
#pragma unroll
    for (int i = 0; i < NB * 16; ++i) o[i / 16][(i / 4) & 3][i & 3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // Q8_0: weights are multiplied by their scale and 2^(15 - wexp); scales
    // above `wmax` = 2^wexp move it up
    float wmul = TYPE == QG_F16 ? 1.f : 0.f, wmax = TYPE == QG_F16 ? 1.f : 0.f, wback = 1.f;

    for (; u < uend; ++u, ++step) {
      const uint32_t valid = (step & 32) ? valid_odd : valid_even;
      if (!((valid >> (step & 31)) & 1)) {  // nothing of this record is seen, or its page is bad
        release();
        release();
        continue;
      }
      const int tok = (int)(((int64_t)sp.unit + (u - i0)) * AT_WARPS + warp) * KV_GROUP;
      const bool masked = tok + KV_GROUP - 1 > hi_all || tok < lo_all;

      // ---- scores of 16 rows x 16 tokens: s[j] tokens 8j + t and 8j + 4 + t
      float s[2][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i >> 2][i & 3] = 0.f;
      const uint32_t kb = arrived();
      const int ktok = (g >> 1) + 4 * (g & 1);  // the token whose row this lane loads, of eight
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        uint32_t q[8];
        if constexpr (C::QSMEM) {
          lds128(smem_u32(s_q) + blk * 1024 + lane * 16, q[0], q[1], q[2], q[3]);
          lds128(smem_u32(s_q) + blk * 1024 + 512 + lane * 16, q[4], q[5], q[6], q[7]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = qf[blk][i];
        }
        const uint32_t a0[4] = {q[0], q[1], q[2], q[3]}, a1[4] = {q[4], q[5], q[6], q[7]};
        if constexpr (TYPE == QG_F16) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t x, y, z, w;
            lds128(kb + blk * 1024 + (8 * j + ktok) * 64 + t * 16, x, y, z, w);
            mma16816_acc(s[j], a0, x, y);
            mma16816_acc(s[j], a1, z, w);
          }
        } else {
          float c0, c1;
          if constexpr (C::QSMEM) {
            const float* sums = reinterpret_cast<const float*>(s_q + NB * 1024) + blk * AT_ROWS;
            c0 = sums[g];
            c1 = sums[g + 8];
          } else {
            c0 = qc[blk][0];
            c1 = qc[blk][1];
          }
          uint32_t d0, d1;
          lds64(kb + KV_GROUP * D + blk * 32 + t * 8, d0, d1);  // scales of tokens t, 4+t | 8+t, 12+t
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t x, y;
            lds64(kb + blk * 512 + (8 * j + ktok) * 32 + t * 8, x, y);
            float part[4] = {c0, c0, c1, c1};
            mma16816_acc(part, a0, __byte_perm(x, 0, 0x4140), __byte_perm(x, 0, 0x4342));
            mma16816_acc(part, a1, __byte_perm(y, 0, 0x4140), __byte_perm(y, 0, 0x4342));
            const uint32_t d = j ? d1 : d0;
            const float e0 = lo_f32(d), e1 = hi_f32(d);
            s[j][0] = fmaf(part[0], e0, s[j][0]);
            s[j][1] = fmaf(part[1], e1, s[j][1]);
            s[j][2] = fmaf(part[2], e0, s[j][2]);
            s[j][3] = fmaf(part[3], e1, s[j][3]);
          }
        }
      }
      release();

      // ---- running maximum and weights
      const float mul = TYPE == QG_F16 ? p.scale : p.scale * 16777216.f;  // Q8_0: u was u 2^-24
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i >> 2][i & 3] *= mul;
      if (masked) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = tok + 8 * j + 4 * (i & 1) + t;
            if (at > row_hi[i >> 1] || at <= row_lo[i >> 1]) s[j][i] = -INFINITY;
          }
      }
      float top[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        top[i] = fmaxf(m[i], x);
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
        const float f0 = top[0] > m[0] ? ex2(m[0] - top[0]) : 1.f, f1 = top[1] > m[1] ? ex2(m[1] - top[1]) : 1.f;
        l[0] *= f0;
        l[1] *= f1;
#pragma unroll
        for (int i = 0; i < NB * 4; ++i) {
          o[i >> 2][i & 3][0] *= f0;
          o[i >> 2][i & 3][1] *= f0;
          o[i >> 2][i & 3][2] *= f1;
          o[i >> 2][i & 3][3] *= f1;
        }
        m[0] = top[0];
        m[1] = top[1];
      }
      {
        const float z0 = m[0] == -INFINITY ? 0.f : m[0], z1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[j][0] = ex2(s[j][0] - z0);
          s[j][1] = ex2(s[j][1] - z0);
          s[j][2] = ex2(s[j][2] - z1);
          s[j][3] = ex2(s[j][3] - z1);
        }
        l[0] += (s[0][0] + s[0][1]) + (s[1][0] + s[1][1]);
        l[1] += (s[0][2] + s[0][3]) + (s[1][2] + s[1][3]);
      }

      // ---- weights times values
      const uint32_t vb = arrived();
      uint8_t* const vp = ring + co_slot * C::SLOT;
      if constexpr (TYPE == QG_F16) {
        if (masked) {
          // Zero weights do not silence a NaN or an infinity in the product. So the rows of tokens that no
          // query row sees are cleared, and values that are not finite are taken out here and added, to the
          // rows that see them, below.
          uint32_t odd = 0;  // tokens with such values
          for (int i = lane; i < KV_GROUP * D / 8; i += 32) {
            uint4* at = reinterpret_cast<uint4*>(vp) + i;
            const int tk = tok + ((i >> 2) & 15);
            if (tk >= sp.hi || tk < sp.lo) {
              *at = make_uint4(0, 0, 0, 0);
            } else {
              const uint4 w = *at;
              const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if ((v[k] & 0x7C00u) == 0x7C00u || (v[k] & 0x7C000000u) == 0x7C000000u) odd |= 1u << ((i >> 2) & 15);
            }
          }
          odd = __reduce_or_sync(0xffffffffu, odd);
          while (odd) {
            const int k = __ffs(odd) - 1;
            odd &= odd - 1;
            const bool see0 = tok + k <= row_hi[0] && tok + k > row_lo[0];
            const bool see1 = tok + k <= row_hi[1] && tok + k > row_lo[1];
            __half* const row = reinterpret_cast<__half*>(vp) + k * 32;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  const float x = __half2float(row[blk * 512 + 8 * t + 4 * c + i]);
                  if (!(fabsf(x) <= 65504.f)) {
                    if (see0) o[blk][i][c] += x;
                    if (see1) o[blk][i][2 + c] += x;
                  }
                }
            __syncwarp();
            for (int e = lane; e < D; e += 32) {
              __half* const x = row + (e >> 5) * 512 + (e & 31);
              if (!(fabsf(__half2float(*x)) <= 65504.f)) *x = __ushort_as_half(0);
            }
          }
          __syncwarp();
        }
        const uint32_t pa[4] = {pack_f16(s[0][0], s[0][1]), pack_f16(s[0][2], s[0][3]),
                                pack_f16(s[1][0], s[1][1]), pack_f16(s[1][2], s[1][3])};
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          uint32_t x[4], y[4];  // tokens t, 4+t, 8+t, 12+t: dimensions 4g, 4g+1 | 4g+2, 4g+3
#pragma unroll
          for (int r = 0; r < 4; ++r) lds64(vb + blk * 1024 + (4 * r + t) * 64 + g * 8, x[r], y[r]);
          mma16816_acc(o[blk][0], pa, __byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
          mma16816_acc(o[blk][1], pa, __byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
          mma16816_acc(o[blk][2], pa, __byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410));
          mma16816_acc(o[blk][3], pa, __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632));
        }
      } else {
        if (masked) {  // scales of tokens that no row sees may be anything
          uint16_t* sc = reinterpret_cast<uint16_t*>(vp + KV_GROUP * D);
          for (int i = lane; i < NB * KV_GROUP; i += 32) {
            const int k = i & 15, tk = tok + (k >> 2) + 4 * (k & 3);
            if (tk >= sp.hi || tk < sp.lo) sc[i] = 0;
          }
          __syncwarp();
        }
        uint32_t d[NB][2];
        __half2 big = __float2half2_rn(0.f);
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          lds64(vb + KV_GROUP * D + blk * 32 + t * 8, d[blk][0], d[blk][1]);
          big = __hmax2(big, __hmax2(*reinterpret_cast<__half2*>(&d[blk][0]), *reinterpret_cast<__half2*>(&d[blk][1])));
        }
        float dmax = fmaxf(__low2float(big), __high2float(big));
        if (__any_sync(0xffffffffu, dmax > wmax)) {
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 1));
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 2));
          // dmax < 2^(e-1): scales may double before the next move, and weights stay below 2^15
          const int e = ((__float_as_int(dmax) >> 23) & 0xff) - 127 + 2;
          const float to = __int_as_float((127 + 15 - e) << 23);  // 2^(15-e)
          const float f = wmax == 0.f ? 1.f : to * wback;
          wmul = to;
          wmax = __int_as_float((127 + e) << 23);
          wback = __int_as_float((127 - 15 + e) << 23);
#pragma unroll
          for (int i = 0; i < NB * 16; ++i) o[i / 16][(i / 4) & 3][i & 3] *= f;
        }
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = s[i >> 2][i & 3] * wmul;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          const float e0 = lo_f32(d[blk][0]), e1 = hi_f32(d[blk][0]), e2 = lo_f32(d[blk][1]), e3 = hi_f32(d[blk][1]);
          float x[8] = {w[0] * e0, w[1] * e1, w[2] * e0, w[3] * e1, w[4] * e2, w[5] * e3, w[6] * e2, w[7] * e3};
          if (masked) {  // a zero weight times a NaN scale (a token that other rows see)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = w[i] == 0.f ? 0.f : x[i];
          }
          const uint32_t pa[4] = {pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7])};
          uint32_t v[4];  // tokens t, 4+t, 8+t, 12+t: dimensions 4g .. 4g+3
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[r] = lds32(vb + blk * 512 + (4 * r + t) * 32 + g * 4);
          const uint32_t lo0 = __byte_perm(v[0], v[1], 0x5140), lo1 = __byte_perm(v[2], v[3], 0x5140);
          const uint32_t hi0 = __byte_perm(v[0], v[1], 0x7362), hi1 = __byte_perm(v[2], v[3], 0x7362);
          const uint32_t k64 = 0x64646464u, k1152 = 0x64806480u;  // f16 1024 + u, less 1152
          mma16816_acc(o[blk][0], pa, hsub2_u(__byte_perm(lo0, k64, 0x4140), k1152), hsub2_u(__byte_perm(lo1, k64, 0x4140), k1152));
          mma16816_acc(o[blk][1], pa, hsub2_u(__byte_perm(lo0, k64, 0x4342), k1152), hsub2_u(__byte_perm(lo1, k64, 0x4342), k1152));
          mma16816_acc(o[blk][2], pa, hsub2_u(__byte_perm(hi0, k64, 0x4140), k1152), hsub2_u(__byte_perm(hi1, k64, 0x4140), k1152));
          mma16816_acc(o[blk][3], pa, hsub2_u(__byte_perm(hi0, k64, 0x4342), k1152), hsub2_u(__byte_perm(hi1, k64, 0x4342), k1152));
        }
      }
      release();
    }

    // ------------------------------------------------ the four warps' sums
    float* const s_m = s_stat + parity * 2 * AT_WARPS * AT_ROWS;
    float* const s_l = s_m + AT_WARPS * AT_ROWS;
    parity ^= 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (t == 0) {
        s_m[warp * AT_ROWS + g + 8 * i] = m[i];
        s_l[warp * AT_ROWS + g + 8 * i] = l[i];
      }
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = s_m[g + 8 * i];
#pragma unroll
      for (int w = 1; w < AT_WARPS; ++w) x = fmaxf(x, s_m[w * AT_ROWS + g + 8 * i]);
      f[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - x) * wback;
    }
    const bool whole = u0 <= i0 && i1 <= u1;
    const size_t part = (size_t)cta * 2 + (i0 < u0 ? 0 : 1);
#pragma unroll
    for (int pass = 0; pass < D / 64; ++pass) {
      if (pass) __syncthreads();  // the buffer has been read
#pragma unroll
      for (int hb = 0; hb < 2; ++hb) {
        const int blk = 2 * pass + hb;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float* dst = s_o + (warp * AT_ROWS + g + 8 * i) * AT_OPITCH + hb * 32 + t * 8;
#pragma unroll
          for (int c = 0; c < 2; ++c)
            *reinterpret_cast<float4*>(dst + 4 * c) =
                f[i] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(o[blk][0][2 * i + c] * f[i], o[blk][1][2 * i + c] * f[i],
                                          o[blk][2][2 * i + c] * f[i], o[blk][3][2 * i + c] * f[i]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < AT_ROWS * 16 / AT_THREADS; ++k) {
        const int row = (tid + k * AT_THREADS) >> 4, dim = ((tid & 15) << 2);
        const int r = tile * AT_ROWS + row;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < AT_WARPS; ++w) top = fmaxf(top, s_m[w * AT_ROWS + row]);
#pragma unroll
        for (int w = 0; w < AT_WARPS; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(s_o + (w * AT_ROWS + row) * AT_OPITCH + dim);
          y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
          const float mw = s_m[w * AT_ROWS + row];
          sum += mw == -INFINITY ? s_l[w * AT_ROWS + row] : s_l[w * AT_ROWS + row] * ex2(mw - top);
        }
        if (r < rows) {
          const int at = pass * 64 + dim;
          if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const size_t yo = (((size_t)b * a.ncols + r / p.group) * a.n_heads + head * p.group + r % p.group) * D + at;
            *reinterpret_cast<uint2*>(a.y + yo) =
                make_uint2(pack_f16(y.x * inv, y.y * inv), pack_f16(y.z * inv, y.w * inv));
          } else {
            *reinterpret_cast<float4*>(p.ws.o + (part * AT_ROWS + row) * D + at) = y;
            if (at == 0) *reinterpret_cast<float2*>(p.ws.ml + (part * AT_ROWS + row) * 2) = make_float2(top, sum);
          }
        }
      }
    }
  }
  if (!ok) {  // a copy was late: wait for what is still in flight, each wait bounded
    for (int i = 0; i < C::SLOTS; ++i) mbar_try_wait(bar_at + 8 * i, (phases >> i) & 1);
  }
}

// Joins the parts of the items that are cut: one CTA for each (first cut of an
// item, row); its warps share the parts out, the lanes the dimensions.
template <int D>
__global__ void __launch_bounds__(AT_THREADS) attn_join_kernel(const __grid_constant__ AttnDev p, int grid) {
  constexpr int V = D / 32;  // dimensions of a lane
  extern __shared__ float s_w[];  // [grid] weights of the parts
  __shared__ float s_y[AT_WARPS][D];
  __shared__ float s_red[2][AT_WARPS];
  pdl_trigger();
  pdl_wait();
  const AttnCut cut = p.ws.cut[blockIdx.x];
  const int row = blockIdx.y, r = cut.tile * AT_ROWS + row;
  if (!cut.first || r >= p.group * p.a.ncols) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = cut.c1 - cut.c0 + 1;
  // part i: the first CTA's run ends in the item (its second slot), the others' start in it
  auto slot = [&](int i) { return ((size_t)(cut.c0 + i) * 2 + (i == 0 ? 1 : 0)) * AT_ROWS + row; };
  float top = -INFINITY;
  for (int i = tid; i < n; i += AT_THREADS) {
    const float m = p.ws.ml[slot(i) * 2];
    s_w[i] = m;
    top = fmaxf(top, m);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) s_red[0][warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < AT_WARPS; ++w) top = fmaxf(top, s_red[0][w]);
  float sum = 0.f;
  for (int i = tid; i < n; i += AT_THREADS) {
    const float m = s_w[i], l = p.ws.ml[slot(i) * 2 + 1];
    const float f = m == -INFINITY ? 0.f : ex2(m - top);
    s_w[i] = f;
    sum += m == -INFINITY ? l : l * f;
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) s_red[1][warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < AT_WARPS; ++w) sum += s_red[1][w];
  float y[V];
#pragma unroll
  for (int k = 0; k < V; ++k) y[k] = 0.f;
#pragma unroll 4
  for (int i = warp; i < n; i += AT_WARPS) {
    const float f = s_w[i];
    const float* o = p.ws.o + slot(i) * D + lane * V;
    if (f != 0.f) {
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float2 x = *reinterpret_cast<const float2*>(o + k);
        y[k] = fmaf(x.x, f, y[k]);
        y[k + 1] = fmaf(x.y, f, y[k + 1]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) s_y[warp][lane * V + k] = y[k];
  __syncthreads();
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  for (int e = tid; e < D; e += AT_THREADS) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < AT_WARPS; ++w) x += s_y[w][e];
    const size_t yo = (((size_t)cut.seq * p.a.ncols + r / p.group) * p.a.n_heads + cut.head * p.group + r % p.group) * D;
    p.a.y[yo + e] = __half_as_ushort(__float2half_rn(x * inv));
  }
}

template <int TYPE, int D>
cudaError_t attn_typed(const AttnArgs& a, cudaStream_t s) {
  using C = AttnCfg<TYPE, D>;
  AttnDev p;
  p.a = a;
  p.group = a.n_heads / a.c.n_kv_heads;
  p.tiles = (p.group * a.ncols + AT_ROWS - 1) / AT_ROWS;
  p.scale = (float)((double)a.scale * 1.4426950408889634);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.ws.cut = reinterpret_cast<AttnCut*>(ws);
  ws += (size_t)C::GRID * sizeof(AttnCut);
  p.ws.ml = reinterpret_cast<float*>(ws);
  ws += (size_t)C::GRID * 2 * AT_ROWS * 8;
  p.ws.o = reinterpret_cast<float*>(ws);
  const size_t smem = C::smem(a.c.n_seq);
  cudaError_t e = prepare_kernel((const void*)attn_kernel<TYPE, D>, smem, false);
  if (e != cudaSuccess) return e;
  // both hold their SMs through shared memory, not L1
  e = launch_pdl(attn_kernel<TYPE, D>, dim3(C::GRID), dim3(AT_THREADS), smem, s, 0, LC_SMEM, p);
  if (e != cudaSuccess) return e;
  const int rows = p.group * a.ncols < AT_ROWS ? p.group * a.ncols : AT_ROWS;
  return launch_pdl(attn_join_kernel<D>, dim3(C::GRID, rows), dim3(AT_THREADS), (size_t)C::GRID * 4, s, 0, LC_SMEM,
                    p, C::GRID);
}

template <int D>
size_t ws_of() {
  constexpr int grid = AttnCfg<QG_F16, D>::GRID;
  static_assert(grid == AttnCfg<QG_Q8_0, D>::GRID, "one workspace size for both types");
  return (size_t)grid * (sizeof(AttnCut) + 2 * AT_ROWS * (8 + D * 4));
}

}  // namespace

bool attn_shape_ok(int n_seq, int n_heads, int n_kv_heads, int head_dim, int ncols) {
  return n_seq >= 1 && n_seq <= QG_KV_MAX_SEQ && n_kv_heads >= 1 && n_kv_heads <= 256 && n_heads >= n_kv_heads &&
         n_heads % n_kv_heads == 0 && n_heads / n_kv_heads <= QG_ATTN_MAX_GROUP &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && ncols >= 1 && ncols <= QG_ATTN_MAX_COLS;
}

size_t attn_ws_bytes(int, int, int, int head_dim, int) {
  return head_dim == 64 ? ws_of<64>() : head_dim == 128 ? ws_of<128>() : ws_of<256>();
}

cudaError_t attn_launch(const AttnArgs& a, cudaStream_t s) {
  if (a.c.type == QG_F16) {
    if (a.c.head_dim == 64) return attn_typed<QG_F16, 64>(a, s);
    if (a.c.head_dim == 128) return attn_typed<QG_F16, 128>(a, s);
    return attn_typed<QG_F16, 256>(a, s);
  }
  if (a.c.head_dim == 64) return attn_typed<QG_Q8_0, 64>(a, s);
  if (a.c.head_dim == 128) return attn_typed<QG_Q8_0, 128>(a, s);
  return attn_typed<QG_Q8_0, 256>(a, s);
}

cudaError_t attn_device_error(int32_t* bits) {
  const int32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_error, sizeof(*bits));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(zero));
}

}  // namespace qg
