// qg_attn.cuh -- attention of new tokens over the paged key/value cache
// (qattn_paged): the kernel templates. Each head size is a translation unit
// (qg_attn_64.cu ...); qg_attn.cu picks one.
//
// Mathematics. For a row (a query of one column and head) with scores s_j over
// the tokens it sees, y = sum_j 2^(m (s_j - z)) V_j / sum_j 2^(m (s_j - z)) for any
// z, with m = scale log2 e. A run of tokens is summed with a reference z of its
// own; two runs are joined by scaling each with 2^(m (z_run - z_both)). So the tokens
// may be cut into runs anywhere, and every byte of the cache is read once. z need
// not be the maximum: it moves up to it only when a score passes z by more than 8 / m
// (weights then stay below 2^8; times 2^7 in f16, at_lift), which is rare after the
// first tokens, so most steps have no maximum to find and nothing to rescale. z is
// a score as it came out of the products, so its own weight is 1 exactly however
// large the scores are (m z, rounded, is off by whole powers of two from scores of
// 2^24 on).
//
// Work. The rows of one kv head (all its query heads, all columns; 8 NT to a
// tile) share its keys and values. An item is a (sequence, kv head, row tile);
// its tokens come in units of 64 (four warps x a record of 16 tokens; 32 where two
// warps share a record). All items' units in a row, with a few empty places behind
// each item for what its end costs, are cut into equal runs, one for each CTA of a
// grid that fills the machine once, so a batch of ragged lengths and one very long
// sequence load every SM alike. A CTA that covers an item whole writes y; where an item is
// cut, each CTA writes its sum, reference and weight to the workspace, and a
// second kernel joins them in CTA order. The cuts, and so the last bits of the
// results, depend on lens, the window, the shape and the cache's type; and on the
// room of the page table where that decides on the form below. (Joining in the CTA that finishes last needs no
// second kernel but a first one that clears its counters, and has one CTA's loads
// to work with: 1,000 tokens of two heads of 256 took 14.3 us so, 10.7 with the
// second kernel.) Where the page table has room for little, each item is a cluster's
// of up to 16 CTAs instead, which join their sums through shared memory: one
// launch, and one length to wait for (ClusterRun).
//
// Inside a CTA each warp is on its own: it has a ring of shared-memory stages,
// fetches its records with bulk copies (one lane for each, a stage refilled as
// soon as it is consumed), and keeps z, the sum
// of weights and its accumulator in registers. The four warps meet only at the
// end of an item. Page numbers of 32 steps are loaded by the 32 lanes at once, a
// batch ahead.
//
// Products (mma m16n8k16, f16 in, f32 sums). Tokens and dimensions take the
// 16-wide side, the rows the 8-wide one: the usual 1 to 8 query heads of a kv
// head fill it, the keys and values are unpacked once for all row tiles, and the
// accumulator is a fourth of D x rows registers. Scores: A = K, B = Q; the 32
// dimensions of a block are given to the four lanes of a quad as 8 neighbouring
// ones each, the same in A and B, so a lane's operands are one load. Values: A =
// V^T, B = weights; the weights come out of the first product with tokens along
// the lanes' rows and are turned by movmatrix; V is turned by transposing
// loads, of bytes for Q8_0.
//
// Q8_0: quants are stored as u = q + 128. As the low byte of an f16, u is the
// subnormal u 2^-24, exact on the tensor cores, so K needs one byte permutation
// for two elements: sum_d Q_d q_d = sum_d Q_d u_d - 128 sum_d Q_d, the last
// term being the initial accumulator. A block's sum is then multiplied by its
// scale in f32. V's u becomes the f16 integer q (exponent trick, exact), and the
// block's scale is multiplied into the f32 weight before the weight is rounded
// to f16 (so V itself is never rounded); a power of two that follows the largest
// scale seen keeps that product in the normal range of f16.
//
// Q4_1: an element is q d + m, q from 0 to 15. Keys: sum_d Q_d k_d = d sum_d Q_d q_d + m sum_d Q_d by blocks. A masked word is two
// quants as f16 subnormals, the high nibbles 16 times as large (one row tile: a sum of their own, times 1/16; more: shifted). The
// blocks' sums of queries are made once an item, as two f16 each scaled by row, and one small product with the blocks' m starts the
// scores. Values: sum_j w_j v_j = sum_j (w_j d_j) (q_j - 8) + sum_j w_j (m_j + 8 d_j). The second part is one product a record for all
// blocks, of weights and m + 8 d, both rounded to f16; in the first w d is rounded once, as in Q8_0, and q - 8 is exact (one packed
// subtraction of subnormals; q itself would make both parts several times the answer). Off 64 bits: 5.9e-4 with q itself and a weight
// that is rounded to f16 before d meets it, 2.6e-4 with neither. The one rounding alone, of 262,143 random tokens: 3.6e-4 without
// it, 3.1e-4 with it, in the same time at heads of 128 (81 us from memory) and 256, 54 and 56 us at heads of 64.
//
// Weights are rounded to f16 because the matrix product with the values takes both
// factors in one type, and values are f16 (or integers that f16 holds): half a step,
// 2^-11 of a weight, or 2^-32 of its run's largest (Q8_0, times the largest scale: 2^-30). Their sum is of the unrounded ones. Scores,
// references, sums and the join are f32.
//
// Bound (times of calls replayed in a graph; from Python 1 to 2 us more). One tile of
// 8 rows: by memory, at 6.1 TB/s in f16 (131,071 tokens of 8 kv
// heads of 128 in 88 us; the bytes alone take 79 at the rate of a large copy), and
// nearly so in Q8_0 (64 ragged sequences, 279 MB, in 50 us, issue slots half
// used). Q4_1, one tile: by instructions, 363 a warp and record of 2,560 bytes, with 16 warps an SM and two thirds of the issue slots
// used: the records alone at 82% of the copy rate, and 11 us around them (262,143 tokens of 8 kv heads of 128, 336 MB: 70.6 us,
// 4.7 TB/s; 64 ragged sequences, 286 MB: 64.5). Two records a step 68.1 and 70.3; five CTAs an SM 73 to 79, as the registers
// do not suffice. More rows: by the latency of the instructions between two matrix
// products, with the 8 to 16 warps that the accumulators leave room for (Q8_0, 32 rows of heads
// of 256: 800 instructions a record and tile of 16 rows, issue slots 38% and
// tensor pipe 25% used, 38 us for 82 MB). One short sequence: by the chain of
// dependent loads length and page, record, and by 1,500 to 2,000 instructions a warp
// that run once (1,000 Q8_0 tokens of two heads of 256: 6.4 us; 8.4 with runs and the
// second kernel).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "qg_async.cuh"
#include "qg_attn.h"
#include "qg_common.cuh"
#include "qg_internal.h"
#include "qg_kv.cuh"
#include "qg_mma.cuh"

namespace qg {

// The device error word of this translation unit's kernels (QG_DEV_ERR_WAIT).
static __device__ int32_t g_attn_error;

namespace {

constexpr int AT_THREADS = AT_WARPS * 32;
constexpr int AT_SMS = 152;
constexpr int AT_CLUSTER = 16;  // CTAs of a cluster, at most
// Units of a CTA of a cluster, at most, of the room that the page table has for a sequence (the lengths are not known on the
// host): a table for 131,072 tokens never gets clusters, and 1,000 Q8_0 tokens of two heads of 256 take 8.3 us with it
// and 6.4 with one for 1,008 (f16, 8 heads of 128: 7.2 and 6.1). The limit: what the join saves (1.9 us of 8.4 at 1,000 tokens, two Q8_0 heads of 256; 0.7 of 7.7 at
// 2,000) is gone at four (4,000 tokens: 8.6 us against 8.5; f16, 8 heads of 128: 9.45 against 9.4).
constexpr int AT_CLUSTER_UNITS = 3;
constexpr float AT_SLACK = 8.f;  // a score may pass its row's reference by this much (log 2)
// f16: every weight is 2^7 times as large, in numerators and sums alike. The largest then lies between 2^7 and 2^15, and what
// rounding to f16 takes from small ones (up to 2^-25 below its normals) is 2^-32 of it: a first token far above 30,000 others,
// whose sum the answer is, else cost those of its warp a quarter of their weight. Q4_1 needs it where weights meet m + 8 d. (Q8_0:
// wmul below does this.)
constexpr float at_lift(int type) { return type == QG_Q8_0 ? 0.f : 7.f; }

template <int TYPE, int D, int NT>
struct AttnCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int TEAM = at_team(D, NT), TEAMS = AT_WARPS / TEAM;
  static constexpr int NB = D / 32 / TEAM;      // blocks of a warp
  static constexpr int ACC = NT * NB * 8;       // accumulator registers
  static constexpr int RECORD = kv_record_bytes(TYPE, D), STAGE = (RECORD + 127) / 128 * 128;
  // Q fragments read from shared memory each time, not kept in registers (Q4_1, one row tile: 262,143 tokens of heads of
  // 128 71.7 us with registers, 70.5 without; heads of 64, long and ragged, as long either way)
  static constexpr bool QSMEM = NT * NB > 4 || TYPE == QG_Q4_1;
  static constexpr int QPITCH = QSMEM ? 2 * D + 64 : 2 * D;  // bytes of a row of Q (+64: no bank conflicts)
  // dimensions joined at a time (32 also where 64 would leave one stage less)
  static constexpr int OD = NT > 2 || (NT == 1 && RECORD == 8192) ? 32 : 64;
  static constexpr int OPITCH = TYPE == QG_Q4_1 ? OD : OD + 4;  // floats: no bank conflicts (Q4_1: by at_swap)
  static constexpr size_t obuf = (size_t)AT_WARPS * ROWS * OPITCH * 4;
  static_assert(TEAM == 1 || obuf >= (size_t)2 * AT_WARPS * NT * 512, "a team's scores pass through the join buffer");
  static constexpr size_t stats = (size_t)2 * (2 * AT_WARPS + 2) * ROWS * 4;  // by parity: z, sums; row's z, sum
  static constexpr size_t qbuf = (size_t)ROWS * QPITCH + (QSMEM && TYPE == QG_Q8_0 ? (size_t)(D / 32) * ROWS * 8 : 0);
  // Stages of a team's ring with n CTAs on an SM (227 KB, with 1 KB of the system's and 600 bytes for up to
  // 72 sequences a CTA). Many more sequences than that may not leave room for as many CTAs, and the grid is then more than
  // one wave: 1,000 f16 tokens a sequence, 16 rows of heads of 64, take 33.0 us for 450 sequences and 42.5 for 460;
  // 8 rows of heads of 128, 46.5 for 460 and 56.8 for 480.
  static constexpr int fit(int n) {
    return (int)(((size_t)(227 * 1024) / n - 1024 - 600 - obuf - stats - qbuf - 256) / ((size_t)TEAMS * STAGE));
  }
  // CTAs per SM, by the registers a thread needs (128 threads: 128, 168 or 255 of them), fewer while a team
  // has not two stages.
  static constexpr int REGS = ACC <= 32 ? 4 : ACC <= 64 ? 3 : 2;
  static constexpr int CPS = fit(REGS) >= 2 || REGS == 2 ? REGS : fit(REGS - 1) >= 2 ? REGS - 1 : 2;
  static constexpr int GRID = AT_SMS * CPS;
  static constexpr int STAGES = fit(CPS) > 4 ? 4 : fit(CPS);
  // With one stage its halves come and go on their own: keys while values are in use, and the other way round.
  static constexpr bool SPLIT = STAGES == 1;
  static_assert(STAGES >= 1 && (TEAM == 1 || !SPLIT), "room for the records in use");
  static_assert(TYPE != QG_Q4_1 || (TEAM == 1 && !SPLIT), "4 bits: a warp on its own, whole records");
  static_assert(NB % 2 == 0, "blocks are looked through in pairs");
  static constexpr int BARS = SPLIT ? 2 : STAGES;
  static constexpr size_t ring = (size_t)TEAMS * STAGES * STAGE;
  static constexpr size_t bars = (size_t)TEAMS * BARS * 8;
  static size_t smem(int n_seq) {
    return ring + obuf + stats + qbuf + bars + (size_t)(2 * n_seq + 1) * 4;
  }
};

struct AttnWs {
  float* zl;      // [GRID][2][ROWS][2] reference and sum of weights of a part
  float* o;       // [GRID][2][ROWS][D] its weighted sum
};

struct AttnDev {
  AttnArgs a;
  AttnWs ws;
  int group;    // query heads of a kv head
  int tiles;    // row tiles of a kv head
  float mul;    // |scale| log2 e, for raw scores (Q8_0: in units of 2^24); 1 for a scale of 0
  float slack;  // AT_SLACK / mul
  __device__ __forceinline__ int head_of(int item) const { return tiles == 1 ? item : item / tiles; }
  uint32_t q_and, q_xor;  // and its sign, applied to the queries
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
__device__ __forceinline__ bool bar_ready(uint32_t bar, uint32_t parity) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(bar), "r"(parity)
      : "memory");
  return r != 0;
}
// 16 bytes to shared memory behind the thread's back; `bytes` 0: zeros instead.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// One arrival on `bar` where `mine`, with a bulk copy of `bytes` to wait for where `has` (which implies `mine`).
__device__ __forceinline__ void fetch_if(bool mine, bool has, uint32_t dst, const void* src, uint32_t bytes,
                                         uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "setp.ne.u32 p, %0, 0;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "selp.u32 n, %4, 0, q;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%5], n;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%2], [%3], %4, [%5];\n\t}" ::"r"((uint32_t)mine),
      "r"((uint32_t)has), "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
// V^T fragments of 32 dimensions x 16 tokens. f16: two 16 x 16 tiles by transposing loads of 8 x 8.
__device__ __forceinline__ void ldsm_x4_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
// Q8_0: two 16 x 16 byte matrices transposed; lane (g, t) gets bytes 4t .. 4t+3 of columns g, g + 8 of each.
__device__ __forceinline__ void ldsm_bytes_trans(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}
// Exclusive or with the place of a row's dimension in shared memory, by row: Q4_1's rows of a quad then differ in their bank.
template <int TYPE>
__device__ __forceinline__ int at_swap(int row) {
  return TYPE == QG_Q4_1 ? ((row & 2) << 1) | ((row & 4) << 2) : 0;
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 d = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&d);
}
// Q4_1: four f16 pairs of a fragment out of two words' low or high quants (bits MASK), as subnormals.
template <uint32_t MASK>
__device__ __forceinline__ void nibbles(uint32_t x, uint32_t y, uint32_t (&a)[4]) {
  a[0] = x & MASK;
  a[1] = y & MASK;
  a[2] = (x >> 8) & MASK;
  a[3] = (y >> 8) & MASK;
}
constexpr uint32_t NIB_LO = 0x000F000Fu, NIB_HI = 0x00F000F0u;
// D = A B of 8 columns of A.
__device__ __forceinline__ void mma1688(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
  const float z = 0.f;
  asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(b), "f"(z));
}
// Transpose of an 8 x 8 matrix of f16 held by a warp, two elements of a row a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

// D = A B + C, C kept.
__device__ __forceinline__ void mma16816_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                              const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

struct SeqSpan {
  int lo;    // first token that any row sees
  int hi;    // one past the last
  int unit;  // first unit
  int n;     // units (at least one, so that every item is written by some CTA)
};
template <int UNIT>
__device__ __forceinline__ SeqSpan span_of(const AttnArgs& a, int len) {
  SeqSpan s;
  const int cap = a.c.max_pages * a.c.page_size;
  s.hi = len < cap ? len : cap;
  const int64_t lo = (int64_t)len - a.ncols - a.window + 1;
  s.lo = a.window > 0 && lo > 0 ? (int)lo : 0;
  s.unit = s.lo / UNIT;
  const int end = (int)(((int64_t)s.hi + UNIT - 1) / UNIT);
  s.n = end - s.unit > 1 ? end - s.unit : 1;
  return s;
}

// Which CTA does what. Two numberings: units in order, u, and places in order, v, where every item has PAD
// places behind its units. Run c of N is the places [c places / N, (c+1) places / N), and the CTA's units are those
// among them. Both kernels of a call work this out for themselves, from lens in shared memory.
struct Unit {
  int seq, item, unit;  // item of the sequence, unit of the item
};
template <int THREADS, int UNIT, int PAD, int GRID>
struct Runs {
  int32_t* first;  // [n_seq + 1] units before a sequence (times its items)
  int32_t* len;    // [n_seq] lengths, none negative
  int n_seq, items, places, N, each, over;  // N: GRID, or less where there are fewer places

  // By all threads; `part`: shared, one int a warp. Ends with a barrier.
  __device__ __forceinline__ Runs(const AttnArgs& a, int tiles, int32_t* mem, int* part, bool report)
      : first(mem), len(mem + a.c.n_seq + 1), n_seq(a.c.n_seq), items(a.c.n_kv_heads * tiles) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (n_seq + THREADS - 1) / THREADS;
    const int b0 = tid * per, b1 = min(b0 + per, n_seq);
    const int cap = a.c.max_pages * a.c.page_size;
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      int l = a.lens[b];
      if ((l < 0 || l > cap) && report && a.err) atomicOr(a.err, QG_KV_BAD_POS);
      l = max(l, 0);
      len[b] = l;
      sum += span_of<UNIT>(a, l).n;
    }
    int run = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, off);
      if (lane >= off) run += up;
    }
    if (lane == 31) part[warp] = run;
    __syncthreads();
    int before = run - sum;
    for (int w = 0; w < warp; ++w) before += part[w];
    for (int b = b0; b < b1; ++b) {
      first[b] = before;
      before += span_of<UNIT>(a, len[b]).n;
    }
    if (b1 == n_seq && b0 < n_seq) first[n_seq] = before;
    __syncthreads();
    places = v_first(n_seq);  // below 2^31 (attn_size_ok)
    N = places < GRID ? places : GRID;
    each = places < GRID ? 1 : places / GRID;
    over = places - each * N;
  }
  __device__ __forceinline__ int units_of(int b) const { return first[b + 1] - first[b]; }
  __device__ __forceinline__ int len_of(int b) const { return len[b]; }
  __device__ __forceinline__ int v_first(int b) const { return (first[b] + b * PAD) * items; }
  __device__ __forceinline__ int v_item(int b, int item) const { return v_first(b) + item * (units_of(b) + PAD); }
  __device__ __forceinline__ int run_start(int c) const { return c < N ? c * each + c * over / GRID : places; }
  __device__ __forceinline__ int run_of(int v) const {
    int c = (int)((float)v * ((float)N / (float)places));  // right, or one off
    c = min(c, N - 1);
    if (run_start(c) > v) --c;
    if (run_start(c + 1) <= v) ++c;
    return c;
  }
  // The first units at or behind run c's first place and its last place's successor, and their numbers; by a warp.
  __device__ __forceinline__ void find(int c, Unit& x0, int& u0, Unit& x1, int& u1) const {
    const int lane = threadIdx.x & 31;
    const int v = run_start(c + (lane & 1));  // even lanes take the first, odd ones the second
    const int v0 = __shfl_sync(0xffffffffu, v, 0), v1 = __shfl_sync(0xffffffffu, v, 1);
    int before0 = 0, before1 = 0;  // sequences that start at or before the place
    for (int b0 = 0; b0 < n_seq; b0 += 32) {
      const int f = b0 + lane < n_seq ? v_first(b0 + lane) : 0x7fffffff;
      before0 += __popc(__ballot_sync(0xffffffffu, f <= v0));
      const uint32_t m = __ballot_sync(0xffffffffu, f <= v1);
      before1 += __popc(m);
      if (m != 0xffffffffu) break;
    }
    Unit x;
    x.seq = ((lane & 1) ? before1 : before0) - 1;
    int n = units_of(x.seq);
    const uint32_t rem = v - v_first(x.seq);
    x.item = rem / (uint32_t)(n + PAD);
    x.unit = rem - x.item * (n + PAD);
    if (x.unit >= n) {  // behind the item's units, or past the end
      x.unit = 0;
      if (++x.item == items) {
        x.item = 0;
        n = ++x.seq < n_seq ? units_of(x.seq) : 0;
      }
    }
    const int u = first[x.seq] * items + x.item * n + x.unit;
    x0 = {__shfl_sync(0xffffffffu, x.seq, 0), __shfl_sync(0xffffffffu, x.item, 0), __shfl_sync(0xffffffffu, x.unit, 0)};
    x1 = {__shfl_sync(0xffffffffu, x.seq, 1), __shfl_sync(0xffffffffu, x.item, 1), __shfl_sync(0xffffffffu, x.unit, 1)};
    u0 = __shfl_sync(0xffffffffu, u, 0);
    u1 = __shfl_sync(0xffffffffu, u, 1);
  }
};

// The same for a cluster of CTAs that has an item to itself. Without a window the units that the table has room for are
// dealt out, in order of rank: where a CTA starts does not depend on the length, and its pages are looked up at
// the same time. With one, the units that are seen.
template <int UNIT>
struct ClusterRun {
  int N, items, seq, item, len, n, u0, u1;
  __device__ __forceinline__ ClusterRun(const AttnArgs& a, int tiles, uint32_t rank, uint32_t ctas)
      : N(1 << 30), items(a.c.n_kv_heads * tiles) {
    const uint32_t i = blockIdx.x / ctas;
    seq = i / (uint32_t)items;
    item = i - seq * items;
    const int cap = a.c.max_pages * a.c.page_size;
    len = a.lens[seq];
    uint32_t all = (uint32_t)(cap + UNIT - 1) / UNIT;  // (few: the host has looked)
    if (a.window > 0) all = span_of<UNIT>(a, max(len, 0)).n;
    u0 = all * rank / ctas;
    u1 = all * (rank + 1) / ctas;
  }
  __device__ __forceinline__ void arrived(const AttnArgs& a, bool report) {
    if (report && (len < 0 || len > a.c.max_pages * a.c.page_size) && item == 0 && a.err) atomicOr(a.err, QG_KV_BAD_POS);
    len = max(len, 0);
    n = span_of<UNIT>(a, len).n;
    u1 = max(min(u1, n), u0);
  }
  __device__ __forceinline__ int units_of(int) const { return n; }
  __device__ __forceinline__ int len_of(int) const { return len; }
};
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t at_rank(const void* mine, uint32_t rank) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(smem_u32(mine)), "r"(rank));
  return d;
}
__device__ __forceinline__ float ld_rank(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_rank2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

// CLUSTER: short contexts; each item is a cluster's, whose CTAs read one another's sums from shared memory and join them.
template <int TYPE, int D, int NT, bool CLUSTER>
__global__ void __launch_bounds__(AT_THREADS, AttnCfg<TYPE, D, NT>::CPS)
    attn_kernel(const __grid_constant__ AttnDev p) {
  using C = AttnCfg<TYPE, D, NT>;
  constexpr int NB = C::NB, ROWS = C::ROWS, TEAM = C::TEAM, UNIT = at_unit(D, NT);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* const s_ring = smem;
  float* const s_o = reinterpret_cast<float*>(smem + C::ring);
  float* const s_stat = reinterpret_cast<float*>(smem + C::ring + C::obuf);
  uint8_t* const s_q = smem + C::ring + C::obuf + C::stats;
  uint64_t* const s_bar = reinterpret_cast<uint64_t*>(s_q + C::qbuf);
  int32_t* const s_runs = reinterpret_cast<int32_t*>(s_bar + C::TEAMS * C::BARS);
  __shared__ int s_part[AT_WARPS];

  __shared__ uint32_t s_k64[32];
  const AttnArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int team = warp / TEAM, share = warp % TEAM;  // the warp has blocks share * NB ... of the team's records
  if (tid < 32) s_k64[tid] = 0x64646464u;
  if (tid < C::TEAMS * C::BARS) {
    mbar_init(s_bar + tid, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();  // (not before: the join reads lens at once)

  const int cta = blockIdx.x;
  uint32_t rank = 0, ctas = 1;
  if constexpr (CLUSTER) {
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
  }
  auto runs = [&] {
    if constexpr (CLUSTER)
      return ClusterRun<UNIT>(a, p.tiles, rank, ctas);
    else
      return Runs<AT_THREADS, UNIT, at_pad(TYPE, NT), C::GRID>(a, p.tiles, s_runs, s_part, cta == 0);
  }();
  if (cta >= runs.N) return;
  const int items = runs.items;
  Unit at, end_at;  // the unit in hand
  int u0, u1;
  if constexpr (CLUSTER) {
    at = {runs.seq, runs.item, u0 = runs.u0};
  } else {
    runs.find(cta, at, u0, end_at, u1);
    if (u1 == u0) return;
  }

  // Queries of an item into shared memory, [row][D] f16, asynchronously: the first before any keys are asked for, the
  // others as soon as the buffer is free (in the middle of the stream a load takes microseconds).
  const int rows = p.group * a.ncols;
  auto stage_q = [&](const Unit& x) {
    const int head = p.head_of(x.item), r0 = (x.item - head * p.tiles) * ROWS;
    for (int i = tid; i < ROWS * (D / 8); i += AT_THREADS) {
      const int row = i / (D / 8), c = i % (D / 8), r = r0 + row;
      const uint16_t* src = a.q;
      if (r < rows)
        src += (((size_t)x.seq * a.ncols + r / p.group) * a.n_heads + head * p.group + r % p.group) * D + 8 * c;
      copy16_async(smem_u32(s_q) + row * C::QPITCH + 16 * c, src, r < rows ? 16 : 0);
    }
  };
  const int gpp = a.c.page_size / KV_GROUP, gpp_log = __ffs(gpp) - 1;  // records of a page and head
  int near_page = -1;  // CLUSTER without a window: the page of lane's step, whether or not there is one
  if constexpr (CLUSTER) {
    const int j = ((u0 + lane) * C::TEAMS + team) >> gpp_log;
    if (a.window <= 0 && j < a.c.max_pages) near_page = a.c.page_table[(size_t)at.seq * a.c.max_pages + j];
    stage_q(at);
    __syncthreads();  // the barriers are ready (Runs has a barrier of its own)
    runs.arrived(a, rank == 0 && tid == 0);
    u1 = runs.u1;
  }
  const int steps = u1 - u0;
  const Unit whose = at;
  // The high bytes of f16 1024 + u. Read from shared memory it stays in a register of each lane; as a constant it is
  // moved from a uniform register at every use (eight moves a block).
  const uint32_t k64 = s_k64[lane];

  // ------------------------------------------------------------ the ring
  uint8_t* const ring = s_ring + (size_t)team * C::STAGES * C::STAGE;
  const uint32_t ring_at = smem_u32(ring), bar_at = smem_u32(s_bar + team * C::BARS);
  // In a half record: where this warp's blocks are, and (Q8_0) from there their scales.
  constexpr int BLOCKS = NB * 32 * KV_GROUP * (TYPE == QG_F16 ? 4 : TYPE == QG_Q8_0 ? 2 : 1) / 2;
  const int own = share * BLOCKS, scales = TEAM * BLOCKS - share * (BLOCKS - NB * 32);
  // Page numbers: lane i looks up step base + i. Raw until the batch is entered,
  // so that the load has the whole batch before to arrive.
  int nx_page = -1, nx_off = 0;
  bool nx_in = false;
  Unit ahead_at = at;  // of the batch's first step
  auto look_up = [&](int base) {
    nx_in = false;
    nx_page = -1;
    Unit x = ahead_at;
    x.unit += lane;
    int n = runs.units_of(x.seq);
    const int most = steps - base;  // steps from here on
    if (lane < most) {
      while (x.unit >= n) {
        x.unit -= n;
        if (++x.item == items) {
          x.item = 0;
          n = runs.units_of(++x.seq);
        }
      }
      const SeqSpan sp = span_of<UNIT>(a, runs.len_of(x.seq));
      const int grp = (sp.unit + x.unit) * C::TEAMS + team;  // group of 16 tokens, hence the comparisons in groups
      if (grp < (sp.hi + KV_GROUP - 1) / KV_GROUP && grp >= sp.lo / KV_GROUP) {
        nx_in = true;
        nx_page = CLUSTER && a.window <= 0 ? near_page : a.c.page_table[(size_t)x.seq * a.c.max_pages + (grp >> gpp_log)];
        nx_off = p.head_of(x.item) * gpp + (grp & (gpp - 1));
      }
    }
    if (most > 32) {  // on to the next batch: one behind lane 31's
      ahead_at.seq = __shfl_sync(0xffffffffu, x.seq, 31);
      ahead_at.item = __shfl_sync(0xffffffffu, x.item, 31);
      ahead_at.unit = __shfl_sync(0xffffffffu, x.unit, 31) + 1;
      if (ahead_at.unit == runs.units_of(ahead_at.seq)) {
        ahead_at.unit = 0;
        if (++ahead_at.item == items) {
          ahead_at.item = 0;
          ++ahead_at.seq;
        }
      }
    }
  };
  const uint8_t* my_rec = nullptr;         // this lane's record of the batch in issue
  uint32_t valid_even = 0, valid_odd = 0;  // steps of the even / odd batches that have a record
  auto enter = [&](int step) {             // step: a multiple of 32
    my_rec = nullptr;
    if (nx_in) {
      if (nx_page >= 0 && nx_page < a.c.n_pages)
        my_rec = static_cast<const uint8_t*>(a.c.pool) +
                 ((size_t)nx_page * a.c.n_kv_heads * gpp + nx_off) * kv_record_bytes(TYPE, D);
      else if (a.err)
        atomicOr(a.err, QG_KV_BAD_PAGE);
    }
    const uint32_t v = __ballot_sync(0xffffffffu, my_rec != nullptr);
    if (step & 32) valid_odd = v; else valid_even = v;
  };
  // Fetch the record of `step` into a stage: the lane that looked it up does, of the team's first warp. A step without a
  // record completes the barrier at once.
  bool ok = true;  // false once a wait gave up: no more copies, no more waits
  constexpr int HALF = kv_half_bytes(TYPE, D);
  auto fetch = [&](int step, int to) {  // SPLIT: `to` is the half
    const bool mine = lane == (step & 31) && step < steps && ok && share == 0;
    if constexpr (C::SPLIT)
      fetch_if(mine, mine && my_rec, ring_at + to * HALF, my_rec + to * HALF, HALF, bar_at + 8 * to);
    else
      fetch_if(mine, mine && my_rec, ring_at + to * C::STAGE, my_rec, C::RECORD, bar_at + 8 * to);
  };
  __syncwarp();
  look_up(0);
  if constexpr (!CLUSTER) stage_q(at);
  enter(0);
#pragma unroll
  for (int i = 0; i < C::BARS; ++i) fetch(C::SPLIT ? 0 : i, i);
  if constexpr (!CLUSTER) look_up(32);
  int stage = 0;        // the stage in use
  uint32_t parity = 0;  // of its barriers
  auto arrived = [&](uint32_t bar) {
    if (!bar_ready(bar, parity) && ok) ok = mbar_wait_slow(bar, parity, &g_attn_error);
  };
  auto team_barrier = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TEAM) : "memory"); };
  // A stage's reads are over: every lane orders its own before the refill. A warp on its own then refills the stage at
  // once; of a team, the first warp does after the next step's barrier, which both pass behind their reads.
  auto reads_done = [&]() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
  };

  // Which token of the record position i of the 16-wide side is. f16, Q4_1: token i. Q8_0: i/2 (i even) or
  // 4 + (i/2 + 2) mod 4 (i odd), and 8 more for i >= 8: the rows of 32 bytes that the lanes of a shared-memory phase
  // read then differ modulo 4 (no bank conflict), and a lane's two tokens, 8 apart, have their scales in one word.
  auto token_of = [](int i) {
    return TYPE != QG_Q8_0 ? i : (i & 8) + ((i & 1) ? 4 + ((((i & 7) >> 1) + 2) & 3) : (i & 7) >> 1);
  };
  const int tok_a = token_of(g);  // this lane's tokens as rows of the scores: tok_a and tok_a + 8
  const uint32_t scale_at = (tok_a & 3) * 8, scale_sel = (tok_a & 4) ? 0x7632u : 0x5410u;
  // this lane's row address for the transposing loads of V
  uint32_t v_at;
  if constexpr (TYPE == QG_F16) {
    v_at = ((lane & 7) + ((lane >> 4) & 1) * 8) * 64 + ((lane >> 3) & 1) * 16;
  } else if constexpr (TYPE == QG_Q4_1) {
    // as below, but bytes 0 and 2 are tokens 2t, 2t+1 and bytes 1 and 3 tokens 2t+8, 2t+9, as nibbles() pairs them; the two
    // matrices are two blocks
    const int j = lane & 15;
    v_at = (2 * (j >> 2) + ((j >> 1) & 1) + 8 * (j & 1)) * 16 + (lane >> 4) * 256;
  } else {
    // row j of the byte matrix goes to byte j mod 4 of lane j / 4: positions 2t, 2t+1, 2t+8, 2t+9
    const int j = lane & 15, i = 2 * (j >> 2) + (j & 1) + 4 * (j & 2);
    v_at = token_of(i) * 32 + (lane >> 4) * 16;
  }

  // CLUSTER: place of (row, dimension) among a warp's sums; the exclusive or keeps a quad's rows on different banks
  auto in_sums = [](int row, int dim) { return row * D + (dim ^ (TYPE == QG_Q4_1 ? at_swap<TYPE>(row) : (row & 6) << 2)); };
  // of a block: the dimension of accumulator 4 blk + e of this lane
  auto dim_of = [&](int e) {
    return TYPE == QG_Q4_1 ? 16 * (e & 1) + 4 * (e >> 1) + 8 * (g >> 2) + ((g & 1) << 1) + ((g >> 1) & 1) : 8 * e + g;
  };

  // --------------------------------------------------------------- items
  int turn = 0;  // of the statistics' two buffers
  int step = 0;
  uint32_t valid = 0;
  while (step < steps) {
    const int b = at.seq, hr = at.item, nu = runs.units_of(b);
    const int todo = nu - at.unit < steps - step ? nu - at.unit : steps - step;  // units of this run in the item
    const bool starts = at.unit == 0, whole = !CLUSTER && starts && todo == nu;
    const int head = p.head_of(hr), tile = hr - head * p.tiles;
    const int len = runs.len_of(b);
    const SeqSpan sp = span_of<UNIT>(a, len);
    // (the last unit's end may pass 2^31, but not the records that are looked at)
    int tok = (int)(((uint32_t)(sp.unit + at.unit) * C::TEAMS + team) * KV_GROUP - UNIT);
    at.unit = 0;  // (the next item's first, if there is one)
    if (++at.item == items) {
      at.item = 0;
      ++at.seq;
    }

    // what row r of the tile sees: tokens lo < j <= hi
    auto row_sees = [&](int i, int& lo, int& hi) {
      const int r = tile * ROWS + i;
      const int64_t pos = (int64_t)len - a.ncols + r / p.group;
      hi = r < rows ? (int)(pos < sp.hi - 1 ? pos : sp.hi - 1) : -1;
      lo = a.window > 0 && pos - a.window > -1 ? (int)(pos - a.window) : -1;
    };
    // tokens that all rows see: no mask needed from `lo_all` up to `hi_all`
    const int hi_all = (int)min((int64_t)sp.hi - 1, (int64_t)len - a.ncols);
    const int lo_all = a.window > 0 ? (int)max((int64_t)0, (int64_t)len - a.window) : 0;

    // Q: the B fragments of a block and row tile, dimensions 8t .. 8t+7 of row g; and, for
    // Q8_0, -128 2^-24 sum of the block's queries of rows 2t and 2t + 1.
    uint32_t qf[C::QSMEM ? 1 : NB][C::QSMEM ? 1 : NT][4];
    float qc[C::QSMEM || TYPE != QG_Q8_0 ? 1 : NB][C::QSMEM || TYPE != QG_Q8_0 ? 1 : NT][4];  // (each twice, as the mma's C)
    // Q4_1: the sums of the blocks' queries as two f16 each (what the first one's rounding leaves is the second), times a power
    // of two by row, as the B fragment of the product with the blocks' m; and that power's inverse of rows 2t, 2t + 1.
    uint32_t qm[NT][D == 256 ? 2 : 1];
    float2 qback[NT];
    const uint32_t q_at = smem_u32(s_q) + g * C::QPITCH + 16 * t + share * (NB * 64);  // this lane's, of the warp's first block
    auto load_q = [&](int blk, int nt, uint32_t (&q)[4]) {
      lds128(q_at + nt * 8 * C::QPITCH + blk * 64, q[0], q[1], q[2], q[3]);
    };
    auto sum_of = [&](const uint32_t (&q)[4]) {  // of row g
      float s = ((lo_f32(q[0]) + hi_f32(q[0])) + (lo_f32(q[1]) + hi_f32(q[1]))) +
                ((lo_f32(q[2]) + hi_f32(q[2])) + (lo_f32(q[3]) + hi_f32(q[3])));
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      return s;
    };
    auto sum_q = [&](const uint32_t (&q)[4]) { return sum_of(q) * -7.62939453125e-06f; };  // -128 * 2^-24
    float* const s_qsum = reinterpret_cast<float*>(s_q + ROWS * C::QPITCH);  // [block][tile][t][4]
    copies_done();
    if (p.q_and != 0xffffffffu || p.q_xor) {  // a scale that is not positive: each thread on what it copied
      for (int i = tid; i < ROWS * (D / 8); i += AT_THREADS) {
        uint4* const x = reinterpret_cast<uint4*>(s_q + i / (D / 8) * C::QPITCH + 16 * (i % (D / 8)));
        *x = make_uint4((x->x & p.q_and) ^ p.q_xor, (x->y & p.q_and) ^ p.q_xor, (x->z & p.q_and) ^ p.q_xor,
                        (x->w & p.q_and) ^ p.q_xor);
      }
    }
    __syncthreads();
    if constexpr (C::QSMEM) {
      if constexpr (TYPE == QG_Q8_0) {
        for (int i = team; i < NB * NT; i += C::TEAMS) {
          uint32_t q[4];
          load_q(i / NT, i % NT, q);
          const float s = sum_q(q);
          if (t < 2) s_qsum[(share * NB * NT + i) * 16 + (g >> 1) * 4 + 2 * t + (g & 1)] = s;
        }
        __syncthreads();
      }
    } else {
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          load_q(blk, nt, qf[blk][nt]);
          if constexpr (TYPE == QG_Q8_0) {
            const float s = sum_q(qf[blk][nt]);
            qc[blk][nt][0] = qc[blk][nt][2] = __shfl_sync(0xffffffffu, s, 8 * t);
            qc[blk][nt][1] = qc[blk][nt][3] = __shfl_sync(0xffffffffu, s, 8 * t + 4);
          }
        }
    }
    if constexpr (TYPE == QG_Q4_1) {
      // lane t has blocks 2 pair, 2 pair + 1, and of them the first f16 (which = 0), the second (1) or neither
      const int pair = t % (NB / 2), which = NB == 8 ? 0 : t / (NB / 2);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float s0 = 0.f, s1 = 0.f, most = 0.f;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          float s;
          if constexpr (C::QSMEM) {
            uint32_t q[4];
            load_q(blk, nt, q);
            s = sum_of(q);
          } else {
            s = sum_of(qf[blk][nt]);
          }
          most = fmaxf(most, fabsf(s));
          if (blk == 2 * pair) s0 = s;
          if (blk == 2 * pair + 1) s1 = s;
        }
        // most, times 2^-up, lies between 2^13 and 2^14 (most is 0 or between 2^-24 and 2^21; infinite or NaN queries leave NaN)
        const int up = most > 0.f ? min(((__float_as_int(most) >> 23) & 0xff) - 127, 40) - 13 : 0;
        const float to = __int_as_float((127 - up) << 23);
        s0 *= to;
        s1 *= to;
        const uint32_t hi = pack_f16(s0, s1), lo = pack_f16(s0 - lo_f32(hi), s1 - hi_f32(hi));
        if constexpr (D == 256) {
          qm[nt][0] = hi;
          qm[nt][1] = lo;
        } else {
          qm[nt][0] = which == 0 ? hi : which == 1 ? lo : 0u;
        }
        const float back = __int_as_float((127 + up - 24) << 23);  // (scores are in units of 2^24)
        qback[nt] = make_float2(__shfl_sync(0xffffffffu, back, 8 * t), __shfl_sync(0xffffffffu, back, 8 * t + 4));
      }
    }
    if (!C::QSMEM && step + todo < steps) {
      __syncthreads();  // the buffer is in all warps' registers
      stage_q(at);
    }

    // o[blk][nt][i][c]: dimension 32 blk + 16 i + 8 (c/2) + g, row 8 nt + 2t + c%2
    float o[NB][NT][2][4];
#pragma unroll
    for (int i = 0; i < NB * NT * 8; ++i) (&o[0][0][0][0])[i] = 0.f;
    // of rows 2t, 2t + 1: the reference z, a raw score (0 while there is none), and the score above which it
    // moves (-inf while there is none); the sum of this lane's tokens' weights
    const float2 mul = make_float2(p.mul, p.mul);
    float z[NT][2], limit[NT][2], l[NT][2];

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        limit[nt][c] = -INFINITY;
        z[nt][c] = l[nt][c] = 0.f;
      }
    auto ref = [&](int nt, int c) { return limit[nt][c] == -INFINITY ? -INFINITY : z[nt][c]; };
    // Q8_0: weights are multiplied by their scale and by wmul = 2^(7-e), so that they stay below 2^15
    // for scales up to wmax = 2^e; larger scales move e up. wback = 1 / wmul. Q4_1: the same with
    // 2^-e, weights being 2^7 times as large from the start, and |d|, which another writer's blocks may have of either sign.
    float wmul = 1.f, wmax = 0.f, wback = 1.f;
    // Q4_1: om[nt][c] of block g (c < 2): sum of weights times m + 8 d, of row 8 nt + 2t + c
    float om[TYPE == QG_Q4_1 ? NT : 1][4];
#pragma unroll
    for (int nt = 0; nt < (TYPE == QG_Q4_1 ? NT : 1); ++nt) om[nt][0] = om[nt][1] = om[nt][2] = om[nt][3] = 0.f;

    const int begin = step;
    for (const int end = step + todo; step < end; ++step) {
      tok += UNIT;
      if ((step & 31) == 0) valid = (step & 32) ? valid_odd : valid_even;
      const uint32_t kb = ring_at + stage * C::STAGE + own, vb = kb + HALF;
      // nothing to do where no token of the record is seen, or its page is bad
      const bool live = (valid >> (step & 31)) & 1;
      const bool masked = tok + KV_GROUP - 1 > hi_all || tok < lo_all;
      // SPLIT: the half just read; otherwise this stage, or a team's stage of the step before
      auto refill = [&](int half) {
        const int ahead = step + C::STAGES - (TEAM > 1);
        const bool new_batch = (ahead & 31) == 0 && ahead < steps;
        if (TEAM > 1 && step == 0) return;
        if (new_batch && half == 0) enter(ahead);
        fetch(ahead, C::SPLIT ? half : TEAM == 1 ? stage : stage ? stage - 1 : C::STAGES - 1);
        if (new_batch && half == (C::SPLIT ? 1 : 0)) look_up(ahead + 32);
      };
      auto next = [&]() {
        if (++stage == C::STAGES) {
          stage = 0;
          parity ^= 1;
        }
      };
      arrived(bar_at + stage * 8);
      if (__builtin_expect(!live, 0)) {
        __syncwarp();  // no lane re-arms a barrier that another still waits on
        if constexpr (TEAM > 1) team_barrier();  // (both warps pass as many, whatever they made of the page table)
        refill(0);
        if constexpr (C::SPLIT) {
          arrived(bar_at + 8);
          __syncwarp();
          refill(1);
        }
        next();
        continue;
      }

      // ---- scores: s[nt][c] of token tok_a + 8 (c/2), row 8 nt + 2t + c%2
      float s[NT][4];
      uint32_t kd[TYPE == QG_Q4_1 ? 2 : 1][TYPE == QG_Q4_1 ? NB / 2 : 1];  // Q4_1: the d of tokens tok_a, tok_a + 8
      if constexpr (TYPE == QG_Q4_1) {
        const uint32_t d_at = kb + scales + tok_a * (2 * NB), m_at = d_at + D + 4 * (t % (NB / 2));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (NB == 2) kd[i][0] = lds32(d_at + i * 8 * 2 * NB);
          if constexpr (NB == 4) lds64(d_at + i * 8 * 2 * NB, kd[i][0], kd[i][1]);
          if constexpr (NB == 8) lds128(d_at + i * 8 * 2 * NB, kd[i][0], kd[i][1], kd[i][2], kd[i][3]);
        }
        const uint32_t m0 = lds32(m_at), m1 = lds32(m_at + 8 * 2 * NB);
        const uint32_t am[4] = {m0, m1, m0, m1};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float part[4];
          if constexpr (NB == 8)
            mma16816(part, am, qm[nt][0], qm[nt][1]);
          else
            mma1688(part, m0, m1, qm[nt][0]);
          const float2 lo = mul2(make_float2(part[0], part[1]), qback[nt]), hi = mul2(make_float2(part[2], part[3]), qback[nt]);
          s[nt][0] = lo.x;
          s[nt][1] = lo.y;
          s[nt][2] = hi.x;
          s[nt][3] = hi.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) s[i >> 2][i & 3] = 0.f;
      }
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        uint32_t a0[4], a1[4];
        float e0 = 0.f, e1 = 0.f;
        if constexpr (TYPE == QG_Q4_1) {
          const uint32_t at = kb + blk * 256 + tok_a * 16 + t * 4;
          const uint32_t x = lds32(at), y = lds32(at + 128);
          nibbles<NIB_LO>(x, y, a0);
          if constexpr (NT == 1)
            nibbles<NIB_HI>(x, y, a1);  // 16 times their values
          else
            nibbles<NIB_LO>(x >> 4, y >> 4, a1);
          e0 = blk & 1 ? hi_f32(kd[0][blk / 2]) : lo_f32(kd[0][blk / 2]);
          e1 = blk & 1 ? hi_f32(kd[1][blk / 2]) : lo_f32(kd[1][blk / 2]);
        } else if constexpr (TYPE == QG_F16) {
          const uint32_t at = kb + blk * 1024 + tok_a * 64 + t * 16;
          lds128(at, a0[0], a0[2], a1[0], a1[2]);
          lds128(at + 512, a0[1], a0[3], a1[1], a1[3]);
        } else {
          const uint32_t at = kb + blk * 512 + tok_a * 32 + t * 8;
          uint32_t x, y, d0, d1;
          lds64(at, x, y);
          a0[0] = __byte_perm(x, 0, 0x4140);
          a0[2] = __byte_perm(x, 0, 0x4342);
          a1[0] = __byte_perm(y, 0, 0x4140);
          a1[2] = __byte_perm(y, 0, 0x4342);
          lds64(at + 256, x, y);
          a0[1] = __byte_perm(x, 0, 0x4140);
          a0[3] = __byte_perm(x, 0, 0x4342);
          a1[1] = __byte_perm(y, 0, 0x4140);
          a1[3] = __byte_perm(y, 0, 0x4342);
          lds64(kb + scales + blk * 32 + scale_at, d0, d1);
          const uint32_t d = __byte_perm(d0, d1, scale_sel);
          e0 = lo_f32(d);
          e1 = hi_f32(d);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t q[4];
          if constexpr (C::QSMEM) {
            load_q(blk, nt, q);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = qf[blk][nt][i];
          }
          if constexpr (TYPE == QG_F16) {
            mma16816_acc(s[nt], a0, q[0], q[1]);
            mma16816_acc(s[nt], a1, q[2], q[3]);
          } else {
            float part[4], c[4];
            if constexpr (TYPE == QG_Q4_1) {
              mma16816(part, a0, q[0], q[1]);
            } else if constexpr (C::QSMEM) {
              const float4 x = *reinterpret_cast<const float4*>(s_qsum + ((share * NB + blk) * NT + nt) * 16 + 4 * t);
              c[0] = x.x; c[1] = x.y; c[2] = x.z; c[3] = x.w;
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) c[i] = qc[blk][nt][i];
            }
            if constexpr (TYPE == QG_Q8_0) mma16816_from(part, a0, q[0], q[1], c);
            if constexpr (TYPE == QG_Q4_1 && NT == 1) {  // (two more instructions a row tile, three less a block than the shift)
              float high[4];
              mma16816(high, a1, q[2], q[3]);
              const float2 k = make_float2(0.0625f, 0.0625f);
              const float2 lo = fma2(make_float2(high[0], high[1]), k, make_float2(part[0], part[1]));
              const float2 hi = fma2(make_float2(high[2], high[3]), k, make_float2(part[2], part[3]));
              part[0] = lo.x;
              part[1] = lo.y;
              part[2] = hi.x;
              part[3] = hi.y;
            } else {
              mma16816_acc(part, a1, q[2], q[3]);
            }
            const float2 lo = fma2(make_float2(part[0], part[1]), make_float2(e0, e0), make_float2(s[nt][0], s[nt][1]));
            const float2 hi = fma2(make_float2(part[2], part[3]), make_float2(e1, e1), make_float2(s[nt][2], s[nt][3]));
            s[nt][0] = lo.x;
            s[nt][1] = lo.y;
            s[nt][2] = hi.x;
            s[nt][3] = hi.y;
          }
        }
      }
      if constexpr (TEAM > 1) {
        // the other half of every sum; two buffers, so one barrier of the team a step
        float4* const x = reinterpret_cast<float4*>(s_o) + ((step & 1) * AT_WARPS + warp) * (NT * 32) + lane;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) x[nt * 32] = make_float4(s[nt][0], s[nt][1], s[nt][2], s[nt][3]);
        team_barrier();
        const float4* const y = x + (share ? -1 : 1) * (NT * 32);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float4 v = y[nt * 32];
          s[nt][0] += v.x;
          s[nt][1] += v.y;
          s[nt][2] += v.z;
          s[nt][3] += v.w;
        }
        refill(0);
      }
      if constexpr (C::SPLIT) {
        reads_done();
        refill(0);
      }

      // ---- weights
      if (__builtin_expect(masked, 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            int lo, hi;
            row_sees(nt * 8 + 2 * t + c, lo, hi);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int at = tok + tok_a + 8 * i;
              if (at > hi || at <= lo) s[nt][2 * i + c] = -INFINITY;
            }
          }
      }
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) up |= fmaxf(s[nt][c], s[nt][2 + c]) > limit[nt][c];
      if (__builtin_expect(__any_sync(0xffffffffu, up), 0)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float f[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(s[nt][c], s[nt][2 + c]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float was = ref(nt, c);
            f[c] = 1.f;
            if (x > was) {
              f[c] = ex2((was - x) * p.mul);
              z[nt][c] = x;
              limit[nt][c] = __fadd_rd(x, p.slack);  // (not a step above: a step may be many times the slack)
              l[nt][c] *= f[c];
            }
          }
          if constexpr (TYPE == QG_Q4_1) {
            om[nt][0] *= f[0];
            om[nt][1] *= f[1];
          }
          if (CLUSTER && step == begin) continue;  // nothing is there yet (with more steps, the test costs more than it saves)
#pragma unroll
          for (int blk = 0; blk < NB; ++blk)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              o[blk][nt][i][0] *= f[0];
              o[blk][nt][i][1] *= f[1];
              o[blk][nt][i][2] *= f[0];
              o[blk][nt][i][3] *= f[1];
            }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 d = sub2(make_float2(s[nt][i], s[nt][i + 1]), make_float2(z[nt][0], z[nt][1]));
          const float2 x = TYPE != QG_Q8_0 ? fma2(d, mul, make_float2(at_lift(TYPE), at_lift(TYPE))) : mul2(d, mul);
          s[nt][i] = ex2(x.x);
          s[nt][i + 1] = ex2(x.y);
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) l[nt][c] += s[nt][c] + s[nt][2 + c];

      // ---- weights times values
      if constexpr (C::SPLIT) arrived(bar_at + 8);
      uint8_t* const vp = ring + stage * C::STAGE + HALF + own;
      if constexpr (TYPE == QG_F16) {
        if (__builtin_expect(masked, 0)) {
          // Zero weights do not silence a NaN or an infinity in the product. So the rows of tokens that no
          // query row sees are cleared, and values that are not finite are taken out here and added, to the
          // rows that see them.
          uint32_t odd = 0;  // tokens with such values
          for (int i = lane; i < NB * KV_GROUP * 4; i += 32) {
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
            __half* const row = reinterpret_cast<__half*>(vp) + k * 32;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                int lo, hi;
                row_sees(nt * 8 + 2 * t + c, lo, hi);
                const bool sees = tok + k <= hi && tok + k > lo;
#pragma unroll
                for (int blk = 0; blk < NB; ++blk)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float x = __half2float(row[blk * 512 + 8 * i + g]);
                    if (sees && !(fabsf(x) <= 65504.f)) o[blk][nt][i >> 1][2 * (i & 1) + c] += x;
                  }
              }
            __syncwarp();
            for (int e = lane; e < NB * 32; e += 32) {
              __half* const x = row + (e >> 5) * 512 + (e & 31);
              if (!(fabsf(__half2float(*x)) <= 65504.f)) *x = __ushort_as_half(0);
            }
          }
          __syncwarp();
        }
        uint32_t w0[NT], w1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          w0[nt] = transpose8(pack_f16(s[nt][0], s[nt][1]));
          w1[nt] = transpose8(pack_f16(s[nt][2], s[nt][3]));
        }
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          uint32_t v0[4], v1[4];
          ldsm_x4_trans(vb + blk * 1024 + v_at, v0);
          ldsm_x4_trans(vb + blk * 1024 + 32 + v_at, v1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816_acc(o[blk][nt][0], v0, w0[nt], w1[nt]);
            mma16816_acc(o[blk][nt][1], v1, w0[nt], w1[nt]);
          }
        }
      } else if constexpr (TYPE == QG_Q4_1) {
        if (__builtin_expect(masked, 0)) {
          // As for Q8_0, for d and m alike: those of tokens that no row sees are cleared, and one that is not finite, of a token
          // that some rows do not see, is taken out and given to the rows that see it.
          uint16_t* sc = reinterpret_cast<uint16_t*>(vp + scales);
#pragma unroll
          for (int two = 0; two < 2 * NB; two += 2) {  // the 16 of each by a half of the warp; from NB on they are m
            uint16_t& x = sc[two * KV_GROUP + lane];
            const uint16_t was = x;
            const int tk = tok + kv_value_token(lane & 15);
            const bool seen = tk < sp.hi && tk >= sp.lo;
            const bool bad = seen && (was & 0x7C00) == 0x7C00;
            if (!seen || bad) x = 0;
            const uint32_t both = __ballot_sync(0xffffffffu, bad);
            if (__builtin_expect(both == 0, 1)) continue;
            const bool is_m = two >= NB;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int blk = (two + h) % NB;
              uint32_t odd = h == 0 ? both & 0xffffu : both >> 16;
              while (odd) {
                const int j = __ffs(odd) - 1, tj = tok + kv_value_token(j);
                odd &= odd - 1;
                const float its = __half2float(__ushort_as_half((uint16_t)__shfl_sync(0xffffffffu, (uint32_t)was, 16 * h + j)));
                const float what = is_m ? its : __int_as_float(0x7fffffff);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    int lo, hi;
                    row_sees(nt * 8 + 2 * t + c, lo, hi);
                    const float add = tj <= hi && tj > lo ? what : 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[blk][nt][e >> 1][2 * (e & 1) + c] += add;
                  }
              }
            }
          }
          __syncwarp();
        }
        uint32_t w0[NT], w1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          w0[nt] = transpose8(pack_f16(s[nt][0], s[nt][1]));
          w1[nt] = transpose8(pack_f16(s[nt][2], s[nt][3]));
        }
        {  // weights times m + 8 d: the blocks on the wide side
          uint32_t am[4] = {0u, 0u, 0u, 0u}, d0, d1;
          lds64(vb + scales + (g & (NB - 1)) * 32 + t * 8, d0, d1);
          lds64(vb + scales + D + (g & (NB - 1)) * 32 + t * 8, am[0], am[2]);
          am[0] = hfma2_u(d0, 0x48004800u, am[0]);
          am[2] = hfma2_u(d1, 0x48004800u, am[2]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816_acc(om[nt], am, w0[nt], w1[nt]);
        }
        uint32_t d[NB];  // of tokens g, g + 8
        __half2 big = __float2half2_rn(0.f);
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          uint32_t d0, d1;
          lds64(vb + scales + blk * 32 + (g >> 1) * 8, d0, d1);
          d[blk] = __byte_perm(d0, d1, g & 1 ? 0x7632u : 0x5410u);
          big = __hmax2(big, __habs2(*reinterpret_cast<__half2*>(&d[blk])));
        }
        float dmax = fmaxf(__low2float(big), __high2float(big));
        if (__builtin_expect(__any_sync(0xffffffffu, dmax > wmax), 0)) {
          dmax = wmax;  // again without infinities, which would cost the others their bits
#pragma unroll
          for (int blk = 0; blk < NB; ++blk) {
            const float x = fabsf(lo_f32(d[blk])), y = fabsf(hi_f32(d[blk]));
            if (x <= 65504.f) dmax = fmaxf(dmax, x);
            if (y <= 65504.f) dmax = fmaxf(dmax, y);
          }
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 4));
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 8));
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 16));
          if (dmax > wmax) {  // as below
            const int e = ((__float_as_int(dmax) >> 23) & 0xff) - 127 + 2;
            const float to = __int_as_float((127 - e) << 23);
            const float f = to * wback;  // at the first move there is nothing to scale yet
            wmul = to;
            wmax = wback = __int_as_float((127 + e) << 23);
            if (!CLUSTER || step != begin)
#pragma unroll
              for (int i = 0; i < NB * NT * 8; ++i) (&o[0][0][0][0])[i] *= f;
          }
        }
        float w[NT][4];
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) w[i >> 2][i & 3] = s[i >> 2][i & 3] * wmul;
#pragma unroll
        for (int two = 0; two < NB; two += 2) {
          uint32_t v[4];  // of four tokens: bytes g, g + 8 of a block, and of the next one
          ldsm_bytes_trans(vb + two * 256 + v_at, v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int blk = two + h;
            uint32_t v0[4], v1[4];
            nibbles<NIB_LO>(v[2 * h], v[2 * h + 1], v0);
            nibbles<NIB_HI>(v[2 * h], v[2 * h + 1], v1);  // 16 times their values: taken off at the item's end
            // Less 8, exact: the sums of quants themselves would be many times what is left of them when m joins, and each product's
            // rounding would weigh as much more. (By two more products with -8 a block: 76.8 us instead of 73.8 for 262,143 tokens
            // of 8 heads of 128, and 3.4e-4 instead of 2.6e-4 off 64 bits.)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v0[i] = hsub2_u(v0[i], 0x00080008u);
              v1[i] = hsub2_u(v1[i], 0x00800080u);
            }
            const float e0 = lo_f32(d[blk]), e1 = hi_f32(d[blk]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {  // (pairs of tokens: e0 and e1 are next to each other as they come)
              const float2 r0 = mul2(make_float2(w[nt][0], w[nt][2]), make_float2(e0, e1));
              const float2 r1 = mul2(make_float2(w[nt][1], w[nt][3]), make_float2(e0, e1));
              const uint32_t b0 = transpose8(pack_f16(r0.x, r1.x));
              const uint32_t b1 = transpose8(pack_f16(r0.y, r1.y));
              mma16816_acc(o[blk][nt][0], v0, b0, b1);
              mma16816_acc(o[blk][nt][1], v1, b0, b1);
            }
          }
        }
      } else {
        if (__builtin_expect(masked, 0)) {
          // As for f16: scales of tokens that no row sees may be anything, and a NaN scale (of a token that
          // some rows do not see) is taken out and given to the rows that see it.
          uint16_t* sc = reinterpret_cast<uint16_t*>(vp + scales);
#pragma unroll
          for (int two = 0; two < NB; two += 2) {  // the 16 scales of each by a half of the warp
            uint16_t& x = sc[two * KV_GROUP + lane];
            const int tk = tok + ((lane & 15) >> 2) + 4 * (lane & 3);
            const bool seen = tk < sp.hi && tk >= sp.lo;
            const bool nan = seen && (x & 0x7FFF) > 0x7C00;
            if (!seen || nan) x = 0;
            const uint32_t both = __ballot_sync(0xffffffffu, nan);
            if (__builtin_expect(both == 0, 1)) continue;
#pragma unroll
            for (int blk = two; blk < two + 2; ++blk) {
              uint32_t odd = blk == two ? both & 0xffffu : both >> 16;
              while (odd) {
                const int j = __ffs(odd) - 1, tj = tok + (j >> 2) + 4 * (j & 3);
                odd &= odd - 1;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    int lo, hi;
                    row_sees(nt * 8 + 2 * t + c, lo, hi);
                    const float add = tj <= hi && tj > lo ? __int_as_float(0x7fffffff) : 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[blk][nt][e >> 1][2 * (e & 1) + c] += add;
                  }
              }
            }
          }
          __syncwarp();
        }
        uint32_t d[NB];
        __half2 big = __float2half2_rn(0.f);
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          uint32_t d0, d1;
          lds64(vb + scales + blk * 32 + scale_at, d0, d1);
          d[blk] = __byte_perm(d0, d1, scale_sel);
          big = __hmax2(big, *reinterpret_cast<__half2*>(&d[blk]));
        }
        float dmax = fmaxf(__low2float(big), __high2float(big));
        if (__builtin_expect(__any_sync(0xffffffffu, dmax > wmax), 0)) {
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 4));
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 8));
          dmax = fmaxf(dmax, __shfl_xor_sync(0xffffffffu, dmax, 16));
          // dmax < 2^(e-1): scales may double before the next move
          const int e = ((__float_as_int(dmax) >> 23) & 0xff) - 127 + 2;
          const float to = __int_as_float((127 + 7 - e) << 23);  // 2^(7-e)
          const float f = to * wback;  // at the first move there is nothing to scale yet
          wmul = to;
          wmax = __int_as_float((127 + e) << 23);
          wback = __int_as_float((127 - 7 + e) << 23);
          if (!CLUSTER || step != begin)
#pragma unroll
            for (int i = 0; i < NB * NT * 8; ++i) (&o[0][0][0][0])[i] *= f;
        }
        float w[NT][4];
#pragma unroll
        for (int i = 0; i < NT * 4; ++i) w[i >> 2][i & 3] = s[i >> 2][i & 3] * wmul;
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {
          uint32_t v[4];  // of four tokens: dimensions g, g + 8, g + 16, g + 24
          ldsm_bytes_trans(vb + blk * 512 + v_at, v);
          const uint32_t k1152 = 0x64806480u;  // f16 1024 + u, less 1152
          const uint32_t v0[4] = {hsub2_u(__byte_perm(v[0], k64, 0x4140), k1152), hsub2_u(__byte_perm(v[1], k64, 0x4140), k1152),
                                  hsub2_u(__byte_perm(v[0], k64, 0x4342), k1152), hsub2_u(__byte_perm(v[1], k64, 0x4342), k1152)};
          const uint32_t v1[4] = {hsub2_u(__byte_perm(v[2], k64, 0x4140), k1152), hsub2_u(__byte_perm(v[3], k64, 0x4140), k1152),
                                  hsub2_u(__byte_perm(v[2], k64, 0x4342), k1152), hsub2_u(__byte_perm(v[3], k64, 0x4342), k1152)};
          const float e0 = lo_f32(d[blk]), e1 = hi_f32(d[blk]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 lo = mul2(make_float2(w[nt][0], w[nt][1]), make_float2(e0, e0));
            const float2 hi = mul2(make_float2(w[nt][2], w[nt][3]), make_float2(e1, e1));
            const uint32_t w0 = transpose8(pack_f16(lo.x, lo.y));
            const uint32_t w1 = transpose8(pack_f16(hi.x, hi.y));
            mma16816_acc(o[blk][nt][0], v0, w0, w1);
            mma16816_acc(o[blk][nt][1], v1, w0, w1);
          }
        }
      }
      reads_done();
      if constexpr (TEAM == 1) refill(C::SPLIT);
      next();
    }

    if constexpr (TYPE == QG_Q4_1) {  // quants came as multiples of 2^-24 and 2^-20; and what is the blocks' joins
      const float back[2] = {wback * 16777216.f, wback * 1048576.f};
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float m = __shfl_sync(0xffffffffu, om[nt][c], 4 * blk + t);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float& x = o[blk][nt][e >> 1][2 * (e & 1) + c];
              x = fmaf(x, back[e >> 1], m);
            }
          }
      wback = 1.f;
    }
    // ------------------------------------------------ the four warps' sums
    const size_t part = (size_t)cta * 2 + (starts ? 1 : 0);
    float* const s_z = s_stat + turn * (2 * AT_WARPS + 2) * ROWS;  // [warp][row]
    float* const s_l = s_z + AT_WARPS * ROWS;                       // [warp][row]
    float* const s_top = s_l + AT_WARPS * ROWS;                     // [row]
    float* const s_sum = s_top + ROWS;                              // [row]
    turn ^= 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[nt][c];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          s_z[warp * ROWS + nt * 8 + 2 * t + c] = ref(nt, c);
          s_l[warp * ROWS + nt * 8 + 2 * t + c] = share ? 0.f : x;  // (a team's warps have the same weights)
        }
      }
    __syncthreads();
    if (C::QSMEM && step < steps) stage_q(at);  // (all warps are through with the queries)
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = nt * 8 + 2 * t + c;
        float x = s_z[row];
#pragma unroll
        for (int w = 1; w < AT_WARPS; ++w) x = fmaxf(x, s_z[w * ROWS + row]);
        f[nt][c] = limit[nt][c] == -INFINITY ? 0.f : ex2((z[nt][c] - x) * p.mul) * wback;
      }
    if (tid < ROWS) {
      float top = s_z[tid], sum = 0.f;
#pragma unroll
      for (int w = 1; w < AT_WARPS; ++w) top = fmaxf(top, s_z[w * ROWS + tid]);
#pragma unroll
      for (int w = 0; w < AT_WARPS; ++w) {
        const float x = s_z[w * ROWS + tid];
        sum += x == -INFINITY ? s_l[w * ROWS + tid] : s_l[w * ROWS + tid] * ex2((x - top) * p.mul);
      }
      s_top[tid] = top;
      s_sum[tid] = sum;
    }
    if constexpr (CLUSTER) {
      // The CTA's only item: the ring is free, and takes all four sums at once.
      float* const s_all = reinterpret_cast<float*>(s_ring);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float* const to = s_all + warp * (ROWS * D) + in_sums(2 * t, dim_of(e));
#pragma unroll
        for (int blk = 0; blk < NB; ++blk)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              to[(nt * 8 + c) * D + blk * 32] = f[nt][c] == 0.f ? 0.f : o[blk][nt][e >> 1][2 * (e & 1) + c] * f[nt][c];
      }
      __syncthreads();
      for (int i = tid * 4; i < ROWS * D; i += AT_THREADS * 4) {
        float4 y = *reinterpret_cast<const float4*>(s_all + i);
#pragma unroll
        for (int w = 1; w < AT_WARPS; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(s_all + w * (ROWS * D) + i);
          y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
        }
        *reinterpret_cast<float4*>(s_all + i) = y;
      }
    } else {
#pragma unroll
      for (int pass = 0; pass < NB * 32 / C::OD; ++pass) {
        if (pass) __syncthreads();  // the buffer has been read
#pragma unroll
        for (int hb = 0; hb < C::OD / 32; ++hb) {
          const int blk = pass * (C::OD / 32) + hb;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                s_o[(warp * ROWS + nt * 8 + 2 * t + c) * C::OPITCH + hb * 32 + (dim_of(e) ^ at_swap<TYPE>(2 * t))] =
                    f[nt][c] == 0.f ? 0.f : o[blk][nt][e >> 1][2 * (e & 1) + c] * f[nt][c];
        }
        __syncthreads();
        constexpr int QUADS = C::OD / 4;  // float4 of a row of each share
#pragma unroll
        for (int k = 0; k < (TEAM * ROWS * QUADS + AT_THREADS - 1) / AT_THREADS; ++k) {
          const int i = tid + k * AT_THREADS, of = i / (ROWS * QUADS), row = i / QUADS % ROWS, dim = (i % QUADS) * 4;
          const int r = tile * ROWS + row;
          if (of >= TEAM || r >= rows) continue;
          float4 y = *reinterpret_cast<const float4*>(s_o + (of * ROWS + row) * C::OPITCH + (dim ^ at_swap<TYPE>(row)));
#pragma unroll
          for (int w = TEAM; w < AT_WARPS; w += TEAM) {
            const float4 x = *reinterpret_cast<const float4*>(s_o + ((of + w) * ROWS + row) * C::OPITCH + (dim ^ at_swap<TYPE>(row)));
            y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
          }
          const int at = of * (NB * 32) + pass * C::OD + dim;
          const float sum = s_sum[row];
          if (whole) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const size_t yo = (((size_t)b * a.ncols + r / p.group) * a.n_heads + head * p.group + r % p.group) * D + at;
            *reinterpret_cast<uint2*>(a.y + yo) =
                make_uint2(pack_f16(y.x * inv, y.y * inv), pack_f16(y.z * inv, y.w * inv));
          } else {
            *reinterpret_cast<float4*>(p.ws.o + (part * ROWS + row) * D + at) = y;
            if (at == 0) *reinterpret_cast<float2*>(p.ws.zl + (part * ROWS + row) * 2) = make_float2(s_top[row], sum);
          }
        }
      }
    }
  }
  if constexpr (CLUSTER) {
    // The CTAs' sums are in the rings (their only item is over), references and weights where the item's end left them.
    static_assert((size_t)AT_WARPS * ROWS * D * 4 <= C::ring && TEAM == 1, "the sums fit the ring");
    float* const s_top = s_stat + 2 * AT_WARPS * ROWS;
    float* const s_sum = s_top + ROWS;
    if (steps == 0) {
      copies_done();
      if (tid < ROWS) {
        s_top[tid] = -INFINITY;
        s_sum[tid] = 0.f;
      }
    }
    __syncwarp();
    cluster_barrier();
    const int head = p.head_of(whose.item), r0 = (whose.item - head * p.tiles) * ROWS;
    const int pairs = (rows - r0 < ROWS ? rows - r0 : ROWS) * (D / 2);
    for (int i = rank * AT_THREADS + tid; i < pairs; i += ctas * AT_THREADS) {
      const int row = i / (D / 2), dim = i % (D / 2) * 2, r = r0 + row;
      const uint32_t v_at = in_sums(row, dim) * 4, z_at = (uint32_t)(reinterpret_cast<uint8_t*>(s_top + row) - smem);
      float z[AT_CLUSTER], l[AT_CLUSTER], top = -INFINITY;
      float2 v[AT_CLUSTER];
#pragma unroll
      for (int j = 0; j < AT_CLUSTER; ++j) {
        z[j] = -INFINITY;
        l[j] = 0.f;
        if (j < ctas) {
          const uint32_t its = at_rank(smem, j);
          z[j] = ld_rank(its + z_at);
          l[j] = ld_rank(its + z_at + ROWS * 4);
          v[j] = ld_rank2(its + v_at);
        }
      }
#pragma unroll
      for (int j = 0; j < AT_CLUSTER; ++j) top = fmaxf(top, z[j]);
      float sum = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
      for (int j = 0; j < AT_CLUSTER; ++j) {
        const float w = z[j] == -INFINITY ? 0.f : ex2((z[j] - top) * p.mul);
        sum += z[j] == -INFINITY ? l[j] : l[j] * w;
        if (w != 0.f) {
          y0 = fmaf(v[j].x, w, y0);
          y1 = fmaf(v[j].y, w, y1);
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const size_t yo = (((size_t)whose.seq * a.ncols + r / p.group) * a.n_heads + head * p.group + r % p.group) * D + dim;
      *reinterpret_cast<uint32_t*>(a.y + yo) = pack_f16(y0 * inv, y1 * inv);
    }
    __syncwarp();
    cluster_barrier();  // nobody leaves while the others read
  }
  if (!ok) {  // a copy was late: wait for what is still in flight, each wait bounded
    for (int i = 0; i < C::BARS; ++i) mbar_try_wait(bar_at + 8 * i, parity);
  }
}

// Joins the parts of the items that are cut. blockIdx.x is an item (by_item) or, where there are more items than CTAs of
// the main kernel, one of those CTAs: the last item that starts in its run is the only one that may be cut. WIDE: a CTA
// joins a row and its warps share the parts out, for few items of many parts; otherwise a warp joins a row.
template <int D, int ROWS, bool WIDE, int GRID, int PAD>
__global__ void __launch_bounds__(WIDE ? 256 : 128, WIDE ? 3 : 8) attn_join_kernel(const __grid_constant__ AttnDev p, int by_item) {
  constexpr int THREADS = WIDE ? 256 : 128, WARPS = THREADS / 32;
  constexpr int V = D / 32;               // dimensions of a lane
  // Parts in flight. A row of its own warp has few parts, and with few registers most of the CTAs find room (and get
  // through their first part) before the main kernel's last CTAs end.
  constexpr int BATCH = V == 2 ? 12 : WIDE && V == 4 ? 8 : 4;
  __shared__ float s_y[WIDE ? WARPS : 1][D];
  __shared__ float2 s_zl[WARPS];
  __shared__ int s_part[WARPS];
  extern __shared__ int32_t s_runs[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = WIDE ? blockIdx.y : blockIdx.y * WARPS + warp;
  pdl_trigger();
  // The main kernel lets this one start once what came before it is complete; so before pdl_wait only its parts are not.
  const Runs<THREADS, at_unit(D, ROWS / 8), PAD, GRID> runs(p.a, p.tiles, s_runs, s_part, false);
  Unit x;
  int c0 = blockIdx.x, n = 0;
  if (by_item) {
    x.seq = blockIdx.x / runs.items;
    x.item = blockIdx.x - x.seq * runs.items;
    const int v = runs.v_item(x.seq, x.item);
    c0 = runs.run_of(v);
    n = runs.run_of(v + runs.units_of(x.seq) - 1) - c0 + 1;
    if (n == 1) n = 0;
  } else if (c0 < runs.N) {
    // cut is the item that run c0 ends in the middle of, if it starts in that run
    Unit first;
    int u0, u1;
    runs.find(c0, first, u0, x, u1);
    if (x.unit > 0) {
      const int v = runs.v_item(x.seq, x.item);
      if (v >= runs.run_start(c0)) n = runs.run_of(v + runs.units_of(x.seq) - 1) - c0 + 1;
    }
  }
  const int head = p.head_of(x.item), tile = x.item - head * p.tiles;
  const int r = tile * ROWS + row;
  pdl_wait();
  if (n == 0 || row >= ROWS || r >= p.group * p.a.ncols) return;
  // part i: the first CTA's run ends in the item (its second slot), the others' start in it
  auto slot = [&](int i) { return ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + row; };
  // a warp's parts, with a reference that moves as they come
  float top = -INFINITY, sum = 0.f, y[V];
#pragma unroll
  for (int k = 0; k < V; ++k) y[k] = 0.f;
  constexpr int STEP = WIDE ? WARPS : 1;
  for (int i0 = WIDE ? warp : 0; i0 < n; i0 += BATCH * STEP) {
    float part[BATCH][V];
    float2 zl[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const int i = i0 + j * STEP;
      zl[j] = make_float2(-INFINITY, 0.f);
      if (i < n) {
        zl[j] = __ldcg(reinterpret_cast<const float2*>(p.ws.zl + slot(i) * 2));
        const float* const o = p.ws.o + slot(i) * D + lane * V;
        if constexpr (V == 2) {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(o));
          part[j][0] = v.x; part[j][1] = v.y;
        } else {
#pragma unroll
          for (int k = 0; k < V; k += 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(o + k));
            part[j][k] = v.x; part[j][k + 1] = v.y; part[j][k + 2] = v.z; part[j][k + 3] = v.w;
          }
        }
      }
    }
    float z = top;
#pragma unroll
    for (int j = 0; j < BATCH; ++j) z = fmaxf(z, zl[j].x);
    const float f = top == -INFINITY ? 0.f : ex2((top - z) * p.mul);
    sum = top == -INFINITY ? sum : sum * f;  // (a part that has seen nothing but NaN has a sum of its own)
#pragma unroll
    for (int k = 0; k < V; ++k) y[k] *= f;
    top = z;
#pragma unroll
    for (int j = 0; j < BATCH; ++j) {
      const float w = zl[j].x == -INFINITY ? 0.f : ex2((zl[j].x - top) * p.mul);
      sum += zl[j].x == -INFINITY ? zl[j].y : zl[j].y * w;
      if (w != 0.f)
#pragma unroll
        for (int k = 0; k < V; ++k) y[k] = fmaf(part[j][k], w, y[k]);
    }
  }
  const size_t yo = (((size_t)x.seq * p.a.ncols + r / p.group) * p.a.n_heads + head * p.group + r % p.group) * D;
  if constexpr (WIDE) {
#pragma unroll
    for (int k = 0; k < V; ++k) s_y[warp][lane * V + k] = y[k];
    if (lane == 0) s_zl[warp] = make_float2(top, sum);
    __syncthreads();
    float z = -INFINITY, l = 0.f, w[WARPS];
#pragma unroll
    for (int i = 0; i < WARPS; ++i) z = fmaxf(z, s_zl[i].x);
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      const float2 t = s_zl[i];
      w[i] = t.x == -INFINITY ? 0.f : ex2((t.x - z) * p.mul);
      l += t.x == -INFINITY ? t.y : t.y * w[i];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = tid; e < D; e += THREADS) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < WARPS; ++i) v += w[i] == 0.f ? 0.f : s_y[i][e] * w[i];
      p.a.y[yo + e] = __half_as_ushort(__float2half_rn(v * inv));
    }
  } else {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int k = 0; k < V; k += 2)
      *reinterpret_cast<uint32_t*>(p.a.y + yo + lane * V + k) = pack_f16(y[k] * inv, y[k + 1] * inv);
  }
}

template <int D, int NT>
constexpr int attn_grid_q4() {
  if constexpr (NT <= at_most(QG_Q4_1, D)) return AttnCfg<QG_Q4_1, D, NT>::GRID;
  return 0;
}
// (the largest of the types': the workspace's size does not depend on it)
template <int D, int NT>
constexpr size_t attn_ws_of() {
  constexpr int of_q8 = AttnCfg<QG_Q8_0, D, NT>::GRID, of_q4 = attn_grid_q4<D, NT>(), grid = of_q8 > of_q4 ? of_q8 : of_q4;
  static_assert(grid >= AttnCfg<QG_F16, D, NT>::GRID, "room for f16, too");
  return (size_t)grid * ((size_t)2 * 8 * NT * (8 + D * 4));
}

template <int TYPE, int D, int NT>
cudaError_t attn_typed(const AttnArgs& a, cudaStream_t s) {
  using C = AttnCfg<TYPE, D, NT>;
  AttnDev p;
  p.a = a;
  p.group = a.n_heads / a.c.n_kv_heads;
  const int all = p.group * a.ncols;
  p.tiles = (all + C::ROWS - 1) / C::ROWS;
  // scores are compared before they are scaled, so the scale's sign goes to the queries
  // Kept within 2^+-100, beyond which the weights no longer depend on it: raw scores of finite queries and keys are 0 or at
  // least 2^-72 apart (products of 2^-24 steps, and the scale's for Q8_0) and below 2^48, so that at 2^100 one step takes a
  // weight to 0 and at 2^-100 all weigh 1.
  const double mul = std::fabs((double)a.scale) * 1.4426950408889634 * (TYPE == QG_F16 ? 1. : 16777216.);
  p.mul = a.scale == 0.f ? 1.f : (float)std::fmin(std::fmax(mul, std::ldexp(1., -100)), std::ldexp(1., 100));
  p.slack = (float)(AT_SLACK / (double)p.mul);
  p.q_and = a.scale == 0.f ? 0u : 0xffffffffu;
  p.q_xor = a.scale < 0.f ? 0x80008000u : 0u;
  const int n_items = a.c.n_seq * a.c.n_kv_heads * p.tiles;
  const int tile_rows = all < C::ROWS ? all : C::ROWS;
  // As many CTAs as there can be places. Where they leave every SM room for another, the kernel is launched early.
  constexpr int unit = at_unit(D, NT);
  int64_t most = ((int64_t)a.c.max_pages * a.c.page_size + unit - 1) / unit;  // units of a sequence
  if (a.window > 0 && a.window / unit + 3 < most) most = a.window / unit + 3;
  if constexpr (NT <= 2) {
    int ctas = AT_CLUSTER;
    while (ctas > 1 && (int64_t)n_items * ctas > 2 * AT_SMS) ctas /= 2;
    if (most <= AT_CLUSTER_UNITS * ctas && (int64_t)n_items * ctas <= C::GRID) {
      const cudaError_t e = prepare_kernel((const void*)attn_kernel<TYPE, D, NT, true>, C::smem(0), true);
      if (e != cudaSuccess) return e;
      return launch_pdl(attn_kernel<TYPE, D, NT, true>, dim3(n_items * ctas), dim3(AT_THREADS), C::smem(0), s, ctas,
                        n_items * ctas <= AT_SMS ? LC_SMEM : LC_FULL, p);
    }
  }
  most = (most + at_pad(TYPE, NT)) * n_items;
  const int grid = most < C::GRID ? (int)most : C::GRID;
  const bool early = grid <= AT_SMS;
  const bool by_item = n_items <= grid, wide = n_items <= 4 * AT_SMS / tile_rows;
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  p.ws.zl = reinterpret_cast<float*>(ws);
  ws += (size_t)C::GRID * 2 * C::ROWS * 8;
  p.ws.o = reinterpret_cast<float*>(ws);
  const size_t smem = C::smem(a.c.n_seq);
  cudaError_t e = prepare_kernel((const void*)attn_kernel<TYPE, D, NT, false>, smem, false);
  if (e != cudaSuccess) return e;
  const auto join = wide ? attn_join_kernel<D, C::ROWS, true, C::GRID, at_pad(TYPE, NT)> : attn_join_kernel<D, C::ROWS, false, C::GRID, at_pad(TYPE, NT)>;
  e = launch_pdl(attn_kernel<TYPE, D, NT, false>, dim3(grid), dim3(AT_THREADS), smem, s, 0, early ? LC_SMEM : LC_FULL, p);
  if (e != cudaSuccess) return e;
  const dim3 join_grid(by_item ? n_items : grid, wide ? tile_rows : (tile_rows + 3) / 4);
  return launch_pdl(join, join_grid, dim3(wide ? 256 : 128), (size_t)(2 * a.c.n_seq + 1) * 4, s, 0, LC_SMEM, p,
                    (int)by_item);
}

inline cudaError_t attn_error_word(int32_t* bits) {
  const int32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_attn_error, sizeof(*bits));
  return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_attn_error, &zero, sizeof(zero));
}

}  // namespace
}  // namespace qg
