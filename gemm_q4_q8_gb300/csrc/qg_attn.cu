// qg_attn.cu -- attention over the paged key/value cache (qattn_paged): the
// choice of kernel (qg_attn.cuh).
#include "qg_attn.h"

namespace qg {

namespace {

// Row tiles of 8 that a CTA handles together: as few as hold the rows of a kv
// head, at most as many as leave the accumulator (8 NT x head_dim over a warp; two
// warps for 32 rows of 256) 128 registers a thread. Q8_0 needs more registers
// beside it and takes at most half as many (64 rows of heads of 64, 16 sequences
// of 8,191 tokens: 121 us with eight tiles, 102 with two times four, f16 85 and
// 102; 32 rows of heads of 128, Q8_0: 58 either way). More rows are further items,
// which read the keys and values again (from L2, mostly).
int tiles_of(int type, int rows, int head_dim) {
  const int most = (head_dim == 64 ? 8 : 4) / (type == QG_F16 ? 1 : 2);
  int nt = 1;
  while (nt < most && nt * 8 < rows) nt *= 2;
  return nt;
}
size_t ws_of(int type, int rows, int head_dim) {
  const int nt = tiles_of(type, rows, head_dim);
  return head_dim == 64 ? attn_ws_64(nt) : head_dim == 128 ? attn_ws_128(nt) : attn_ws_256(nt);
}

}  // namespace

bool attn_shape_ok(int n_seq, int n_heads, int n_kv_heads, int head_dim, int ncols) {
  return n_seq >= 1 && n_seq <= QG_KV_MAX_SEQ && n_kv_heads >= 1 && n_kv_heads <= 256 && n_heads >= n_kv_heads &&
         n_heads % n_kv_heads == 0 && n_heads / n_kv_heads <= QG_ATTN_MAX_GROUP &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && ncols >= 1 && ncols <= QG_ATTN_MAX_COLS;
}

// The kernel numbers an item's units, and its at_pad places behind them, in 32 bits: no more than a whole number of 32 tokens,
// a partly filled unit and 7 places.
bool attn_size_ok(const qg_kvcache& c, int n_heads, int ncols) {
  static_assert(at_unit(256, 4) >= 32 && at_unit(64, 8) >= 32 && at_pad(1) <= 7 && at_pad(8) <= 7, "units + 8 are enough");
  const int rows = n_heads / c.n_kv_heads * ncols, nt = tiles_of(c.type, rows, c.head_dim);
  const int64_t tiles = (rows + 8 * nt - 1) / (8 * nt);
  const int64_t units = (int64_t)c.max_pages * c.page_size / 32 + 8;
  return units * c.n_seq * c.n_kv_heads * tiles < ((int64_t)1 << 31);
}

// (the larger of the two types': the call does not name one)
size_t attn_ws_bytes(int, int n_heads, int n_kv_heads, int head_dim, int ncols) {
  const int rows = n_heads / n_kv_heads * ncols;
  const size_t a = ws_of(QG_F16, rows, head_dim), b = ws_of(QG_Q8_0, rows, head_dim);
  return a > b ? a : b;
}

cudaError_t attn_launch(const AttnArgs& a, cudaStream_t s) {
  const int nt = tiles_of(a.c.type, a.n_heads / a.c.n_kv_heads * a.ncols, a.c.head_dim);
  return a.c.head_dim == 64    ? attn_launch_64(a, nt, s)
         : a.c.head_dim == 128 ? attn_launch_128(a, nt, s)
                               : attn_launch_256(a, nt, s);
}

cudaError_t attn_device_error(int32_t* bits) {
  *bits = 0;
  for (auto read : {attn_error_64, attn_error_128, attn_error_256}) {
    int32_t b = 0;
    const cudaError_t e = read(&b);
    if (e != cudaSuccess) return e;
    *bits |= b;
  }
  return cudaSuccess;
}

}  // namespace qg
