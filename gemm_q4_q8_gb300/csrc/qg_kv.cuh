// qg_kv.cuh -- the byte layout of the paged key/value cache, shared by the
// kernels that write it (qg_rope.cu), read it back (qg_kv.cu) and attend over
// it (qg_attn.cuh).
//
// The unit is the record of 16 consecutive tokens of one head: its key half,
// then its value half, each contiguous, so one bulk copy fetches either. Inside
// a half the D dimensions are split in blocks of 32 and the 16 tokens' rows of a
// block lie next to each other: in the attention kernel the eight lanes of a
// shared-memory access phase then read neighbouring rows, without bank
// conflicts, whatever D is. Q8_0 scales are stored in the order in which a lane
// needs them: lane t of a quad owns tokens t, t + 4, t + 8, t + 12.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "qgemm.h"

namespace qg {

constexpr int KV_GROUP = 16;  // tokens of a record

__host__ __device__ constexpr int kv_half_bytes(int type, int d) {
  return type == QG_F16 ? 32 * d : 17 * d;
}
__host__ __device__ constexpr int kv_record_bytes(int type, int d) { return 2 * kv_half_bytes(type, d); }
__host__ __device__ inline size_t kv_page_bytes(int type, int heads, int d, int page_size) {
  return (size_t)heads * (page_size / KV_GROUP) * kv_record_bytes(type, d);
}
// Place of token i's scale among the 16 of a block.
__host__ __device__ constexpr int kv_scale_place(int i) { return 4 * (i & 3) + (i >> 2); }

// The page of position `pos` of sequence `seq`, or -1 with the reason ORed into
// *bits. pos >= 0.
__device__ __forceinline__ int kv_page_of(const qg_kvcache& c, int seq, int pos, int* bits) {
  if (seq < 0 || seq >= c.n_seq) {
    *bits |= QG_KV_BAD_SEQ;
    return -1;
  }
  const int j = pos / c.page_size;
  if (j >= c.max_pages) {
    *bits |= QG_KV_BAD_POS;
    return -1;
  }
  const int page = c.page_table[(size_t)seq * c.max_pages + j];
  if (page < 0 || page >= c.n_pages) {
    *bits |= QG_KV_BAD_PAGE;
    return -1;
  }
  return page;
}

}  // namespace qg
