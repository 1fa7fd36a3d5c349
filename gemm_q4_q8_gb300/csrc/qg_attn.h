// qg_attn.h -- the attention's launchers by head size, between its translation
// units. nt: row tiles of 8 that a CTA handles together, a power of two, up to at_most.
#pragma once
#include "qg_internal.h"
#include "qg_kv.cuh"

namespace qg {

constexpr int AT_WARPS = 4;
// Row tiles of a CTA, at most: as many as leave the accumulator (8 nt x head_dim over a warp; two warps for 32 rows of 256)
// 128 registers a thread. The quantised types need more registers beside it and take at most half as many (Q8_0, 64 rows of
// heads of 64, 16 sequences of 8,191 tokens: 121 us with eight tiles, 102 with two times four, f16 85 and 102; 32 rows of heads
// of 128: 58 either way).
__host__ __device__ constexpr int at_most(int type, int d) { return (d == 64 ? 8 : 4) / (type == QG_F16 ? 1 : 2); }
// Warps that share a record: 32 rows of heads of 256 are split between two, 128 dimensions each, which add their scores
// up; each then has the registers of a warp on heads of 128. (16 sequences of 8,191 f16 tokens, two kv heads, 32 rows:
// 68 us, against 90 for two tiles of 16 rows that read everything twice. For fewer rows, and for Q8_0, a warp on its own
// is faster: f16, 8 rows 47 us against 50, 16 rows 51 against 56; Q8_0, 16 rows 36 against 42, 32 rows 56 as two tiles
// of 16 against 65 or, as one, 68.)
__host__ __device__ constexpr int at_team(int d, int nt) { return d == 256 && nt == 4 ? 2 : 1; }
// Tokens of a unit: a record of 16 for every team of the CTA.
__host__ __device__ constexpr int at_unit(int d, int nt) { return AT_WARPS / at_team(d, nt) * KV_GROUP; }
// An item's end (four warps' sums joined, the next queries taken up) costs a CTA about as much as this many units, and
// the runs are cut as if it were that many more (measured: 1.2 units at 8 rows of heads of 128, 4.3 at 32 rows of 64). Q4_1, 64
// ragged sequences, 8 heads of 128: 68.4 us with 2, 64.5 with 3, 65.4 with 4, 66.2 with 5; 16 rows 96.9 with 3, 94.3 with 4, 97.8 with 6.
// Others of 32 to 8,192 tokens with 2, 3 and 4: 8 heads of 64 40.1, 36.0 and 36.0 us, 4 heads of 256 54.4, 50.3 and 48.3.
__host__ __device__ constexpr int at_pad(int type, int nt) { return nt > 1 ? 4 : type == QG_Q4_1 ? 3 : 2; }

cudaError_t attn_launch_64(const AttnArgs& a, int nt, cudaStream_t s);
cudaError_t attn_launch_128(const AttnArgs& a, int nt, cudaStream_t s);
cudaError_t attn_launch_256(const AttnArgs& a, int nt, cudaStream_t s);
size_t attn_ws_64(int nt);
size_t attn_ws_128(int nt);
size_t attn_ws_256(int nt);
cudaError_t attn_error_64(int32_t* bits);
cudaError_t attn_error_128(int32_t* bits);
cudaError_t attn_error_256(int32_t* bits);

}  // namespace qg
