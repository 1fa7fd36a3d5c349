// qg_attn.h -- the attention's launchers by head size, between its translation
// units. nt: row tiles of 8 that a CTA handles together, a power of two: up to 8 at
// heads of 64 and 4 above, half of that for Q8_0.
#pragma once
#include "qg_internal.h"
#include "qg_kv.cuh"

namespace qg {

constexpr int AT_WARPS = 4;
// Warps that share a record: 32 rows of heads of 256 are split between two, 128 dimensions each, which add their scores
// up; each then has the registers of a warp on heads of 128. (16 sequences of 8,191 f16 tokens, two kv heads, 32 rows:
// 68 us, against 90 for two tiles of 16 rows that read everything twice. For fewer rows, and for Q8_0, a warp on its own
// is faster: f16, 8 rows 47 us against 50, 16 rows 51 against 56; Q8_0, 16 rows 36 against 42, 32 rows 56 as two tiles
// of 16 against 65 or, as one, 68.)
__host__ __device__ constexpr int at_team(int d, int nt) { return d == 256 && nt == 4 ? 2 : 1; }
// Tokens of a unit: a record of 16 for every team of the CTA.
__host__ __device__ constexpr int at_unit(int d, int nt) { return AT_WARPS / at_team(d, nt) * KV_GROUP; }
// An item's end (four warps' sums joined, the next queries taken up) costs a CTA about as much as this many units, and
// the runs are cut as if it were that many more (measured: 1.2 units at 8 rows of heads of 128, 4.3 at 32 rows of 64).
__host__ __device__ constexpr int at_pad(int nt) { return nt == 1 ? 2 : 4; }

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
