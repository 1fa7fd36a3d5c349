// qg_attn.h -- the attention's launchers by head size, between its translation
// units. nt: row tiles of 8 that a CTA handles together, a power of two: up to 8 at
// heads of 64 and 4 above, half of that for Q8_0.
#pragma once
#include "qg_internal.h"

namespace qg {

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
