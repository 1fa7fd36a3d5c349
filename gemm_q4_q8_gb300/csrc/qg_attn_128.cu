// qg_attn_128.cu -- attention over the paged cache, heads of 128 (kernels in qg_attn.cuh).
#include "qg_attn.cuh"
#include "qg_attn.h"

namespace qg {

cudaError_t attn_launch_128(const AttnArgs& a, int nt, cudaStream_t s) {
  const bool f16 = a.c.type == QG_F16;
  switch (nt) {
    case 1: return f16 ? attn_typed<QG_F16, 128, 1>(a, s) : attn_typed<QG_Q8_0, 128, 1>(a, s);
    case 2: return f16 ? attn_typed<QG_F16, 128, 2>(a, s) : attn_typed<QG_Q8_0, 128, 2>(a, s);
    case 4: return f16 ? attn_typed<QG_F16, 128, 4>(a, s) : cudaErrorInvalidValue;
  }
  return cudaErrorInvalidValue;
}

size_t attn_ws_128(int nt) {
  switch (nt) {
    case 1: return attn_ws_of<128, 1>();
    case 2: return attn_ws_of<128, 2>();
    case 4: return attn_ws_of<128, 4>();
  }
  return 0;
}

cudaError_t attn_error_128(int32_t* bits) { return attn_error_word(bits); }

}  // namespace qg
