// qg_attn_128.cu -- attention over the paged cache, heads of 128 (kernels in qg_attn.cuh).
#include "qg_attn.cuh"
#include "qg_attn.h"

namespace qg {

template <int NT>
static cudaError_t launch_tiles(const AttnArgs& a, cudaStream_t s) {
  if (a.c.type == QG_F16) return attn_typed<QG_F16, 128, NT>(a, s);
  if constexpr (NT <= at_most(QG_Q8_0, 128)) {
    if (a.c.type == QG_Q8_0) return attn_typed<QG_Q8_0, 128, NT>(a, s);
    if (a.c.type == QG_Q4_1) return attn_typed<QG_Q4_1, 128, NT>(a, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t attn_launch_128(const AttnArgs& a, int nt, cudaStream_t s) {
  switch (nt) {
    case 1: return launch_tiles<1>(a, s);
    case 2: return launch_tiles<2>(a, s);
    case 4: return launch_tiles<4>(a, s);
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
