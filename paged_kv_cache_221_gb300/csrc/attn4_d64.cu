// Attention over 4-bit pages, head_dim 64.
#include "pa_attn4.cuh"

namespace pa {

cudaError_t launch_attn4_d64(const AttnParams& p, int rows, unsigned units, cudaStream_t s) {
  return launch_attn4<64>(p, rows, units, s);
}

cudaError_t take_error_attn4_d64(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
