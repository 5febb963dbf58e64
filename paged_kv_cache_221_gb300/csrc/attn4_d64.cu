// Attention over 4-bit pages, head_dim 64.
#include <algorithm>

#include "pa_attn4.cuh"

namespace pa {

cudaError_t launch_attn4_d64(const Attn4Params& p, int rows, cudaStream_t s) {
  return launch_attn4<64>(p, rows, s);
}

cudaError_t take_error_attn4_d64(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
