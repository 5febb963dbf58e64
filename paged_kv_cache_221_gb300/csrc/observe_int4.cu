// Accumulated attention weights over int4 K pages.
#include "pa_observe.cuh"

namespace pa {

cudaError_t launch_observe_int4(const ObserveParams& p, int head_dim, int rows, cudaStream_t s) {
  return head_dim == 64 ? launch_observe<kPageInt4, 64>(p, rows, s)
                        : launch_observe<kPageInt4, 128>(p, rows, s);
}

cudaError_t take_error_observe_int4(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
