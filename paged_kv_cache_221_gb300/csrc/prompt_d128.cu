// Prompt attention, head_dim 128.
#include "pa_prompt.cuh"

namespace pa {

cudaError_t launch_prompt_d128(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const PromptParams& p, bool kv8, cudaStream_t s) {
  return kv8 ? launch_prompt_as<128, true>(tq, tk, tv, p, s)
             : launch_prompt_as<128, false>(tq, tk, tv, p, s);
}

cudaError_t take_error_prompt_d128(unsigned* bits) { return read_error_word(bits); }

}  // namespace pa
