// Prompt attention whose items several CTAs share (pkv_prompt_body.cuh): a unit of
// its own, so that both compile at a time.
#include "pkv_prompt_body.cuh"

namespace pkv {

cudaError_t launch_prompt_shared(const PromptArgs& a, int d_head, long long ctas,
                                 const CUtensorMap* tq, const CUtensorMap* tk,
                                 const CUtensorMap* tv, cudaStream_t stream) {
  return launch_prompt<true>(a, d_head, ctas, tq, tk, tv, stream);
}

// Device address of this unit's error word on the current device.
cudaError_t prompt_shared_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_prompt_error);
}

unsigned read_prompt_shared_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_prompt_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

}  // namespace pkv
