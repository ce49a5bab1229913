// Attention of whole prompts (pkv_prompt_body.cuh), and the choice between items
// of one CTA and items that several CTAs share.
#include "pkv_prompt_body.cuh"

namespace pkv {

int prompt_tile_rows() { return kPrRows; }
int prompt_tile_keys() { return kPrKeys; }

cudaError_t launch_prompt_attention(PromptArgs a, int d_head, int num_sms, const CUtensorMap* tq,
                                    const CUtensorMap* tk, const CUtensorMap* tv,
                                    cudaStream_t stream) {
  const int tpc = kPrRows / (a.q_heads / a.kv_heads) * kPrTiles;
  const long long items = (a.total_q / tpc + (long long)a.num_seqs) * a.kv_heads;  // at most
  // Few items: as many CTAs to each as there are SMs, two key tiles or more a CTA.
  a.split = 1;
  while (a.split < kPrMaxSplit && items * a.split * 2 <= num_sms &&
         a.max_keys / kPrKeys >= a.split * 4)
    a.split *= 2;
  if (a.split > 1)
    return launch_prompt_shared(a, d_head, items * a.split, tq, tk, tv, stream);
  return launch_prompt<false>(a, d_head, std::min<long long>(items, num_sms), tq, tk, tv, stream);
}

// Device address of this unit's error word on the current device.
cudaError_t prompt_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_prompt_error);
}

unsigned read_prompt_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_prompt_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

}  // namespace pkv
