// The tile kernel of prefill and split verify with a sliding window and sinks: bf16 and E4M3 caches.
#include "pa_prefill.cuh"

namespace pa {

cudaError_t prefill_window_form(const AttnParams& p, const Launch& l, int max_q_len, int32_t* tiles,
                                const CUtensorMap& tk, const CUtensorMap& tv) {
  if (l.head_dim == 128)
    return l.kv == kKvE4m3 ? prefill_form<128, kKvE4m3, kFormWindow>(p, l, max_q_len, tiles, tk, tv)
                           : prefill_form<128, kKvBf16, kFormWindow>(p, l, max_q_len, tiles, tk, tv);
  if (l.head_dim == 64)
    return l.kv == kKvE4m3 ? prefill_form<64, kKvE4m3, kFormWindow>(p, l, max_q_len, tiles, tk, tv)
                           : prefill_form<64, kKvBf16, kFormWindow>(p, l, max_q_len, tiles, tk, tv);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
