// The tile kernel of prefill and split verify over 4-bit caches, with and without a window.
#include "pa_prefill.cuh"

namespace pa {

cudaError_t prefill_fp4_form(const AttnParams& p, const Launch& l, int max_q_len, int32_t* tiles) {
  const CUtensorMap none = {};  // 4-bit pages move as plain bulk copies
  const bool win = p.window > 0;
  if (l.head_dim == 128)
    return win ? prefill_form<128, kKvFp4, true>(p, l, max_q_len, tiles, none, none)
               : prefill_form<128, kKvFp4, false>(p, l, max_q_len, tiles, none, none);
  if (l.head_dim == 64)
    return win ? prefill_form<64, kKvFp4, true>(p, l, max_q_len, tiles, none, none)
               : prefill_form<64, kKvFp4, false>(p, l, max_q_len, tiles, none, none);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
