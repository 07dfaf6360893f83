// A few rows per kv head with a window over bf16 and E4M3 caches (verify, and decode of the groups that
// the decode kernel has no form for).
#include "pa_rows_mma.cuh"

namespace pa {

cudaError_t rows_window_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  if (l.head_dim == 128)
    return l.fp8 ? rows_tiles<128, kKvE4m3, kFormWindow>(p, l, tk, tv) : rows_tiles<128, kKvBf16, kFormWindow>(p, l, tk, tv);
  if (l.head_dim == 64)
    return l.fp8 ? rows_tiles<64, kKvE4m3, kFormWindow>(p, l, tk, tv) : rows_tiles<64, kKvBf16, kFormWindow>(p, l, tk, tv);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
