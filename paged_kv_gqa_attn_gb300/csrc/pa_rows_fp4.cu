// A few rows per kv head over 4-bit caches: decode and verify, with and without a window.
#include "pa_rows_mma.cuh"

namespace pa {

cudaError_t rows_fp4_form(const AttnParams& p, const Launch& l) {
  const CUtensorMap none = {};  // 4-bit pages move as 16-byte cp.async pieces
  const bool win = p.window > 0;
  if (l.head_dim == 128)
    return win ? rows_tiles<128, kKvFp4, true>(p, l, none, none) : rows_tiles<128, kKvFp4, false>(p, l, none, none);
  if (l.head_dim == 64)
    return win ? rows_tiles<64, kKvFp4, true>(p, l, none, none) : rows_tiles<64, kKvFp4, false>(p, l, none, none);
  return cudaErrorInvalidConfiguration;
}

}  // namespace pa
