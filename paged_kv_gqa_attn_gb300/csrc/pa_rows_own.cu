// A few rows per kv head behind a prefix that a group of sequences shares, every cache type.
#include "pa_rows_mma.cuh"

namespace pa {

cudaError_t rows_own_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return rows_any<kFormOwn>(p, l, tk, tv);
}

}  // namespace pa
