// A few rows per kv head that keep their scores for the tokens' weights, every cache type.
#include "pa_rows_mma.cuh"

namespace pa {

cudaError_t rows_scores_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return l.join ? rows_any<kFormScores, true>(p, l, tk, tv) : rows_any<kFormScores>(p, l, tk, tv);
}

}  // namespace pa
