// Decode that keeps its scores for the tokens' weights.
#include "pa_decode_mma.cuh"

namespace pa {

cudaError_t decode_scores_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return l.join ? decode_any<kFormScores, true>(p, l, tk, tv) : decode_any<kFormScores>(p, l, tk, tv);
}

}  // namespace pa
