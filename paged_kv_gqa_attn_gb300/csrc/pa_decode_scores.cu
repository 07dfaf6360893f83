// Decode that keeps its scores for the tokens' weights.
#include "pa_decode_mma.cuh"

namespace pa {

cudaError_t decode_scores_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return decode_any<kFormScores>(p, l, tk, tv);
}

}  // namespace pa
