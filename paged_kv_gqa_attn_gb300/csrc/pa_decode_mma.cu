// Decode over every token and over a window of them, and the choice between the decode kernel's forms.
#include "pa_decode_mma.cuh"

namespace pa {

cudaError_t launch_decode_mma(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  switch (l.form) {
    case kFormAll: return decode_any<kFormAll>(p, l, tk, tv);
    case kFormWindow: return decode_any<kFormWindow>(p, l, tk, tv);
    case kFormBlocks: return decode_blocks_form(p, l, tk, tv);
    case kFormOwn: return decode_own_form(p, l, tk, tv);
    case kFormScores: return decode_scores_form(p, l, tk, tv);
    default: return cudaErrorInvalidConfiguration;
  }
}

}  // namespace pa
