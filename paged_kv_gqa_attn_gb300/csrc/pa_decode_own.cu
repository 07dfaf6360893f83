// Decode behind a prefix that a group of sequences shares.
#include "pa_decode_mma.cuh"

namespace pa {

cudaError_t decode_own_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return decode_any<kFormOwn>(p, l, tk, tv);
}

}  // namespace pa
