// Decode over the blocks that a list names.
#include "pa_decode_mma.cuh"

namespace pa {

cudaError_t decode_blocks_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return l.join ? decode_any<kFormBlocks, true>(p, l, tk, tv) : decode_any<kFormBlocks>(p, l, tk, tv);
}

}  // namespace pa
