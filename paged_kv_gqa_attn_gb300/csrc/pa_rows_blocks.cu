// A few rows per kv head over the blocks that a list names, every cache type.
#include "pa_rows_mma.cuh"

namespace pa {

cudaError_t rows_blocks_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return l.join ? rows_any<kFormBlocks, true>(p, l, tk, tv) : rows_any<kFormBlocks>(p, l, tk, tv);
}

}  // namespace pa
