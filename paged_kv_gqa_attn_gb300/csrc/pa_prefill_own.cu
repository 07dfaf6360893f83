// The tile kernel over what lies behind a shared prefix: verify of more rows than the rows kernel takes.
#include "pa_prefill.cuh"

namespace pa {

cudaError_t tiles_own_form(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return split_any<kFormOwn>(p, l, tk, tv);
}

}  // namespace pa
