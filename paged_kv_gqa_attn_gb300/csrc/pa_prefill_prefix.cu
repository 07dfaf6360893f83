// The tile kernel over a prefix that the sequences of a group share.
#include "pa_prefill.cuh"

namespace pa {

int prefix_tile_tokens(int group) { return PfTraits<128>::kRows / group; }

int prefix_tiles(int num_seqs, int q_len, int group, int num_groups) {
  const int tt = prefix_tile_tokens(group);
  return (num_seqs * q_len + tt - 1) / tt + num_groups - 1;
}

cudaError_t launch_prefix(const AttnParams& p, const Launch& l, const CUtensorMap& tk, const CUtensorMap& tv) {
  return split_any<kFormPrefix>(p, l, tk, tv);
}

}  // namespace pa
