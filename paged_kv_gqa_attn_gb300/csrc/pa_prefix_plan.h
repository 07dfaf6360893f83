// How shared prefixes are split into partitions.  Host code without CUDA, so that a test can run it.
#pragma once

#include <math.h>
#include <stdint.h>

namespace pa {

struct PrefixSplit {
  int pages, parts;  // of a partition (whole 64-token steps); partitions of the longest prefix
};

// What the prefixes' grid has to do, in (tile of rows, kv head) pairs over the longest prefix, as far as the host knows.
// Tiles: as many as full groups would take, one a group at least, and half of what every group but one may add, a tile
// part full.  Lengths: one group has the longest, the others five eighths of it on average.
inline double prefix_units(int num_seqs, int q_len, int tokens_of_a_tile, int num_groups, int num_kv_heads) {
  const int64_t full = ((int64_t)num_seqs * q_len + tokens_of_a_tile - 1) / tokens_of_a_tile;
  const int64_t least = full > num_groups ? full : num_groups;
  return 0.5 * (double)(least + full + num_groups - 1) * num_kv_heads * (5. * num_groups + 3.) / (8. * num_groups);
}

// The split of `units` such pairs over a longest prefix of `pages` pages, beside `own` pages of own tokens.  In pages of a
// tile's work, n partitions of P pages cost about
//   sqrt((waves (P + 16))^2 + ((units (pages + 16 n) + 2 own) / slots)^2) + n:
// the longest chain of a slot (two CTAs an SM; 16 a CTA's start and end; a quarter of the way from whole waves to CTAs
// that fill up each other's, as the groups' lengths are not known here), all of the work over all slots, and the merge.
// The least of up to `most` partitions is taken.  Measured over the splits of 704 shapes (1 to 12 groups of equal and
// unequal lengths, 4 to 256 sequences, prefixes of 256 to 32768 tokens, own tokens from 16 to 2048, decode and verify
// rows, 9 head layouts, each cache type, inputs cold): 5.2 % above the best split on average; one group 4.0, equal groups
// 6.4, unequal ones 4.8 %, a tenth of each more than 12, 19 and 15 %.  12 to 20 in the place of 16, none to half of the
// way, 2 to 3 for own's factor and 0.6 to 0.7 for five eighths stay within 1 % of that.
inline PrefixSplit plan_prefix(double units, int64_t pages, int64_t own, int slots, int most, int forced) {
  if (pages < 1) pages = 1;
  const double kFixed = 16.;
  PrefixSplit best = {0, 0};
  double least = 0.;
  for (int64_t n = forced > 0 ? forced : 1; n <= (forced > 0 ? forced : most); ++n) {
    const int64_t P = n < pages ? n : pages;
    const int64_t per = ((pages + P - 1) / P + 3) / 4 * 4;
    const int parts = (int)((pages + per - 1) / per);
    const double x = units * parts / slots, all = (units * (pages + kFixed * parts) + 2. * own) / slots;
    if (best.parts > 0 && all + parts >= least) break;  // (this much only grows with n)
    const double fill = 0.75 * ceil(x) + 0.25 * (x + 0.5), chain = (fill > 1. ? fill : 1.) * (per + kFixed);
    const double t = sqrt(chain * chain + all * all) + parts;
    if (best.parts == 0 || t < least) {
      least = t;
      best = {(int)per, parts};
    }
    if (P == pages) break;
  }
  return best;
}

}  // namespace pa
