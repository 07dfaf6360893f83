"""The split of shared prefixes (csrc/pa_prefix_plan.h): it covers the prefix, and follows what the work is instead of how many
groups it is called.  Host code only."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_attn_gb300", "csrc")
MAIN = r"""
#include <cstdio>
#include "pa_prefix_plan.h"
int main() {
  double units;
  int seqs, q_len, tokens, groups, heads, slots, most, forced;
  long long pages, own;
  while (scanf("%d %d %d %d %d %lld %lld %d %d %d", &seqs, &q_len, &tokens, &groups, &heads, &pages, &own, &slots, &most, &forced) == 10) {
    units = pa::prefix_units(seqs, q_len, tokens, groups, heads);
    const pa::PrefixSplit s = pa::plan_prefix(units, pages, own, slots, most, forced);
    printf("%.17g %d %d\n", units, s.pages, s.parts);
  }
}
"""
SLOTS = 304


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("prefix_split")
    (at / "main.cpp").write_text(MAIN)
    exe = os.fspath(at / "main")
    subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, os.fspath(at / "main.cpp"), "-o", exe],
                   check=True)

    def run(shapes):
        """(seqs, q_len, tokens of a tile, groups, heads, pages, own, slots, most, forced) each -> (units, pages, parts)."""
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        lines = subprocess.run([exe], input=text, stdout=subprocess.PIPE, text=True, check=True).stdout.split("\n")
        return [(float(u), int(p), int(n)) for u, p, n in (s.split() for s in lines if s)]
    return run


def _shape(seqs=64, q_len=1, group=4, groups=1, heads=8, prefix=8192, own=512, forced=0, slots=SLOTS):
    return (seqs, q_len, 128 // group, groups, heads, prefix // 16, seqs * heads * -(-own // 16), slots, 64, forced)


SHAPES = [_shape(s, r, g, n, h, p, o) for s in (1, 5, 64, 300, 65535) for r in (1, 5) for g in (1, 4, 16) for n in (1, 2, 9)
          for h in (1, 8) for p in (16, 64, 80, 2048, 8192, 1 << 20, 1 << 30) for o in (1, 64, 2048)]


def test_whole_steps_that_cover_the_prefix(plan):
    for s, (_, pages, parts) in zip(SHAPES, plan(SHAPES)):
        assert pages % 4 == 0 and 1 <= parts <= 64, s
        assert pages * parts >= s[5] > pages * (parts - 1), s


@pytest.mark.parametrize("forced", [1, 2, 7, 100, 4096])
def test_forced_partitions(plan, forced):
    for s, (_, pages, parts) in zip(SHAPES, plan([s[:9] + (forced,) for s in SHAPES])):
        want = min(forced, s[5])
        per = (-(-s[5] // want) + 3) // 4 * 4
        assert (pages, parts) == (per, -(-s[5] // per)), s


def test_units_lie_between_the_least_and_the_most(plan):
    """Tiles between what full groups take (one a group at least) and a part tile more for every group but one; groups but one
    between five eighths and the whole of the longest prefix."""
    for s, (units, _, _) in zip(SHAPES, plan(SHAPES)):
        full = -(-s[0] * s[1] // s[2])
        share = (1 + 5 / 8 * (s[3] - 1)) / s[3]
        assert units >= share * full * s[4] * (1 - 1e-9), s
        assert s[3] > s[0] or units <= (full + s[3] - 1) * s[4] * (1 + 1e-9), s


def test_a_group_of_nothing_changes_little(plan):
    """An empty group beside a real one counts as a tile a kv head at most, and takes 3/16 of the length: what the split rests
    on is between 13/16 of one group's and, with that tile, 13/16 (1 + 1 / tiles) of it.  It rests on nothing else of them."""
    for seqs in (8, 32, 64, 256, 1000):
        (one, *_), (two, *_) = plan([_shape(seqs), _shape(seqs, groups=2)])
        assert 13 / 16 * one <= two * (1 + 1e-9) and two <= 13 / 16 * (one + 8) * (1 + 1e-9), (seqs, one, two)
    # half the sequences and twice the heads: other numbers, the same units, the same split
    same = plan([(64, 1, 32, 1, 8, 512, 1000, SLOTS, 64, 0), (32, 1, 32, 1, 16, 512, 1000, SLOTS, 64, 0)])
    assert same[0] == same[1]


def test_more_own_tokens_never_take_more_partitions(plan):
    """d cost / d own = 2 / slots * B / sqrt(A^2 + B^2), B the work over all slots and A the longest chain.  Of two splits neither of
    which has both smaller, the one of more partitions has the larger B and the smaller A, so that its cost grows faster."""
    for seqs in (8, 64, 256):
        for prefix in (2048, 8192, 16384):
            parts = [n for _, _, n in plan([(seqs, 1, 32, 1, 8, prefix // 16, own, SLOTS, 64, 0)
                                            for own in (int(100 * 1.01 ** i) for i in range(700))])]
            assert all(b <= a for a, b in zip(parts, parts[1:]))


def test_a_wave_that_is_nearly_full_is_not_passed(plan):
    """One group of 64 sequences, 32 heads, 8192 tokens: 64 pairs, and a fifth partition of each would start a second wave."""
    for own in (64, 1500):
        units, _, parts = plan([_shape(64, heads=32, prefix=8192, own=own)])[0]
        assert units == 64 and 64 * parts <= SLOTS, parts
