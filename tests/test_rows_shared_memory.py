"""Shared memory of the rows kernel: only launches whose CTAs join their partials make room for them.  The compiler checks
csrc/pa_rows_mma.cuh itself; no GPU."""

import os
import subprocess

from paged_kv_gqa_attn_gb300 import build

CHECKS = r"""
#include "pa_rows_mma.cuh"

namespace pa {
namespace {

template <int D, int NT, int KV>
constexpr bool rows_hold() {
  using Alone = RowsTraits<D, NT, KV, false>;
  using Joined = RowsTraits<D, NT, KV, true>;
  // the warps' page stages, and in the same place in the end their outputs, maxima and sums
  constexpr int merge = 4 * 8 * NT * (D + 2) * 4;
  constexpr int data = Alone::kStageRegion > merge ? Alone::kStageRegion : merge;
  // what a cluster joins: normalised rows, their masses (two floats), the rows' totals (two)
  constexpr int join = 8 * NT * (D + 4) * 4;
  constexpr int joined = Alone::kStageRegion > merge + join ? Alone::kStageRegion : merge + join;
  static_assert(Alone::kDataRegion == data, "no room for partials that nobody joins");
  static_assert(Joined::kDataRegion == joined, "room for the partials to join");
  static_assert(Joined::kSmem - Alone::kSmem == joined - data, "nothing else differs");
  return true;
}

template <int D, int KV>
constexpr bool all_rows() {
  return rows_hold<D, 1, KV>() && rows_hold<D, 2, KV>() && rows_hold<D, 3, KV>() && rows_hold<D, 4, KV>();
}

static_assert(all_rows<64, kKvBf16>() && all_rows<64, kKvE4m3>() && all_rows<64, kKvFp4>(), "");
static_assert(all_rows<128, kKvBf16>() && all_rows<128, kKvE4m3>() && all_rows<128, kKvFp4>(), "");

}  // namespace
}  // namespace pa
"""


def test_only_joined_launches_make_room_for_partials(tmp_path):
    src = tmp_path / "rows.cu"
    src.write_text(CHECKS)
    cmd = [build.nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-c", str(src), "-o", os.fspath(tmp_path / "rows.o")]
    done = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert done.returncode == 0, done.stdout
