"""The prefill work list's packing (csrc/pa_work_item.h) over everything that the host admits.  Host code."""

import os
import shutil
import subprocess

import pytest

import paged_kv_gqa_attn_gb300 as pa

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_attn_gb300", "csrc")
FAKE = 1 << 20  # a 16-byte aligned non-null address that is never dereferenced

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "pa_work_item.h"
int main() {
  const int seqs[] = {0, 1, 4095, 32767, 32768, pa::kWorkSeqs - 1};
  long bad = 0;
  for (int s : seqs)
    for (int t = 0; t < pa::kWorkTiles; ++t) {
      const int32_t item = pa::work_item(s, t);
      bad += pa::work_seq(item) != s || pa::work_tile(item) != t;
    }
  for (int s = 0; s < pa::kWorkSeqs; ++s)
    for (int t : {0, 32767, 32768, pa::kWorkTiles - 1}) {
      const int32_t item = pa::work_item(s, t);
      bad += pa::work_seq(item) != s || pa::work_tile(item) != t;
    }
  std::printf("%ld %d %d", bad, pa::kWorkSeqs, pa::kWorkTiles);
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_admitted_pair_survives_its_word(tmp_path):
    src, exe = tmp_path / "item.cc", tmp_path / "item"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=120)
    bad, seqs, tiles = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True,
                                               timeout=120).stdout.split())
    assert bad == 0
    # both ends of the list pack and unpack with it
    planner = open(os.path.join(CSRC, "pa_prefill.cu"), encoding="utf-8").read()
    kernel = open(os.path.join(CSRC, "pa_prefill.cuh"), encoding="utf-8").read()
    assert "= work_item(" in planner and "work_seq(" in kernel and "work_tile(" in kernel
    assert "<< 16)" not in planner and "tiles[1 + rank] " not in kernel
    # the host's limits are the words': a group of 8 has 16 new tokens a tile (no rows: no call reaches a GPU)
    fn = pa.load_library().paged_attn_prefill
    for n_seqs, max_q, status in ((seqs, 1, pa.PA_OK), (seqs + 1, 1, pa.PA_ERR_UNSUPPORTED),
                                  (1, tiles * 16, pa.PA_OK), (1, tiles * 16 + 1, pa.PA_ERR_UNSUPPORTED)):
        assert fn(*[FAKE] * 6, n_seqs, 0, max_q, 4, 8, 64, 8, 1, 64, 16, 0.1, 0, None, None, FAKE, None) == status
