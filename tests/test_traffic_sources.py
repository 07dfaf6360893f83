"""A recorded traffic figure is valid while its kernel's sources are unchanged: the lists of them hold every file
that the kernels' translation units include."""

import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "paged_kv_gqa_attn_gb300", "csrc")


def _closure(files):
    todo, seen = list(files), set()
    while todo:
        f = todo.pop()
        if f in seen or not os.path.exists(os.path.join(CSRC, f)):
            continue
        seen.add(f)
        todo += re.findall(r'^#include "([^"]+)"', open(os.path.join(CSRC, f), encoding="utf-8").read(), flags=re.M)
    return seen


@pytest.mark.parametrize("op", sorted(bench.KERNEL_SOURCES))
def test_every_included_file_is_listed(op):
    listed = set(bench.KERNEL_SOURCES[op])
    assert _closure(listed) == listed
