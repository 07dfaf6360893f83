"""Kernels launched as programmatic dependents: some CTA of each waits for the grid it depends on whatever the
data are.  A grid whose CTAs all returned before such a wait could end, and let the next work on the stream begin,
while the kernel before it still writes.  Read from the sources; no GPU."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_gqa_attn_gb300", "csrc")
WAIT = "griddepcontrol.wait"


def _body(text, name):
    """The braces of the __global__ function `name`."""
    at = re.search(r"__global__[^;{]*\b%s\b" % name, text).start()
    start = text.index("{", text.index(")", text.index(name + "(", at)))
    depth, i = 1, start + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return re.sub(r"//[^\n]*", "", text[start:i])


def _all_sources():
    return {f: open(os.path.join(CSRC, f), encoding="utf-8").read() for f in sorted(os.listdir(CSRC))}


def test_the_list_of_dependents_is_whole():
    launched = set()
    for text in _all_sources().values():
        if "launch_pdl(" in text or "ProgrammaticStreamSerialization" in text:
            launched |= {m for m in re.findall(r"\b(\w+_kernel)<", text) if WAIT in _with_wait(m)}
    assert launched == {"merge_kernel", "verify_merge_kernel", "verify_tc_kernel", "accept_pick_kernel", "prefill_tc_kernel"}


def _with_wait(name):
    for text in _all_sources().values():
        if re.search(r"__global__[^;{]*\b%s\b" % name, text):
            return _body(text, name)
    return ""


def test_what_a_dependent_reads_may_not_move_above_its_wait():
    # loads through a const __restrict__ pointer count as reads of memory that never changes
    for f, text in _all_sources().items():
        for head in re.findall(r"__global__[^{;]*\{", text):
            name = re.search(r"(\w+_kernel)\(", head)
            if name and WAIT in _with_wait(name.group(1)):
                assert "__restrict__" not in head, (f, name.group(1))


@pytest.mark.parametrize("name", ["merge_kernel", "verify_merge_kernel", "accept_pick_kernel", "prefill_tc_kernel"])
def test_no_cta_0_returns_before_it_waits(name):
    body = _with_wait(name)
    before = body[: body.index("return;")]
    assert WAIT in before, name
    # unconditional (but for what the launch is), or for CTA 0 whatever the data, or on the branch that returns
    line = before[: before.index(WAIT)].rstrip().splitlines()[-1].strip()
    assert line.startswith("asm volatile") or "blockIdx.x == 0" in line, line
