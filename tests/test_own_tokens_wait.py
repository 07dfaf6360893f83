"""The kernels over own tokens run beside the grid over the prefixes, and the merge behind them reads what both leave: the last
thing that their first CTA does is to wait for that grid.  Read from the sources as the product library compiles them (without
the instrumented variant's parts), and shown to notice a wait that is gone.  Host code only."""

import re

import pytest

from test_dependent_launches import _all_sources, _body
from test_sparse_operator_checks import BESIDE

WAIT_LINE = "if constexpr (OWN) after_prefixes();"


def _product(text):
    """The text without what only -DPA_TIMELINE compiles."""
    out, depth = [], 0
    for line in text.splitlines():
        word = line.strip()
        if depth:
            depth += word.startswith("#if") - word.startswith("#endif")
            assert not (depth == 1 and word.startswith("#el")), "a block with an other side is not cut"
        elif word.startswith("#ifdef PA_TIMELINE"):
            depth = 1
        else:
            out.append(line)
    assert depth == 0
    return "\n".join(out)


def _last_statement(text, kernel):
    lines = [s.strip() for s in _body(_product(text), kernel).splitlines()]
    lines = [s for s in lines if s and not s.startswith("//")]
    while lines and set(lines[-1]) <= {"}"}:
        lines.pop()
    return lines[-1]


def _source(kernel):
    return next(t for t in _all_sources().values() if re.search(r"__global__[^;{]*\b%s\(" % kernel, t))


@pytest.mark.parametrize("kernel", sorted(BESIDE))
def test_the_wait_is_the_last_statement(kernel):
    assert _last_statement(_source(kernel), kernel) == WAIT_LINE


@pytest.mark.parametrize("kernel", sorted(BESIDE))
def test_a_wait_that_is_gone_is_noticed(kernel):
    head, tail = _source(kernel).rsplit(WAIT_LINE, 1)
    assert _last_statement(head + tail, kernel) != WAIT_LINE
