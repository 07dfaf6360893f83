"""Shared prefixes at their bound on the GPU: what is flagged is a group whose whole blocks pass it, not the part of a block behind
them, which each row reads for itself, and not a group of no sequences.  Results against fp64 in every case."""

import pytest
import torch

from form_cases import causal, check
from test_gpu_shared_prefix import make, run
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

KV = ["bf16", "e4m3", "fp4"]


def _hold(c, flagged, **kw):
    check(c, run(c, pa.PA_ERR_DEVICE_BOUNDS if flagged else pa.PA_OK, **kw), causal(c["lens"], c["rows"][0]), tiles=True)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r", [1, 4, 12])
def test_the_last_part_of_a_block_passes_the_bound(kv, r):
    # 64 whole tokens of 79 are shared; the longest context is shorter than 79, or the bound lies between
    c = make(kv, [(3, 79)], [r, r + 2], r, 8, 2, 64, seed=r)
    assert max(c["lens"]) < 79
    _hold(c, False, max_context_len=max(c["lens"]))
    _hold(c, False, max_prefix_len=79, max_context_len=max(c["lens"]))
    for bound in (64, 70, 78):
        _hold(c, False, max_prefix_len=bound)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("many", [1, 40])
def test_a_group_of_no_sequences_has_any_prefix(kv, many):
    c = make(kv, [(2, 48), (3, 32)], [20, 33], 1, 8, 2, 64, seed=many)
    starts, prefixes = c["starts"], c["prefixes"]
    c["starts"], c["prefixes"] = [0] * many + [0, 2] + [2] * many + [5], [10 ** 6] * many + [48] + [2 ** 31 - 1] * many + [32]
    assert len(c["starts"]) == len(c["prefixes"]) + 1
    _hold(c, False)
    _hold(c, False, max_prefix_len=48, max_own_len=40, max_context_len=max(c["lens"]))
    c["starts"], c["prefixes"] = starts, prefixes
    _hold(c, False)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("prefix,bound", [(80, 79), (80, 64), (128, 17), (96, 95)])
def test_whole_blocks_past_the_bound_are_flagged(kv, prefix, bound):
    c = make(kv, [(3, prefix)], [20, 30], 1, 8, 2, 64, seed=bound)
    c["call_table"] = c["table"]  # what is cut off is looked up in each row
    _hold(c, True, max_prefix_len=bound)
    _hold(c, False, max_prefix_len=prefix)


def test_contexts_past_their_bound_with_prefixes_past_it_are_flagged():
    c = make("bf16", [(2, 128)], [20, 30], 1, 8, 2, 64, seed=1)
    c["call_table"] = c["table"]
    got = run(c, pa.PA_ERR_DEVICE_BOUNDS, max_context_len=100)
    cut = dict(c, lens=[100, 100])
    check(cut, got, causal(cut["lens"], 1), tiles=True)
    assert torch.isfinite(got).all()
