"""Attention behind shared prefixes has the precision of ordinary decode, on the GPU against fp64: prefixes whose softmax has few
heavy tokens, so that a weight's rounding shows, and rows outside every prefix, which only the own tokens' kernels compute.

The bound is form_cases.check's for the decode and rows kernels (tiles=False): the output's rounding to bf16 (2^-8 |out|), bf16
weights as a pair or f16 ones (2^-14, 2^-11 of sum p |v|), twice the error of a score.  What joins the partials adds less than
its room: a log2-sum-exp below 32 in fp32 is off by 2^-20, two exponentials by 2^-22 each, all times ln 2: 2^-19 of the spread.
E4M3 caches of head_dim 128 take the prefix's scores from the query in two E4M3 terms, each off by at most 2^-4 of what it
stands for: 2^-8 |q| in all, times 2 for the exponential's own rounding as in the rest of the bound."""

import numpy as np
import pytest
import torch

import attn_cases as A
from form_cases import causal, check, on_gpu
from test_gpu_shared_prefix import make, run
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

OWN = [1, 3, 17, 2, 40, 16]


def _peaked(c, mul):
    """The case with its scores a few times as large: few tokens have most of a row's weight."""
    c["scale"] *= mul
    return c


LAYOUTS = [(8, 2, 128), (8, 8, 64), (16, 2, 64), (4, 2, 128), (6, 2, 128), (16, 1, 64)]


# (E4M3 scores at head_dim 128 have their own bound, below)
@pytest.mark.parametrize("kv,hq,hkv,d", [(kv, *h) for kv in ("bf16", "fp4", "e4m3") for h in LAYOUTS if kv != "e4m3" or h[2] != 128])
@pytest.mark.parametrize("groups", [[(5, 400)], [(2, 64), (3, 1000), (4, 160)], [(33, 208)]])
def test_decode_behind_a_prefix(kv, groups, hq, hkv, d):
    c = _peaked(make(kv, groups, OWN, 1, hq, hkv, d, seed=hq + d), 3)
    check(c, run(c), causal(c["lens"], 1), tiles=False)


@pytest.mark.parametrize("kv,r,hq,hkv,d", [
    (kv, *shape) for kv in ("bf16", "fp4", "e4m3") for shape in [(2, 8, 2, 128), (5, 8, 2, 64), (9, 16, 2, 128), (7, 8, 1, 64),
                                                                 (16, 8, 1, 64), (1, 32, 1, 128), (1, 64, 2, 64)]
    if kv != "e4m3" or shape[3] != 128])
def test_rows_behind_a_prefix(kv, r, hq, hkv, d):
    # verify, and decode of large groups: 8 to 128 rows a kv head, own tokens on the rows and on the tile kernel
    c = _peaked(make(kv, [(3, 64), (1, 333), (4, 0), (2, 400)], [1, 3, 70, 16, 200], r, hq, hkv, d, seed=r + hq), 3)
    check(c, run(c), causal(c["lens"], r), tiles=False)


@pytest.mark.parametrize("parts", [1, 3, 100])
def test_decode_behind_a_split_prefix(parts):
    pa.set_max_partitions(parts)
    try:
        c = _peaked(make("bf16", [(3, 700), (2, 333)], OWN, 1, 32, 8, 128, seed=parts), 3)
        check(c, run(c), causal(c["lens"], 1), tiles=False)
    finally:
        pa.set_max_partitions(0)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (16, 2)])
def test_e4m3_scores_of_a_prefix(hq, hkv):
    """head_dim 128: the wider bound of a score holds, and rows without a prefix stay within the tight one."""
    c = make("e4m3", [(3, 400), (3, 0), (2, 160)], OWN, 1, hq, hkv, 128, seed=hq)
    got = run(c)
    check(c, got, causal(c["lens"], 1), tiles=True)
    alone = [b for b in range(8) if 3 <= b < 6]
    few = dict(c, lens=[c["lens"][b] for b in alone], rows=[1] * 3, table=c["table"][alone], q=c["q"][alone])
    check(few, got[alone], causal(few["lens"], 1), tiles=False)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (16, 2, 128), (6, 2, 64), (15, 1, 128)])
def test_rows_outside_every_prefix(kv, hq, hkv, d):
    # prefixes below a block, of nothing, and sequences in no group: the decode and rows kernels alone
    lens = [1, 16, 17, 130, 333, 700, 64, 48]
    c = _peaked(A.make(kv, lens, [1] * 8, hq, hkv, d, seed=hq), 3)
    c["starts"], c["prefixes"], c["call_table"] = [1, 3, 5, 6], [15, 0, -3], c["table"]
    check(c, run(c), causal(lens, 1), tiles=False)
    c["starts"], c["prefixes"] = [8], []
    check(c, run(c), causal(lens, 1), tiles=False)


def test_the_error_is_that_of_ordinary_decode():
    """Root mean square error against fp64, of the whole context by decode and behind its prefix.  Both round nearly the same
    numbers to bf16, 2^-8 of each at most, and differ by pairs of 2^-14 before that: within a tenth."""
    c = _peaked(make("bf16", [(16, 1024)], [5, 9, 30], 1, 32, 8, 128, seed=9), 3)
    ref = check(c, run(c), causal(c["lens"], 1), tiles=False)[0]
    (q, k, v, _, lens), _ = on_gpu(c)
    plain = pa.decode(q, k, v, c["table"].cuda(), lens, c["scale"])
    assert pa.check_device_errors() == pa.PA_OK
    off = [float(np.sqrt(np.mean((t.float().cpu().double().numpy().reshape(ref.shape) - ref) ** 2))) for t in (run(c), plain)]
    assert off[0] <= 1.1 * off[1], off
    assert torch.equal(run(c), run(c))
