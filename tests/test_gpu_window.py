"""Sliding-window attention with sinks on the GPU against the plain fp64 form: decode, verify and
prefill over every cache type, windows and sinks that end inside a block, cover everything or leave
one token, blocks out of sight given back (their table entries would be flagged if read), NaN in every
token out of sight, empty contexts, forced splits, streams, graphs and refusals."""

import numpy as np
import pytest
import torch

import attn_cases as A
from oracle import plain
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

KV = ["bf16", "e4m3", "fp4"]
LENS = [1, 5, 16, 17, 40, 130, 333, 700, 64]


def _run(c, form, expect=None, **more):
    got = A.call(c, form, **more)
    assert pa.check_device_errors() == (pa.PA_OK if expect is None else expect)
    return A.check(c, form, got), got


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (15, 4), (33, 16), (100, 17), (256, 100), (10000, 3),
                                          (64, 10000)])
def test_decode_windows(kv, window, sinks):
    _run(A.make(kv, LENS, [1] * len(LENS), 8, 2, 128, seed=window + sinks, window=window, sinks=sinks), "decode")


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 2, 128), (8, 2, 64), (16, 2, 128), (6, 2, 64), (7, 1, 128), (32, 2, 64),
                                      (40, 8, 128), (64, 1, 128)])
def test_decode_head_groups(kv, hq, hkv, d):
    _run(A.make(kv, LENS, [1] * len(LENS), hq, hkv, d, seed=hq, window=50, sinks=4), "decode")


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("parts", [1, 2, 5])
@pytest.mark.parametrize("form", ["decode", "verify"])
def test_forced_splits(kv, parts, form):
    r = 1 if form == "decode" else 4
    pa.set_max_partitions(parts)
    try:
        _run(A.make(kv, [700, 20, 333], [r] * 3, 8, 2, 128, seed=parts, window=300, sinks=20), form)
    finally:
        pa.set_max_partitions(0)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r", [1, 2, 5, 16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (40, 0), (64, 4), (129, 70), (5000, 1)])
def test_verify_windows(kv, r, window, sinks):
    lens = [max(n, r) for n in LENS]
    _run(A.make(kv, lens, [r] * len(lens), 8, 2, 128, seed=r + window, window=window, sinks=sinks), "verify")


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d,r", [(4, 4, 64, 9), (24, 8, 64, 5), (16, 2, 128, 16), (5, 1, 64, 3)])
def test_verify_head_groups(kv, hq, hkv, d, r):
    lens = [max(n, r) for n in LENS]
    _run(A.make(kv, lens, [r] * len(lens), hq, hkv, d, seed=hq, window=37, sinks=5), "verify")


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (64, 4), (100, 0), (200, 65), (4096, 4)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (2, 2, 128)])
def test_prefill_windows(kv, window, sinks, hq, hkv, d):
    lens, rows = [1, 37, 500, 333, 900, 129, 64], [1, 37, 5, 200, 33, 128, 1]
    _run(A.make(kv, lens, rows, hq, hkv, d, seed=window + hq, window=window, sinks=sinks), "prefill")


@pytest.mark.parametrize("kv", KV)
def test_a_window_over_everything_is_no_window(kv):
    for form, rows in (("decode", [1] * 4), ("verify", [9] * 4), ("prefill", [20, 1, 9, 64])):
        c = A.make(kv, [20, 77, 300, 64], rows, 16, 2, 128, seed=3, junk=False)
        want = A.call(c, form)
        got = A.call({**c, "window": 300, "sinks": 0}, form)
        A.check(c, form, want)
        A.check(c, form, got)
        assert pa.check_device_errors() == pa.PA_OK


@pytest.mark.parametrize("form,r", [("decode", 1), ("verify", 3)])
def test_contexts_shorter_than_the_rows(form, r):
    c = A.make("bf16", [40, 40, 40], [r] * 3, 8, 2, 64, seed=5, window=10, sinks=2)
    c["lens"] = [40, 0, r - 1 if r > 1 else 0]
    got = A.call({**c, "table": c["table"].clone()}, form)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    one = {**c, "lens": [40], "rows": [r], "table": c["table"][:1], "q": c["q"][:r]}
    A.check(one, form, got[:r])
    assert not got[r: 2 * r].any()
    assert not got[2 * r].any()  # the first row of the last sequence sees nothing


def test_bad_blocks_in_sight_are_flagged_and_left_out():
    for form, r in (("decode", 1), ("verify", 4)):
        c = A.make("bf16", [100, 100], [r, r], 8, 2, 128, seed=6, window=40, sinks=3)
        c["table"][1, 5] = -3
        _run(c, form, expect=pa.PA_ERR_DEVICE_BOUNDS)


def test_a_row_tile_deep_in_a_long_context():
    # sinks and window far apart, sequences of one step and of many, a bound far above the lengths
    lens, rows = [6000, 4097, 70], [130, 1, 70]
    for kv in KV:
        c = A.make(kv, lens, rows, 8, 1, 128, seed=7, window=1000, sinks=4)
        _run(c, "prefill", max_q_len=500, max_context_len=6000)


def test_streams_and_graphs():
    cases = {"decode": A.make("bf16", [300, 77], [1, 1], 8, 2, 128, seed=8, window=64, sinks=4),
             "verify": A.make("e4m3", [300, 77], [5, 5], 8, 2, 128, seed=9, window=64, sinks=4),
             "prefill": A.make("fp4", [300, 77], [50, 1], 8, 2, 128, seed=10, window=64, sinks=4)}
    for form, c in cases.items():
        dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
        want = A.call(c, form)
        lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
        starts = torch.tensor(np.concatenate(([0], np.cumsum(c["rows"]))), dtype=torch.int32, device="cuda")
        kw = {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"], "window": 64, "sinks": 4}

        def one(**more):
            if form == "prefill":
                return pa.prefill(dev["q"], dev["k"], dev["v"], dev["table"], lens, starts, c["scale"], max_q_len=50, **kw,
                                  **more)
            q = dev["q"].view(2, -1, 8, 128)
            return (pa.decode if form == "decode" else pa.verify)(q, dev["k"], dev["v"], dev["table"], lens, c["scale"],
                                                                  **kw, **more).flatten(0, 1)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        side = one(stream=s)
        s.synchronize()
        assert torch.equal(want, side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = one()
        out.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert pa.check_device_errors() == pa.PA_OK


def test_refusals():
    c = A.make("bf16", [40], [1], 8, 2, 64, seed=11, window=8, sinks=0)
    for bad in ({"window": 0}, {"window": -1}, {"window": 8, "sinks": -1}):
        with pytest.raises(pa.PagedAttnError):
            A.call({**c, **bad}, "decode")
    with pytest.raises(ValueError):
        A.call({**c, "window": None}, "decode", sinks=4)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    with pytest.raises(ValueError):
        pa.tree_verify(dev["q"][None], dev["k"], dev["v"], dev["table"], torch.tensor([40], dtype=torch.int32).cuda(),
                       torch.ones(1, 1, dtype=torch.int32).cuda(), 0.1, window=8)
