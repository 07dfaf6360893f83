"""The window, 4-bit and norm-and-rotation operators where they could go wrong together: drawn shapes, caches
past 4 GiB, two calls at once, captured graphs that share the library's scratch, outputs on side streams."""

import numpy as np
import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def _drawn(seed):
    r = np.random.RandomState(seed)
    form = ["decode", "verify", "prefill"][seed % 3]
    kv = ["bf16", "e4m3", "fp4"][r.randint(3)]
    d = [64, 128][r.randint(2)]
    hkv = [1, 2, 3, 8][r.randint(4)]
    group = [1, 2, 4, 8][r.randint(4)] if form == "prefill" else [1, 2, 3, 4, 5, 7, 8][r.randint(7)]
    B = r.randint(1, 9)
    if form == "prefill":
        rows = r.randint(1, [2, 40, 300][r.randint(3)] + 1, B).tolist()
    else:
        rows = [1 if form == "decode" else int(r.randint(1, 17))] * B
    lens = [n + int(r.randint(0, [1, 30, 500, 2000][r.randint(4)] + 1)) for n in rows]
    window = None if kv == "fp4" and r.randint(2) else int(np.exp(r.uniform(0, np.log(2500))))
    sinks = [0, 1, 4, 16, 33, 200][r.randint(6)] if window is not None else 0
    return form, A.make(kv, lens, rows, hkv * group, hkv, d, seed=seed, window=window, sinks=sinks)


@pytest.mark.parametrize("seed", range(60))
def test_drawn_shapes(seed):
    form, c = _drawn(seed)
    if form == "verify" and c["rows"][0] * (c["q"].shape[1] // c["kf"].shape[1]) > 128:
        with pytest.raises(pa.PagedAttnError):
            A.call(c, form)
        return
    got = A.call(c, form)
    assert pa.check_device_errors() == pa.PA_OK
    A.check(c, form, got)


def test_4_bit_blocks_past_4_gib():
    hkv, d, lens = 8, 128, [100, 37, 260]
    nb = (1 << 32) // (hkv * 9 * d) + 64  # blocks: the last lie past byte 2^32
    caches = {n: torch.zeros(nb, hkv, 16, 9 * d // 16, dtype=torch.uint8, device="cuda") for n in "kv"}
    for form, rows in (("decode", [1, 1, 1]), ("verify", [5, 5, 5]), ("prefill", [30, 1, 64])):
        c = A.make("fp4", lens, rows, 32, hkv, d, seed=41)
        want = A.call(c, form)
        far = {**c}
        used = c["k"].shape[0]
        for n in "kv":
            caches[n][nb - used:] = c[n].cuda()
            far[n] = caches[n]
        far["table"] = torch.where(c["table"] == A.BAD_ID, c["table"], c["table"] + (nb - used))
        assert torch.equal(A.call(far, form), want)
    table = far["table"].cuda()
    cl = torch.tensor(lens, dtype=torch.int32).cuda()
    k, v = pa.read_kv(caches["k"], caches["v"], table, cl, 3)
    pa.append_kv(k.neg(), v.neg(), caches["k"], caches["v"], table, cl)
    k2, v2 = pa.read_kv(caches["k"], caches["v"], table, cl, 3)
    assert torch.equal(k2, -k) and torch.equal(v2, -v)
    assert pa.check_device_errors() == pa.PA_OK


def test_two_calls_at_once():
    cases = [("decode", A.make("fp4", [3000, 200], [1, 1], 32, 8, 128, seed=51)),
             ("verify", A.make("fp4", [900, 2000], [5, 5], 32, 8, 128, seed=52, window=700, sinks=4)),
             ("decode", A.make("bf16", [3000, 77], [1, 1], 32, 8, 128, seed=53, window=2000, sinks=4)),
             ("prefill", A.make("fp4", [500, 300], [100, 40], 8, 2, 64, seed=54))]
    dev = [{n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()} for _, c in cases]
    want = [A.call(c, form) for form, c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for (form, _), c, s in zip(cases, dev, streams):
            with torch.cuda.stream(s):
                got.append(A.call(c, form))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert pa.check_device_errors() == pa.PA_OK


def test_two_graphs_replayed_in_turn_and_at_once():
    graphs, outs, want = [], [], []
    for i, (form, kv) in enumerate((("decode", "fp4"), ("decode", "bf16"), ("verify", "fp4"))):
        r = 1 if form == "decode" else 4
        c = A.make(kv, [2500, 600], [r, r], 16, 4, 128, seed=61 + i, window=None if kv == "fp4" else 1500)
        dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
        lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
        kw = {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"]}
        if c["window"]:
            kw["window"] = c["window"]
        q = dev["q"].view(2, r, 16, 128)
        fn = pa.decode if form == "decode" else pa.verify

        def one():
            return fn(q, dev["k"], dev["v"], dev["table"], lens, c["scale"], **kw)

        want.append(one())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(one())
        graphs.append((g, dev, lens, q))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_outputs_made_on_a_side_stream_outlive_their_caller():
    # an output dropped while a side stream still writes it must not be handed out again at once
    c = A.make("fp4", [4000] * 4, [1] * 4, 32, 8, 128, seed=71)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    q = dev["q"].view(4, 1, 32, 128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        pa.decode(q, dev["k"], dev["v"], dev["table"], lens, c["scale"], k_scale=dev["k_scale"], v_scale=dev["v_scale"],
                  stream=s)
        fresh = torch.full_like(q, 7.0)
        torch.cuda.synchronize()
        assert (fresh == 7).all()


def test_prefill_leaves_rows_behind_the_last_sequence():
    c = A.make("fp4", [50, 20], [10, 3], 8, 2, 128, seed=81, window=30, sinks=1)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    q = torch.cat((dev["q"], dev["q"][:4]))
    out = torch.full_like(q, 5.0)
    pa.prefill(q, dev["k"], dev["v"], dev["table"], torch.tensor([50, 20], dtype=torch.int32).cuda(),
               torch.tensor([0, 10, 13], dtype=torch.int32).cuda(), c["scale"], window=30, sinks=1, out=out,
               k_scale=dev["k_scale"], v_scale=dev["v_scale"])
    assert (out[13:] == 5).all()
    A.check(c, "prefill", out[:13])
