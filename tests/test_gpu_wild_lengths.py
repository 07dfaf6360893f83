"""Context lengths and row offsets of any 32-bit value, as uninitialised memory holds them: the affected sequences
are skipped or zeroed and flagged, the others are served, nothing outside is read or written."""

import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

LOW = -(1 << 31)
WILD = [LOW, LOW + 1, LOW + 3, LOW + 40, -(1 << 30), -17, -1]


def _with_wild(c, wild):
    """The case's one sequence in the middle of a batch whose other lengths are wild."""
    n = len(wild)
    table = torch.full((n + 1, c["table"].shape[1]), -1, dtype=torch.int32)
    table[n // 2] = c["table"][0]
    lens = wild[: n // 2] + [c["lens"][0]] + wild[n // 2:]
    return table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), n // 2


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("window", [None, 40])
@pytest.mark.parametrize("form,hq,r", [("decode", 8, 1), ("decode", 6, 1), ("verify", 8, 5), ("verify", 16, 9), ("prefill", 8, 30)])
def test_attention(form, hq, r, window, kv):
    c = A.make(kv, [200], [r], hq, 2, 128, seed=r + hq, window=window, sinks=4 if window else 0)
    table, lens, at = _with_wild(c, WILD)
    B = len(WILD) + 1
    q = torch.randn(B * r, hq, 128, generator=torch.Generator().manual_seed(1)).bfloat16()
    q[at * r: (at + 1) * r] = c["q"]
    q, dev = q.cuda(), {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    out = torch.full_like(q, float("nan"))
    kw = {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"]}
    if window:
        kw |= {"window": window, "sinks": 4}
    if form == "prefill":
        starts = torch.arange(B + 1, dtype=torch.int32, device="cuda") * r
        pa.prefill(q, dev["k"], dev["v"], table, lens, starts, c["scale"], max_q_len=r, out=out, **kw)
    else:
        fn = pa.decode if form == "decode" else pa.verify
        fn(q.view(B, r, hq, 128), dev["k"], dev["v"], table, lens, c["scale"], out=out.view(B, r, hq, 128), **kw)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    A.check(c, form, out[at * r: (at + 1) * r])
    out[at * r: (at + 1) * r] = 0
    assert (out == 0).all()  # rows that see no token


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("n", [1, 20])
def test_append_and_read(kv, n):
    c = A.make(kv, [200], [1], 8, 2, 128, seed=n, junk=False)
    wild = WILD + [(1 << 31) - 1, (1 << 31) - 16, 1 << 20]
    table, lens, at = _with_wild(c, wild)
    B = len(wild) + 1
    dev = {x: (t.cuda() if torch.is_tensor(t) else t) for x, t in c.items()}
    kw = {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"]}
    one = {"table": dev["table"], "lens": torch.tensor([200], dtype=torch.int32, device="cuda")}
    want = pa.read_kv(dev["k"], dev["v"], one["table"], one["lens"], n, **kw)
    assert pa.check_device_errors() == pa.PA_OK
    got = pa.read_kv(dev["k"], dev["v"], table, lens, n, **kw)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    for g, w in zip(got, want):
        assert torch.equal(g[at], w[0])
        g[at] = 0
        assert (g == 0).all()
    new = [torch.randn(B, n, 2, 128, device="cuda").bfloat16() for _ in "kv"]
    caches = [[dev[x].clone() for x in "kv"] for _ in range(2)]
    scales = [[t.clone() if t is not None else None for t in kw.values()] for _ in range(2)]
    pa.append_kv(*(x[at: at + 1].contiguous() for x in new), *caches[0], one["table"], one["lens"],
                 k_scale=scales[0][0], v_scale=scales[0][1])
    assert pa.check_device_errors() == pa.PA_OK
    pa.append_kv(*new, *caches[1], table, lens, k_scale=scales[1][0], v_scale=scales[1][1])
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    for a, b in zip(caches[0] + scales[0], caches[1] + scales[1]):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
@pytest.mark.parametrize("starts", [[0, 30, LOW + 9, LOW + 9], [0, 30, (1 << 31) - 4, LOW + 5], [0, 30, (1 << 31) - 1, (1 << 31) - 1],
                                    [0, 30, -1, 4], [0, 30, 29, 61]])
def test_row_offsets(kv, starts):
    c = A.make(kv, [200], [30], 8, 2, 128, seed=3)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    q = torch.cat((dev["q"], dev["q"]))
    out = torch.full_like(q, 5.0)
    pa.prefill(q, dev["k"], dev["v"], dev["table"].expand(3, -1).contiguous(), torch.full((3,), 200, dtype=torch.int32, device="cuda"),
               torch.tensor(starts, dtype=torch.int32, device="cuda"), c["scale"], max_q_len=60, out=out,
               k_scale=dev["k_scale"], v_scale=dev["v_scale"])
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    A.check(c, "prefill", out[:30])
    assert (out[30:] == 5).all()
