"""Attention over the 4-bit cache on the GPU against the plain fp64 form: decode, verify, tree verify
and prefill, every head grouping, both head dims, contexts that end anywhere in a block, forced splits,
extreme queries and scales, junk past the contexts, bad tables, and a step as it is used (norm and
rotation, append, attention)."""

import numpy as np
import pytest
import torch

import attn_cases as A
from oracle import plain
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

LENS = [1, 5, 16, 17, 40, 130, 333, 64]


def _run(c, form, expect=pa.PA_OK, **more):
    got = A.call(c, form, **more)
    assert pa.check_device_errors() == expect
    A.check(c, form, got)
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (8, 2), (16, 2), (6, 2), (5, 1), (7, 1), (32, 2), (64, 1)])
def test_decode_head_groups(hq, hkv, d):
    _run(A.make("fp4", LENS, [1] * len(LENS), hq, hkv, d, seed=hq + d), "decode")


@pytest.mark.parametrize("parts", [1, 2, 3, 7])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (6, 2, 128)])
def test_decode_forced_splits(parts, hq, hkv, d):
    pa.set_max_partitions(parts)
    try:
        _run(A.make("fp4", [700, 20, 333, 512], [1] * 4, hq, hkv, d, seed=parts), "decode")
    finally:
        pa.set_max_partitions(0)


@pytest.mark.parametrize("hq,hkv,d,r", [(8, 2, 128, 2), (8, 2, 64, 5), (16, 2, 128, 9), (8, 8, 64, 16), (16, 2, 64, 16),
                                        (6, 2, 128, 4), (32, 8, 128, 5), (5, 1, 64, 7), (4, 1, 128, 3), (2, 2, 128, 11)])
def test_verify(hq, hkv, d, r):
    lens = [max(n, r) for n in LENS]
    _run(A.make("fp4", lens, [r] * len(lens), hq, hkv, d, seed=hq + r), "verify")


@pytest.mark.parametrize("parts", [1, 3])
def test_verify_forced_splits(parts):
    pa.set_max_partitions(parts)
    try:
        for hq, r in ((8, 5), (16, 2), (4, 3)):
            _run(A.make("fp4", [700, 20, 333], [r] * 3, hq, 2, 128, seed=parts), "verify")
    finally:
        pa.set_max_partitions(0)


@pytest.mark.parametrize("hq,hkv,d,r", [(8, 2, 128, 5), (4, 4, 64, 8), (16, 2, 128, 9)])
def test_tree_verify(hq, hkv, d, r):
    lens = [max(n, r) for n in LENS]
    c = A.make("fp4", lens, [r] * len(lens), hq, hkv, d, seed=hq + r)
    g = torch.Generator().manual_seed(r)
    masks = torch.zeros(len(lens), r, dtype=torch.int32)
    for b in range(len(lens)):
        for i in range(r):
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            masks[b, i] = (1 << i) | (int(masks[b, parent]) if parent >= 0 else 0)
    c["masks"] = masks.flatten().numpy()
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    got = pa.tree_verify(dev["q"].view(len(lens), r, hq, d), dev["k"], dev["v"], dev["table"],
                         torch.tensor(lens, dtype=torch.int32).cuda(), masks.cuda(), c["scale"], k_scale=dev["k_scale"],
                         v_scale=dev["v_scale"])
    assert pa.check_device_errors() == pa.PA_OK
    A.check(c, "verify", got.flatten(0, 1))


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (2, 2, 128), (4, 2, 64)])
def test_prefill(hq, hkv, d):
    lens, rows = [1, 37, 500, 333, 900, 129, 64], [1, 37, 5, 200, 33, 128, 1]
    _run(A.make("fp4", lens, rows, hq, hkv, d, seed=hq + d), "prefill")


@pytest.mark.parametrize("form,rows", [("decode", [1, 1, 1]), ("verify", [5, 5, 5]), ("prefill", [9, 1, 40])])
def test_no_head_scales_and_extreme_values(form, rows):
    c = A.make("fp4", [40, 100, 260], rows, 8, 2, 128, seed=21, head_scales=False)
    _run(c, form)
    big = {**c, "q": c["q"] * 2.0 ** 60, "scale": c["scale"] * 2.0 ** -60}
    _run(big, form)
    small = {**c, "q": c["q"] * 2.0 ** -60, "scale": c["scale"] * 2.0 ** 60}
    _run(small, form)
    peaked = {**c, "scale": c["scale"] * 30}  # one token takes nearly all of the softmax
    _run(peaked, form)
    flipped = {**c, "scale": -c["scale"]}
    _run(flipped, form)


@pytest.mark.parametrize("form,rows", [("decode", [1, 1]), ("verify", [5, 5]), ("prefill", [30, 70])])
def test_scales_over_the_whole_range(form, rows):
    # E4M3 scales from the smallest subnormal to the largest value, tokens apart by 2^17 in size
    c = A.make("fp4", [100, 70], rows, 8, 2, 128, seed=22, head_scales=False, junk=False)
    for n in ("k", "v"):
        codes, scales = plain.fp4_unpack(c[n].numpy(), 128)
        g = np.random.RandomState(5)
        scales = g.choice([0, 1, 2, 7, 8, 56, 100, 126], size=scales.shape, p=[.1, .2, .2, .1, .1, .1, .1, .1]).astype(np.uint8)
        c[n] = torch.from_numpy(plain.fp4_pack(codes, scales))
        c[n + "f"] = plain.fp4_values(c[n].numpy(), 128, np.ones(2))
    c["scale"] = 2.0 ** -14
    _run(c, form)


def test_bad_blocks_and_short_contexts():
    for form, r in (("decode", 1), ("verify", 5)):
        c = A.make("fp4", [100, 100, 100], [r] * 3, 8, 2, 128, seed=23)
        c["table"][1, 2] = -1
        _run(c, form, expect=pa.PA_ERR_DEVICE_BOUNDS)
        short = A.make("fp4", [40, 40], [r] * 2, 8, 2, 128, seed=24)
        short["lens"] = [40, r - 1]
        got = A.call(short, form)
        assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
        A.check({**short, "lens": [40], "rows": [r], "table": short["table"][:1], "q": short["q"][:r]}, form, got[:r])
        assert not got[r].any()


def test_the_same_call_twice_is_the_same():
    c = A.make("fp4", [700, 333, 12], [1] * 3, 32, 8, 128, seed=25)
    assert torch.equal(A.call(c, "decode"), A.call(c, "decode"))


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
@pytest.mark.parametrize("window", [None, 48])
def test_steps_as_they_are_used(kv, window):
    """A prompt chunk, then decode steps: norm and rotation of a packed projection, append, attention."""
    B, hq, hkv, d, steps, chunk = 3, 8, 2, 128, 4, 45
    g = torch.Generator().manual_seed(31)
    table = torch.randperm(B * 6, generator=g).to(torch.int32).view(B, 6).cuda()
    shape = (B * 6, hkv, 16, d if kv == "bf16" else 9 * d // 16)
    kc = torch.zeros(shape, dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
    vc = kc.clone()
    hs = {} if kv == "bf16" else {"k_scale": torch.full((hkv,), 2.0 ** -7).cuda(), "v_scale": torch.full((hkv,), 2.0 ** -7).cuda()}
    ang = torch.arange(100)[:, None].double() * 100.0 ** (-torch.arange(0, d, 2).double() / d)
    cs = torch.cat((ang.cos(), ang.sin()), 1).float().cuda()
    w = [(1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    kw = dict(hs)
    if window:
        kw |= {"window": window, "sinks": 2}
    n = 0
    for step in range(steps):
        r = chunk if step == 0 else 1
        n += r
        lens = torch.full((B,), n, dtype=torch.int32).cuda()
        qkv = torch.randn(B * r, (hq + 2 * hkv) * d, generator=g).to(torch.bfloat16).cuda()
        pos = (torch.arange(r, dtype=torch.int32) + n - r).repeat(B).cuda()
        q, k = pa.qk_norm_rope(qkv[:, : hq * d].unflatten(1, (hq, d)), qkv[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d)),
                               *w, cs, pos)
        v = qkv[:, (hq + hkv) * d:].contiguous().view(B, r, hkv, d)
        pa.append_kv(k.view(B, r, hkv, d), v, kc, vc, table, lens, **hs)
        rk, rv = pa.read_kv(kc, vc, table, lens, r, **hs)
        if kv == "bf16":
            assert torch.equal(rk, k.view(B, r, hkv, d)) and torch.equal(rv, v)
        if step == 0:
            starts = torch.arange(0, B * r + 1, r, dtype=torch.int32).cuda()
            out = pa.prefill(q, kc, vc, table, lens, starts, d ** -0.5, **kw)
        else:
            out = pa.decode(q.view(B, 1, hq, d), kc, vc, table, lens, d ** -0.5, **kw).flatten(0, 1)
        assert pa.check_device_errors() == pa.PA_OK
        c = {"kv": kv, "d": d, "lens": [n] * B, "rows": [r] * B, "window": window, "sinks": 2 if window else 0, "q": q,
             "table": table.cpu(), "scale": d ** -0.5}
        for name, cache in (("kf", kc), ("vf", vc)):
            c[name] = plain.to_f64(cache) if kv == "bf16" else plain.fp4_values(cache.cpu().numpy(), d, np.full(hkv, 2.0 ** -7))
        A.check(c, "prefill" if step == 0 else "decode", out)
