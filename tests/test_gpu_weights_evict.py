"""Decode that keeps the tokens' attention weights, and eviction by them, on the GPU: weights against fp64, evicted caches bit
for bit, every cache type, ties, infinities and NaNs among the sums, lengths of zero to past the keys' shared memory."""

import numpy as np
import pytest
import torch

import attn_cases as A
from form_cases import BAD_ID, causal, check, on_gpu
from oracle import append as OA
from oracle import forms, plain
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

KV = ["bf16", "e4m3", "fp4"]
LENS = [1, 5, 16, 17, 40, 130, 333, 700, 64]


def _sums(c, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.exp(2 * torch.randn(c["k"].shape[0], c["k"].shape[1], 16, generator=g))


def _hold_weights(c, before, after, decay, dots, probs):
    """The sums' bound, relative to the step's weight of each head: twice the error of a score (as in
    form_cases.check; the row's log2-sum-exp has it as well), four roundings of a base-2 score, the row sum's n
    additions, and the exponentials' own (2^-19); where partial rows meet in memory also the log2-sum-exps that they are
    kept as, of a part and of the row: the logarithm of a sum below 2^16 is below 16, so that two units in its last place
    (2^-20) are 2^-19, and the sum with the maximum, below 32, rounds by 2^-20, twice each and times ln 2 < 0.7; then
    decay * sum + weight in fp32, decay the fp32 number that the call takes (a product's and a sum's rounding, 2^-23 of it)."""
    decay = float(np.float32(decay))
    want = before.double().numpy().copy()
    slack = np.zeros(want.shape)
    hkv, d = want.shape[1], c["d"]
    for b, n in enumerate(c["lens"]):
        g = dots.shape[2] // hkv
        for h in range(hkv):
            p = probs[b][h, 0]  # [G, n]
            y = dots[b, 0, h * g: (h + 1) * g]
            rel = 4 * d * 2.0 ** -24 * y + 4 * 2.0 ** -22 * y + n * 2.0 ** -24 + 2.0 ** -19 + \
                0.7 * 2 * (2.0 ** -19 + 2.0 ** -20)
            for j in range(n):
                at = (int(c["table"][b, j // 16]), h, j % 16)
                old = 0.0 if j == n - 1 else decay * want[at] if decay else 0.0
                want[at] = old + p[:, j].sum()
                slack[at] = (p[:, j] * rel[:, 0]).sum() + 2.0 ** -23 * abs(want[at]) + 1e-37
    got = after.double().numpy()
    touched = slack > 0
    assert np.array_equal(got[~touched], before.double().numpy()[~touched], equal_nan=True)
    over = np.abs(got - want)[touched] - slack[touched]
    assert (over <= 0).all(), (over.max(), int((over > 0).sum()))


def _decode(c, sums, decay, expect=None, **kw):
    args, scales = on_gpu(c)
    w = sums.cuda()
    got = pa.decode(*args, c["scale"], weights=w, decay=decay, **scales, **kw)
    assert pa.check_device_errors() == (expect or pa.PA_OK)
    _, dots, probs = check(c, got, causal(c["lens"], 1), tiles=False)
    _hold_weights(c, sums, w.cpu(), decay, dots, probs)
    return w, got


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 2, 128), (8, 2, 64), (16, 2, 128), (6, 2, 64), (7, 1, 128), (32, 2, 64),
                                      (40, 8, 128), (32, 1, 128)])
def test_weights_head_groups(kv, hq, hkv, d):
    c = A.make(kv, LENS, [1] * len(LENS), hq, hkv, d, seed=hq)
    _decode(c, _sums(c), 1.0)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("parts", [1, 2, 7])
@pytest.mark.parametrize("decay", [0.0, 0.9, 1.0, -1.0])
def test_weights_splits_and_decay(kv, parts, decay):
    c = A.make(kv, [700, 20, 333], [1] * 3, 8, 2, 128, seed=parts)
    sums = _sums(c)
    for b, n in enumerate(c["lens"]):  # the new token's slot holds whatever its block's last user left
        sums[int(c["table"][b, (n - 1) // 16]), :, (n - 1) % 16] = float("nan")
    if decay == 0:
        sums[:] = float("nan")
    pa.set_max_partitions(parts)
    try:
        _decode(c, sums, decay, max_context_len=700)
    finally:
        pa.set_max_partitions(0)


def test_weights_of_a_step_sum_to_the_heads():
    c = A.make("bf16", [5000], [1], 8, 2, 64, seed=3, junk=False)
    w, _ = _decode(c, torch.zeros(c["k"].shape[0], 2, 16), 0.0)
    ids = c["table"][0].long().cuda()
    assert torch.allclose(w[ids].sum((0, 2)), torch.full((2,), 4.0, device="cuda"), rtol=1e-5)


@pytest.mark.parametrize("kv", KV)
def test_weights_of_empty_contexts_and_bad_blocks(kv):
    c = A.make(kv, [40, 33, 64], [1] * 3, 8, 2, 64, seed=4)
    args, scales = on_gpu(c)
    sums = _sums(c)
    c["lens"] = [40, 0, 64]
    c["table"][2, 1] = 1 << 29
    args[4][1] = 0
    args[3][2, 1] = 1 << 29
    w = sums.cuda()
    got = pa.decode(*args, c["scale"], weights=w, **scales)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert (got[1] == 0).all()
    _, dots, probs = check(c, got, causal(c["lens"], 1), tiles=False)
    keep = c["table"].clone()
    c["table"][2, 1] = c["k"].shape[0]  # (its tokens have no slot: a row behind the pool in the expectation)
    pad = torch.cat((sums, torch.zeros(1, 2, 16)))
    _hold_weights(c, pad, torch.cat((w.cpu(), torch.zeros(1, 2, 16))), 1.0, dots, probs)
    c["table"] = keep


def test_weights_refusals():
    c = A.make("bf16", [40, 33], [1] * 2, 8, 2, 64, seed=5)
    args, _ = on_gpu(c)
    w = _sums(c).cuda()
    with pytest.raises(ValueError):
        pa.decode(*args, 0.1, weights=w[:, :1].contiguous())
    with pytest.raises(TypeError):
        pa.decode(*args, 0.1, weights=w.double())
    with pytest.raises(ValueError):
        pa.verify(*args, 0.1, weights=w)
    with pytest.raises(ValueError):
        pa.decode(*args, 0.1, decay=0.5)
    for decay in (float("nan"), float("inf")):
        with pytest.raises(pa.PagedAttnError):
            pa.decode(*args, 0.1, weights=w, decay=decay)
    with pytest.raises(pa.PagedAttnError):  # a group of 40
        pa.decode(args[0].repeat(1, 1, 10, 1), *args[1:], 0.1, weights=w)


# ---- eviction ---------------------------------------------------------------------------------

def _fresh(c, keep):
    """A table of unused blocks at the end of a grown pool, out of order, and the grown case."""
    nb, B = c["k"].shape[0], len(c["lens"])
    m = (keep + 15) // 16
    g = torch.Generator().manual_seed(7)
    table = (nb + torch.randperm(B * m + 2, generator=g)[: B * m]).view(B, m).int()
    for n in ("k", "v"):
        c[n] = torch.cat((c[n], torch.full((B * m + 2, *c[n].shape[1:]), 0x5A, dtype=torch.uint8).view(c[n].dtype)
                          if c[n].dtype == torch.uint8 else torch.full((B * m + 2, *c[n].shape[1:]), 9.0, dtype=c[n].dtype)))
        if c["kv"] == "e4m3":
            c[n + "_scale"] = torch.cat((c[n + "_scale"], torch.full((B * m + 2, c[n].shape[1]), -5.0)))
    return table


def _expected_evict(c, sums, fresh, keep, sinks, recent):
    k, v, w = c["k"].clone(), c["v"].clone(), sums.clone()
    ks, vs = (None if c["k_scale"] is None else c[n].clone() for n in ("k_scale", "v_scale"))
    if c["k_scale"] is None:
        ks = vs = None
    hkv, d = k.shape[1], c["d"]
    lens = []
    for b, n in enumerate(c["lens"]):
        n = max(n, 0)
        lens.append(min(n, keep))
        ids = c["table"][b].long()
        j = torch.arange(n)
        for g in range(hkv):
            s = sums[ids[j // 16], g, j % 16].numpy().astype(np.float64) if n else np.zeros(0)
            pos = torch.from_numpy(forms.evict_positions(s, keep, sinks, recent)) if n > keep else j
            src, at = ids[pos // 16], pos % 16
            to, slot = fresh[b].long()[torch.arange(len(pos)) // 16], torch.arange(len(pos)) % 16
            w[to, g, slot] = sums[src, g, at]
            for out, cache, scale, new in ((k, c["k"], c["k_scale"], ks), (v, c["v"], c["v_scale"], vs)):
                if c["kv"] == "bf16":
                    out[to, g, slot] = cache[src, g, at]
                elif c["kv"] == "fp4":
                    flat, dst = cache.view(len(cache), hkv, -1), out.view(len(cache), hkv, -1)
                    for size, base in ((d // 2, 0), (d // 16, 8 * d)):
                        col = torch.arange(size)
                        dst[to[:, None], g, base + slot[:, None] * size + col] = \
                            flat[src[:, None], g, base + at[:, None] * size + col]
                else:
                    table = np.array([OA.e4m3_decode(i) for i in range(256)], np.float32)
                    val = table[cache[src, g, at].numpy()] * scale[src, g].numpy()[:, None]
                    for i in range(0, len(pos), 16):
                        x = val[i: i + 16].astype(np.float32)
                        amax = np.abs(x).max()
                        sc = np.float32(amax / np.float32(448)) if amax > 0 else np.float32(1)
                        code = [[OA.e4m3_encode(np.float32(y / sc)) for y in row] for row in x]
                        out[to[i], g, : len(x)] = torch.tensor(code, dtype=torch.uint8)
                        new[to[i], g] = float(sc)
    return k, v, ks, vs, w, lens


def _evict(c, sums, keep, sinks, recent, expect=None, **kw):
    fresh = _fresh(c, keep)
    sums = torch.cat((sums, torch.full((c["k"].shape[0] - sums.shape[0], *sums.shape[1:]), 3.0)))
    want = _expected_evict(c, sums, fresh, keep, sinks, recent)
    (_, k, v, table, lens), scales = on_gpu({**c, "q": torch.zeros(len(c["lens"]), c["k"].shape[1], c["d"], dtype=torch.bfloat16),
                                             "rows": [1] * len(c["lens"])})
    w = sums.cuda()
    if c["kv"] != "e4m3":
        scales = {}
    got = pa.evict(k, v, w, table, lens, fresh.cuda(), keep, sinks=sinks, recent=recent, head_dim=c["d"], **scales, **kw)
    assert pa.check_device_errors() == (expect or pa.PA_OK)
    assert got.tolist() == want[5]

    def bits(t):
        return t.cpu().contiguous().view(torch.uint8 if t.dtype == torch.uint8 else torch.int16 if t.dtype == torch.bfloat16
                                         else torch.int32)
    assert torch.equal(bits(w), bits(want[4]))
    for a, b in ((k, want[0]), (v, want[1])):
        assert torch.equal(bits(a), bits(b))
    if c["kv"] == "e4m3":
        assert torch.equal(scales["k_scale"].cpu(), want[2]) and torch.equal(scales["v_scale"].cpu(), want[3])
    return k, v, w, got, fresh, scales


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hkv,d", [(1, 64), (2, 128), (5, 64), (8, 128)])
@pytest.mark.parametrize("keep,sinks,recent", [(1, 0, 0), (1, 0, 1), (20, 4, 5), (33, 0, 33), (64, 64, 0), (100, 1, 7), (1000, 4, 100)])
def test_evict(kv, hkv, d, keep, sinks, recent):
    lens = [1, 16, 17, 40, 130, 333, 64, 0, 100]
    if kv == "e4m3":
        lens, hkv = lens[:5] + lens[7:8], min(hkv, 2)  # (the oracle encodes one value at a time)
    c = A.make(kv, lens, [1] * len(lens), hkv, hkv, d, seed=keep)
    _evict(c, _sums(c, keep), keep, sinks, recent)


def test_ties_go_to_the_earliest_token():
    c = A.make("bf16", [700, 333], [1] * 2, 2, 2, 64, seed=3, junk=False)
    g = torch.Generator().manual_seed(3)
    few = torch.tensor([0.0, -0.0, 1.0, 2.0])
    for sums in (torch.ones(c["k"].shape[0], 2, 16), few[torch.randint(0, 4, (c["k"].shape[0], 2, 16), generator=g)]):
        for keep in (17, 200, 600):
            _evict(dict(c), sums.clone(), keep, 4, 8)


def test_infinities_nans_and_negative_sums():
    c = A.make("bf16", [700, 333], [1] * 2, 2, 2, 64, seed=4, junk=False)
    g = torch.Generator().manual_seed(4)
    odd = torch.tensor([float("inf"), float("-inf"), float("nan"), -1.0, 1e-40, -1e-40, 3e38])
    sums = odd[torch.randint(0, 7, (c["k"].shape[0], 2, 16), generator=g)] * torch.rand(c["k"].shape[0], 2, 16, generator=g)
    for keep in (17, 300, 650):
        _evict(dict(c), sums.clone(), keep, 4, 8)


@pytest.mark.parametrize("n", [2048, 2049, 4097, 50016, 98304, 98305, 120000])
def test_lengths_of_every_variant(n):
    c = A.make("bf16", [n, 100], [1] * 2, 1, 1, 64, seed=5, junk=False)
    _evict(c, _sums(c), 500, 4, 100, max_context_len=n)


def test_contexts_past_their_bound_are_cut_and_bad_blocks_flagged():
    c = A.make("bf16", [100, 64], [1] * 2, 2, 2, 64, seed=6, junk=False)
    sums = _sums(c)
    fresh = _fresh(c, 32)
    sums = torch.cat((sums, torch.zeros(c["k"].shape[0] - sums.shape[0], 2, 16)))
    (_, k, v, table, lens), _ = on_gpu({**c, "q": torch.zeros(2, 2, 64, dtype=torch.bfloat16)})
    got = pa.evict(k, v, sums.cuda(), table, lens, fresh.cuda(), 32, recent=4, max_context_len=80)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert got.tolist() == [32, 32]
    pos = forms.evict_positions(sums[c["table"][0].long()[torch.arange(80) // 16], 1, torch.arange(80) % 16].numpy(), 32, 0, 4)
    new = torch.stack([k[int(fresh[0, i // 16]), 1, i % 16] for i in range(32)]).cpu()
    assert torch.equal(new, torch.stack([c["k"][int(c["table"][0, j // 16]), 1, j % 16] for j in pos.tolist()]))
    # a block that is not there: its tokens count as sum 0 and read as zeros; a page that cannot be written is left out
    table[1, 1] = 1 << 29
    fresh2 = fresh.clone()
    fresh2[0, 0] = -3
    sums2 = torch.where(sums > 0, -sums, sums).cuda()
    got = pa.evict(k, v, sums2, table, lens, fresh2.cuda(), 32)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    for i in range(16):  # sequence 1: all 16 of the lost tokens stand above the negative sums
        pass
    rows = torch.stack([k[int(fresh[1, i // 16]), 0, i % 16] for i in range(32)])
    assert int((rows == 0).all(1).sum()) == 16
    for wild in (-1, -2 ** 31):
        got = pa.evict(k, v, sums2, table, torch.full_like(lens, wild), fresh.cuda(), 32)
        assert got.tolist() == [0, 0] and pa.check_device_errors() == pa.PA_OK


def test_shared_blocks_stay_whole():
    c = A.make("bf16", [100, 100], [1] * 2, 2, 2, 64, seed=7, junk=False)
    c["table"][1, :4] = c["table"][0, :4]
    old = c["k"].clone()
    k, *_ = _evict(c, _sums(c), 32, 4, 8)
    assert torch.equal(k[: len(old)].cpu(), old)


def test_evict_refusals():
    c = A.make("bf16", [100, 100], [1] * 2, 2, 2, 64, seed=8, junk=False)
    (_, k, v, table, lens), _ = on_gpu({**c, "q": torch.zeros(2, 2, 64, dtype=torch.bfloat16)})
    w = torch.zeros(len(k), 2, 16, device="cuda")
    fresh = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    for keep, kw in ((0, {}), (33, {}), (8, {"sinks": 4, "recent": 5}), (8, {"sinks": -1}), (8, {"recent": -1}),
                     (8, {"max_context_len": 10 ** 6}), (8, {"sinks": 2 ** 31, "recent": 2 ** 31})):
        with pytest.raises(pa.PagedAttnError):
            pa.evict(k, v, w, table, lens, fresh, keep, **kw)
    with pytest.raises(ValueError):
        pa.evict(k, v, w[:, :1].contiguous(), table, lens, fresh, 8)
    with pytest.raises(ValueError):
        pa.evict(k, v, w, table, lens, fresh[:1], 8)
    with pytest.raises(TypeError):
        pa.evict(k, v, w, table, lens, fresh.long(), 8)
    assert pa.evict(k, v, w, table[:0], lens[:0], fresh[:0], 8).shape == (0,)
    assert pa.check_device_errors() == pa.PA_OK


# ---- the operators together -------------------------------------------------------------------

@pytest.mark.parametrize("kv", KV)
def test_a_serving_run(kv):
    """Steps of a batch: append, bounds of the new token, selection, sparse attention; weights kept by full decodes; then
    eviction, and attention over what is left equals the definition's over the kept tokens."""
    g = torch.Generator().manual_seed(11)
    hq, hkv, d, B = 8, 2, 64, 3
    lens = [100, 333, 47]
    c = A.make(kv, lens, [1] * B, hq, hkv, d, seed=12, junk=False)
    m = c["table"].shape[1]
    (q, k, v, table, n), s = on_gpu(c)
    codes = torch.zeros(len(k), hkv, 2, d, dtype=torch.int8, device="cuda")
    scale = torch.ones(len(k), hkv, device="cuda")
    w = torch.zeros(len(k), hkv, 16, device="cuda")
    pa.block_bounds(k, table, n, 333, codes, scale, k_scale=s["k_scale"])
    kn, vn = (torch.randn(B, 1, hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    n = n - 5
    for _ in range(5):
        n = n + 1
        if kv == "bf16":
            pa.append_kv(kn, vn, k, v, table, n)
        pa.block_bounds(k, table, n, 1, codes, scale, k_scale=s["k_scale"])
        blocks = pa.select_blocks(q, codes, scale, table, n, m, recent_blocks=2)  # every block: the same as without
        sparse = pa.decode(q, k, v, table, n, c["scale"], blocks=blocks, **s)
        full = pa.decode(q, k, v, table, n, c["scale"], weights=w, **s)
        assert (sparse.float() - full.float()).abs().max() < 2.0 ** -6
        assert torch.equal(full, pa.decode(q, k, v, table, n, c["scale"], weights=w.clone(), decay=0.0, **s))
    keep = 40
    fresh_c = {**c, "k": k.cpu(), "v": v.cpu(), **{x: (None if t is None else t.cpu()) for x, t in s.items()}}
    fresh = _fresh(fresh_c, keep)
    (_, k, v, table, _), s = on_gpu(fresh_c)
    w = torch.cat((w, torch.zeros(len(k) - len(w), hkv, 16, device="cuda")))
    new = pa.evict(k, v, w, table, n, fresh.cuda(), keep, sinks=2, recent=10, head_dim=d, **s)
    assert new.tolist() == [40, 40, 40]
    out = pa.decode(q, k, v, fresh.cuda(), new, c["scale"], **s)
    assert pa.check_device_errors() == pa.PA_OK
    # the definition over the old cache, restricted to the kept tokens
    vals = {"bf16": lambda x, sc: plain.to_f64(x), "e4m3": lambda x, sc: plain.e4m3_values(x.cpu().numpy(), sc.cpu().numpy()),
            "fp4": lambda x, sc: plain.fp4_values(x.cpu().numpy(), d, sc.cpu().numpy())}[kv]
    kf, vf = vals(k, s["k_scale"]), vals(v, s["v_scale"])
    sums = w.cpu()
    ids = c["table"].long()

    def see(b):
        r = np.zeros((hkv, 1, int(n[b])), bool)
        j = torch.arange(int(n[b]))
        for h in range(hkv):
            r[h, 0, forms.evict_positions(sums[ids[b, j // 16], h, j % 16].numpy().astype(np.float64), keep, 2, 10)] = True
        return r
    ref, spread, _, _ = forms.attend(plain.to_f64(q), kf, vf, c["table"].numpy(), n.tolist(), c["scale"], see)
    # (E4M3 pages are re-encoded: half a step of 2^-4 of each value, keys' scores and values alike)
    tol = 0.25 if kv == "e4m3" else 2.0 ** -6
    assert np.abs(plain.to_f64(out) - ref).max() < tol
