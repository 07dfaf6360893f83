"""Bounds of cache blocks and the selection of blocks on the GPU: every code, scale and index equal to the exact ones."""

import math

import numpy as np
import pytest
import torch

import attn_cases as A
from form_cases import on_gpu
from oracle import forms, plain
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

KV = ["bf16", "e4m3", "fp4"]
LENS = [1, 5, 16, 17, 40, 130, 333, 0, 64]


def _new_bounds(c, fill=77):
    nb, hkv = c["k"].shape[:2]
    codes = torch.full((nb, hkv, 2, c["d"]), fill, dtype=torch.int8, device="cuda")
    return codes, torch.full((nb, hkv), -3.0, device="cuda")


def _expected(c, n, codes, scale):
    for b, L in enumerate(c["lens"]):
        for col in range(max(0, L - n) // 16, (L + 15) // 16):
            pb = int(c["table"][b, col])
            if not 0 <= pb < len(codes):
                continue
            for g in range(codes.shape[1]):
                keys = c["kf"][pb, g, : min(16, L - 16 * col)].astype(np.float32).astype(np.float64)
                codes[pb, g], scale[pb, g] = forms.block_bounds(keys)
    return codes, scale


def _check_bounds(c, n):
    codes, scale = _new_bounds(c)
    want = _expected(c, n, codes.cpu().numpy(), scale.cpu().numpy())
    (_, k, _, table, lens), s = on_gpu(c)
    pa.block_bounds(k, table, lens, n, codes, scale, k_scale=s["k_scale"])
    assert pa.check_device_errors() == pa.PA_OK
    assert np.array_equal(codes.cpu().numpy(), want[0])
    assert np.array_equal(scale.cpu().numpy(), want[1])
    return codes, scale


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hkv", [1, 3, 8, 20])
@pytest.mark.parametrize("n", [1, 2, 17, 10000])
def test_bounds(kv, d, hkv, n):
    # tokens behind a context hold NaN, and so do the blocks that nobody owns
    _check_bounds(A.make(kv, LENS, [1] * len(LENS), hkv, hkv, d, seed=n + hkv), n)


@pytest.mark.parametrize("mag", [0.0, 2.0 ** -130, 2.0 ** -120, 1e-3, 3e38 / 8])
def test_bounds_of_extreme_bf16_keys(mag):
    c = A.make("bf16", [40, 16, 3], [1] * 3, 2, 2, 64, seed=3, junk=False)
    c["k"] = (c["k"].double() * mag).to(torch.bfloat16)
    c["kf"] = plain.to_f64(c["k"])
    _check_bounds(c, 100)


def test_bounds_at_the_edges_of_a_power_of_two():
    # amax on both sides of 127 / 64 2^e, where the exponent steps
    c = A.make("bf16", [64], [1], 1, 1, 64, seed=4, junk=False)
    k = torch.zeros_like(c["k"])
    for i, a in enumerate((127 / 64, 255 / 128, 2.0, 63.5)):
        k[int(c["table"][0, i]), 0, 3, 7] = a
        k[int(c["table"][0, i]), 0, 5, 9] = -a * 0.3
    c["k"], c["kf"] = k, plain.to_f64(k)
    _check_bounds(c, 64)


@pytest.mark.parametrize("sign", [-1.0, 0.0])
def test_bounds_of_odd_e4m3_scales(sign):
    c = A.make("e4m3", [40, 90], [1, 1], 2, 2, 128, seed=5)
    c["k_scale"] = c["k_scale"] * sign
    c["kf"] = plain.e4m3_values(c["k"].numpy(), c["k_scale"].numpy())
    _check_bounds(c, 90)


def test_bounds_flag_bad_blocks_and_lengths():
    c = A.make("bf16", [40, 40], [1, 1], 2, 2, 64, seed=6)
    c["table"][0, 1] = 1 << 29
    codes, scale = _new_bounds(c)
    want = _expected(c, 40, codes.cpu().numpy(), scale.cpu().numpy())
    (_, k, _, table, lens), _ = on_gpu(c)
    pa.block_bounds(k, table, lens, 40, codes, scale)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert np.array_equal(codes.cpu().numpy(), want[0])
    before = codes.clone()
    for wild in (49, -1, 2 ** 31 - 1, -2 ** 31):  # past the table's 48 tokens, negative
        pa.block_bounds(k, table, torch.full_like(lens, wild), 2, codes, scale)
        assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(codes, before)


# ---- selection --------------------------------------------------------------------------------

def _select(q, codes, scale, table, lens, count, **kw):
    got = pa.select_blocks(q.cuda(), codes.cuda(), scale.cuda(), table.cuda(), lens.cuda(), count, **kw)
    return got.cpu().numpy()


def _problem(lens, r, hq, hkv, d, seed, nb=None):
    g = torch.Generator().manual_seed(seed)
    width = max(1, max((n + 15) // 16 for n in lens))
    nb = nb or sum((n + 15) // 16 for n in lens) + 2
    codes = torch.randint(-127, 128, (nb, hkv, 2, d), generator=g, dtype=torch.int8).sort(2, descending=True).values
    scale = torch.exp2(torch.randint(-3, 3, (nb, hkv), generator=g).float())
    table = torch.full((len(lens), width), A.BAD_ID, dtype=torch.int32)
    ids, at = torch.randperm(nb, generator=g), 0
    for b, n in enumerate(lens):
        m = (n + 15) // 16
        table[b, :m] = ids[(at + torch.arange(m)) % nb].int()
        at += m
    q = torch.randn(len(lens), r, hq, d, generator=g).to(torch.bfloat16)
    return q, codes.contiguous(), scale, table, torch.tensor(lens, dtype=torch.int32)


def _want(q, codes, scale, table, lens, count, sinks, recent):
    B, r, hq, d = q.shape
    hkv = codes.shape[1]
    out = np.full((B, hkv, count), -1, np.int32)
    for b in range(B):
        nb = max(0, (int(lens[b]) + 15) // 16)
        ids = table[b, :nb].long().numpy()
        rows = plain.to_f64(q[b]).reshape(r, hkv, hq // hkv, d)
        for g in range(hkv):
            s = forms.scores(rows[:, g].reshape(-1, d), codes.numpy()[ids, g], scale.numpy()[ids, g])
            got = forms.pick(s, count, sinks, recent)
            out[b, g, : len(got)] = got
    return out


def _check_select(p, count, sinks=1, recent=2, **kw):
    got = _select(*p, count, sink_blocks=sinks, recent_blocks=recent, **kw)
    assert pa.check_device_errors() == pa.PA_OK
    want = _want(*p, count, sinks, recent)
    assert np.array_equal(got, want), np.argwhere(got != want)[:5].tolist()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("r,hq,hkv", [(1, 4, 4), (1, 32, 8), (1, 7, 1), (5, 8, 2), (1, 32, 1), (4, 40, 5), (3, 9, 1)])
@pytest.mark.parametrize("count", [3, 8, 64])
def test_select(d, r, hq, hkv, count):
    _check_select(_problem([3000, 47, 16 * 64, 16 * 64 + 1, 1, 0, 5000], r, hq, hkv, d, seed=hq + count), count)


@pytest.mark.parametrize("sinks,recent,count", [(0, 0, 5), (0, 1, 1), (5, 0, 5), (0, 7, 9), (40, 40, 80), (4, 8, 64)])
def test_select_ends(sinks, recent, count):
    _check_select(_problem([2000, 600, 70], 1, 8, 2, 64, seed=count), count, sinks, recent)


def test_ties_go_to_the_lowest_block():
    q, codes, scale, table, lens = _problem([5000, 1111], 1, 8, 2, 64, seed=9)
    codes[:] = codes[:1]  # every block alike
    scale[:] = 1.0
    _check_select((q, codes, scale, table, lens), 17)
    codes[int(table[0, 200])] = (codes[0].int() + 1).clamp(max=127).to(torch.int8)  # (int8 addition would wrap 127)
    _check_select((q, codes, scale, table, lens), 17)


def test_a_few_values_make_many_ties():
    q, codes, scale, table, lens = _problem([16 * 3000], 1, 4, 1, 64, seed=10)
    codes[:] = 0
    codes[:, :, 0, 0] = torch.randint(0, 3, codes.shape[:2], dtype=torch.int8)
    scale[:] = 1.0
    for count in (4, 500, 1500, 2999):
        _check_select((q, codes, scale, table, lens), count)


@pytest.mark.parametrize("mag", [0.0, 2.0 ** -126, 2.0 ** -60, 1.0, 2.0 ** 60])
def test_select_extreme_queries(mag):
    q, codes, scale, table, lens = _problem([900, 333], 2, 4, 2, 128, seed=11)
    q = (q.double() * mag).to(torch.bfloat16)
    q[0, 0, 0] = 0
    _check_select((q, codes, scale, table, lens), 6)


@pytest.mark.parametrize("n", [16 * 700, 16 * 3000, 16 * 9001, 16 * 52000])
def test_select_lengths_of_every_variant(n):
    # CTAs of each size, and more blocks than shared memory holds
    _check_select(_problem([n, 100], 1, 2, 1, 64, seed=12, nb=min(n // 16 + 10, 9100)), 100)


def test_select_flags_bad_blocks_and_lengths():
    q, codes, scale, table, lens = _problem([900, 333], 1, 4, 2, 64, seed=13)
    table[0, 20] = -5
    got = _select(q, codes, scale, table, lens, 12)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    t2 = table.clone()
    t2[0, 20] = 0
    want = _want(q, codes, scale, t2, lens, 57, 1, 2)  # every block, in order
    assert not (got[0] == 20).any() and set(got[0].ravel()) <= set(want[0].ravel())
    # longer than the bound: cut to it
    got = _select(q, codes, scale, t2, lens, 12, max_context_len=640)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert np.array_equal(got, _want(q, codes, scale, t2, torch.clamp(lens, max=640), 12, 1, 2))
    assert (_select(q, codes, scale, t2, torch.full_like(lens, -2 ** 31), 12) == -1).all()


def test_a_bound_holds_for_every_token():
    # the score of a block is at least the largest q . k of its tokens, for the rounded query
    c = A.make("bf16", [600], [1], 4, 2, 128, seed=14, junk=False)
    codes, scale = _check_bounds(c, 600)
    q = plain.to_f64(c["q"])[0].reshape(2, 2, 128)
    ids = c["table"][0].long().numpy()
    for g in range(2):
        s = forms.scores(q[g], codes.cpu().numpy()[ids, g], scale.cpu().numpy()[ids, g])
        rounded = []
        for row in q[g]:
            f = forms.code_exp(np.abs(row).max())
            rounded.append(np.ldexp(np.rint(np.ldexp(row, -f)), f))
        for j, pb in enumerate(ids):
            k = c["kf"][pb, g, : min(16, 600 - 16 * j)]
            assert (np.array(rounded) @ k.T).max() <= s[j] + 1e-9


def test_refusals():
    q, codes, scale, table, lens = (t.cuda() for t in _problem([900, 333], 1, 4, 2, 64, seed=15))
    ok = pa.select_blocks(q, codes, scale, table, lens, 8)
    assert ok.shape == (2, 2, 8)
    for kw, count in (({"sink_blocks": 5, "recent_blocks": 4}, 8), ({"sink_blocks": -1}, 8),
                      ({"max_context_len": 10 ** 6}, 8)):
        with pytest.raises(pa.PagedAttnError):
            pa.select_blocks(q, codes, scale, table, lens, count, **kw)
    with pytest.raises(ValueError):
        pa.select_blocks(q, codes, scale, table, lens, 0)
    with pytest.raises(TypeError):
        pa.select_blocks(q, codes.float(), scale, table, lens, 8)
    with pytest.raises(ValueError):
        pa.select_blocks(q, codes[:, :, :1].contiguous(), scale, table, lens, 8)
    with pytest.raises(pa.PagedAttnError):  # 33 rows a kv head
        pa.select_blocks(q.repeat(1, 17, 1, 1), codes, scale, table, lens, 8)
    with pytest.raises(ValueError):
        pa.block_bounds(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda"), table, lens, 1, codes, scale)
    assert pa.select_blocks(q[:0], codes, scale, table[:0], lens[:0], 8).shape == (0, 2, 8)
    pa.block_bounds(torch.zeros(*codes.shape[:2], 16, 64, dtype=torch.bfloat16, device="cuda"), table[:0], lens[:0], 1,
                    codes, scale)
