"""Drawn shapes of the forms over listed blocks, shared prefixes and kept weights, of selection and of eviction: every
route that a launch may take (clusters or scratch, one kernel or two, heads together or apart) is among them."""

import random

import numpy as np
import pytest
import torch

import attn_cases as A
import test_gpu_block_selection as S
import test_gpu_shared_prefix as P
import test_gpu_sparse_attention as B
import test_gpu_weights_evict as W
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

KV = ["bf16", "e4m3", "fp4"]
HEADS = [(4, 4), (8, 2), (16, 2), (2, 1), (6, 2), (7, 1), (8, 1), (20, 4), (9, 3), (16, 1), (32, 2)]


def _lens(rng, n, top, least=1):
    return [max(least, int(round(top ** rng.random()))) for _ in range(n)]


@pytest.mark.parametrize("seed", range(24))
def test_sparse(seed):
    rng = random.Random(seed)
    kv, (hq, hkv), d = rng.choice(KV), rng.choice(HEADS), rng.choice([64, 128])
    r = rng.choice([1, 1, rng.randint(2, max(2, min(16, 32 * hkv // hq)))])
    lens = _lens(rng, rng.randint(1, 12), 3000, r)
    c = A.make(kv, lens, [r] * len(lens), hq, hkv, d, seed=seed)
    B._run(c, B._lists(c, hkv, rng.randint(1, 60), seed), as_verify=r > 1)


@pytest.mark.parametrize("seed", range(24))
def test_prefix(seed):
    rng = random.Random(100 + seed)
    kv, (hq, hkv), d = rng.choice(KV), rng.choice(HEADS), rng.choice([64, 128])
    r = rng.choice([1, 1, rng.randint(2, max(2, min(16, 128 * hkv // hq)))])
    groups = [(rng.randint(1, 9), rng.choice([0, 16, 40, rng.randint(1, 1500)])) for _ in range(rng.randint(1, 6))]
    c = P.make(kv, groups, _lens(rng, 7, 600, r), r, hq, hkv, d, seed=seed)
    more = {}
    if rng.random() < 0.5:
        own = [n - p // 16 * 16 for n, p in zip(c["lens"], [p for n, p in groups for _ in range(n)])]
        more = {"max_prefix_len": max(p for _, p in groups), "max_own_len": max(own), "max_context_len": max(c["lens"])}
    P.hold(c, as_verify=r > 1, **more)


@pytest.mark.parametrize("seed", range(16))
def test_weights(seed):
    rng = random.Random(200 + seed)
    kv, (hq, hkv), d = rng.choice(KV), rng.choice(HEADS), rng.choice([64, 128])
    lens = _lens(rng, rng.randint(1, 8), 3000)
    c = A.make(kv, lens, [1] * len(lens), hq, hkv, d, seed=seed)
    W._decode(c, W._sums(c, seed), rng.choice([0.0, 0.9, 1.0]),
              **rng.choice([{}, {"max_context_len": max(lens)}]))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64), (7, 1, 64), (32, 1, 128), (3, 3, 128)])
def test_weights_of_contexts_that_no_cluster_holds(kv, hq, hkv, d):
    # more kept scores than fit beside the ring stages: they go through scratch
    c = A.make(kv, [9000, 17], [1, 1], hq, hkv, d, seed=hq)
    W._decode(c, W._sums(c), 0.9)


@pytest.mark.parametrize("seed", range(16))
def test_selection(seed):
    rng = random.Random(300 + seed)
    hq, hkv = rng.choice(HEADS)
    r = rng.randint(1, max(1, min(16, 32 * hkv // hq)))
    lens = _lens(rng, rng.randint(1, 8), 20000)
    sinks, recent = rng.randint(0, 3), rng.randint(0, 4)
    S._check_select(S._problem(lens, r, hq, hkv, rng.choice([64, 128]), seed), rng.randint(sinks + recent + 1, 80), sinks, recent)


@pytest.mark.parametrize("r,hq,hkv,d", [(1, 8, 4, 128), (3, 15, 5, 64), (2, 24, 4, 128), (4, 32, 4, 64), (1, 6, 3, 64)])
def test_selection_for_many_sequences(r, hq, hkv, d):
    # scores in scratch, heads of the same blocks together where there are four
    lens = [100 + 37 * i % 3000 for i in range(60)]
    S._check_select(S._problem(lens, r, hq, hkv, d, seed=hq, nb=500), 20)


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
@pytest.mark.parametrize("n,hkv", [(3, 2), (50, 4), (200, 2)])
def test_eviction_of_few_and_many(kv, n, hkv):
    rng = random.Random(n)
    lens = [rng.choice([0, 1, 15, 40, 200, rng.randint(1, 400)]) for _ in range(n)]
    c = A.make(kv, lens + [400], [1] * (n + 1), hkv, hkv, 64, seed=n)
    W._evict(c, W._sums(c, n), 50, 3, 10)


def test_e4m3_eviction_of_many():
    c = A.make("e4m3", [40, 20, 33, 17, 60], [1] * 5, 8, 8, 64, seed=3)
    W._evict(c, W._sums(c, 3), 20, 1, 3)


def test_the_largest_batches():
    # the largest grid dimensions, every sequence a token
    B_, i32 = 65535, dict(dtype=torch.int32, device="cuda")
    k = torch.randn(4, 1, 16, 64, device="cuda").to(torch.bfloat16)
    v = torch.randn_like(k)
    q = torch.randn(B_, 1, 1, 64, device="cuda").to(torch.bfloat16)
    table = torch.zeros(B_, 1, **i32)
    lens = torch.ones(B_, **i32)
    want = v[0, 0, 0].expand(B_, 1, 1, 64)
    codes, scale = torch.zeros(4, 1, 2, 64, dtype=torch.int8, device="cuda"), torch.ones(4, 1, device="cuda")
    pa.block_bounds(k, table, lens, 1, codes, scale)
    blocks = pa.select_blocks(q, codes, scale, table, lens, 3)
    assert (blocks[..., 0] == 0).all() and (blocks[..., 1:] == -1).all()
    assert torch.equal(pa.decode(q, k, v, table, lens, 0.1, blocks=blocks), want)
    assert torch.equal(pa.decode(q, k, v, table, lens, 0.1, group_starts=torch.tensor([0, B_], **i32),
                                 prefix_lens=torch.tensor([0], **i32)), want)
    new = pa.evict(k, v, torch.zeros(4, 1, 16, device="cuda"), table, lens, torch.ones(B_, 1, **i32), 5)
    assert (new == 1).all() and torch.equal(k[1, 0, 0], k[0, 0, 0])
    assert pa.check_device_errors() == pa.PA_OK
    with pytest.raises(pa.PagedAttnError):
        pa.decode(q[:1].repeat(65536, 1, 1, 1), k, v, table[:1].repeat(65536, 1), lens[:1].repeat(65536), 0.1,
                  blocks=blocks[:1].repeat(65536, 1, 1))


@pytest.mark.parametrize("n", [1, 200])
def test_a_bound_of_no_tokens_at_all(n):
    # max_context_len 0: every context is cut to nothing and flagged, on either route of each call
    c = A.make("bf16", [40] * n, [1] * n, 4, 2, 64, seed=1, junk=False)
    (q, k, v, table, lens), _ = S.on_gpu(c)
    nb = len(k)
    codes, scale = torch.zeros(nb, 2, 2, 64, dtype=torch.int8, device="cuda"), torch.ones(nb, 2, device="cuda")
    w = torch.ones(nb, 2, 16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    kw = {"max_context_len": 0}
    blocks = pa.select_blocks(q, codes, scale, table, lens, 4, **kw)
    assert (blocks == -1).all() and pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    starts, pre = torch.tensor([0, n], **i32), torch.tensor([16], **i32)
    for more in ({"blocks": blocks}, {"weights": w}, {"group_starts": starts, "prefix_lens": pre}):
        assert (pa.decode(q, k, v, table, lens, 0.1, **kw, **more) == 0).all()
        assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert (w == 1).all()
    assert (pa.evict(k, v, w, table, lens, table.clone(), 5, **kw) == 0).all()
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS


def test_4_bit_caches_without_head_scales():
    lens = [40, 333, 17]
    c = A.make("fp4", lens, [1] * 3, 8, 2, 128, seed=2, head_scales=False)
    S._check_bounds(c, 400)
    B._run(c, B._lists(c, 2, 9, 3))
    c = A.make("fp4", lens, [1] * 3, 8, 2, 128, seed=2, head_scales=False)
    W._decode(c, W._sums(c), 1.0)
    W._evict(c, W._sums(c), 30, 2, 5)


@pytest.mark.parametrize("sign", [-1.0, 0.0, 2.0 ** -20])
def test_odd_e4m3_scales(sign):
    def odd(c):
        from oracle import plain

        c["k_scale"][::2] *= sign
        c["v_scale"][1::2] *= sign
        c["kf"], c["vf"] = (plain.e4m3_values(c[n].numpy(), c[n + "_scale"].numpy()) for n in ("k", "v"))
        return c
    lens = [40, 333, 170]
    for r in (1, 3):
        c = odd(A.make("e4m3", lens, [r] * 3, 8, 2, 64, seed=4, junk=False))
        B._run(c, B._lists(c, 2, 9, 3), as_verify=r > 1)
    W._decode(odd(A.make("e4m3", lens, [1] * 3, 8, 2, 64, seed=4, junk=False)), W._sums(c), 1.0)
    (q, k, v, table, n), s = S.on_gpu(odd(A.make("e4m3", lens, [1] * 3, 8, 2, 64, seed=4, junk=False)))
    table[1:, :2] = table[0, :2]
    got = pa.decode(q, k, v, table, n, 0.125, group_starts=torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                    prefix_lens=torch.tensor([32], dtype=torch.int32, device="cuda"), **s)
    ref = pa.decode(q, k, v, table, n, 0.125, **s)
    # two kernels' roundings of the same rows: 2^-8 of the outputs each, f16 weights 2^-11 of the values' sizes each
    assert (got.float() - ref.float()).abs().max() <= 2.0 ** -6 * ref.float().abs().max()
    assert pa.check_device_errors() == pa.PA_OK


@pytest.mark.parametrize("at", [1, 33, 69])
def test_wrong_groups_are_flagged_wherever_they_stand(at):
    n = 70
    c = A.make("bf16", [40] * n, [1] * n, 4, 2, 64, seed=3, junk=False)
    (q, k, v, table, lens), _ = S.on_gpu(c)
    table[1:] = table[:1]
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, prefixes = torch.arange(n + 1, **i32), torch.full((n,), 16, **i32)
    kw = {"group_starts": starts, "prefix_lens": prefixes, "max_prefix_len": 16}
    ref = pa.decode(q, k, v, table, lens, 0.1, **kw)
    assert pa.check_device_errors() == pa.PA_OK
    prefixes[at] = 32  # past its bound: cut to it
    assert torch.equal(pa.decode(q, k, v, table, lens, 0.1, **kw), ref)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    prefixes[at] = 16
    starts[at + 1] = n + 5  # the group, and the next one, share nothing
    got = pa.decode(q, k, v, table, lens, 0.1, **kw)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(got[:at], ref[:at])
    assert (got.float() - ref.float()).abs().max() <= 2.0 ** -6 * ref.float().abs().max()


@pytest.mark.parametrize("r,hq,hkv,d", [(1, 8, 4, 128), (1, 32, 8, 64), (3, 8, 2, 128), (1, 40, 2, 64), (1, 30, 1, 128), (2, 5, 5, 64)])
def test_many_sequences_behind_a_wide_table(r, hq, hkv, d):
    # more pairs than SMs and a bound past 16384 tokens: scores in scratch, whatever the lengths are
    rng = random.Random(hq)
    lens = _lens(rng, 160 // hkv + 40, 3000, 0)
    q, codes, scale, table, n = S._problem(lens, r, hq, hkv, d, seed=hq, nb=3000)
    wide = torch.full((len(lens), 2100), A.BAD_ID, dtype=torch.int32)
    wide[:, : table.shape[1]] = table
    S._check_select((q, codes, scale, wide, n), 24)
    S._check_select((q, codes, scale, table, n), 24)


@pytest.mark.parametrize("d", [64, 128])
def test_bounds_of_infinities_and_nans(d):
    # an infinity takes the largest code of the widest scale, 2^122; a NaN gives way to the block's other tokens
    k = torch.randn(3, 2, 16, d, generator=torch.Generator().manual_seed(d)).to(torch.bfloat16)
    plain_k = k.clone()
    k[0, 0, 5, 7], k[0, 0, 6, 8], k[0, 1, 0, 9] = float("inf"), float("-inf"), 3.3e38
    k[1, 0, 0, 3] = k[1, 1, 15, 4] = k[2, 0, 7, 5] = float("nan")
    plain_k[1, 0, 0, 3] = plain_k[1, 0, 1, 3]  # a token of the same block in the NaN's place
    plain_k[1, 1, 15, 4] = plain_k[1, 1, 2, 4]
    plain_k[2, 0, 7, 5] = plain_k[2, 0, 8, 5]
    table, lens = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda"), torch.tensor([48], dtype=torch.int32, device="cuda")

    def bounds(keys):
        codes, scale = torch.zeros(3, 2, 2, d, dtype=torch.int8, device="cuda"), torch.zeros(3, 2, device="cuda")
        pa.block_bounds(keys.cuda(), table, lens, 48, codes, scale)
        assert pa.check_device_errors() == pa.PA_OK
        return codes.cpu(), scale.cpu()
    codes, scale = bounds(k)
    want, want_scale = bounds(plain_k)
    assert torch.equal(codes[1:], want[1:]) and torch.equal(scale[1:], want_scale[1:])
    assert scale[0].tolist() == [2.0 ** 122, 2.0 ** 121 if float(k[0, 1, 0, 9]) <= 127 * 2.0 ** 121 else 2.0 ** 122]
    assert codes[0, 0, 0, 7] == 127 and codes[0, 0, 1, 8] == -127
    assert codes[0, 0, 0, 0] == 1 and codes[0, 0, 1, 0] == -1  # ordinary keys beside them: rounded outwards
    assert codes[0, 1, 0, 9] == int(np.ceil(float(k[0, 1, 0, 9]) / float(scale[0, 1])))
