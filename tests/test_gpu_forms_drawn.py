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
