"""Attention of sequences that share prefixes on the GPU against the definition in fp64: groups of every size and shape,
prefixes of zero to many blocks, entries of the other rows never read, every cache type, splits and refusals."""

import numpy as np
import pytest
import torch

import attn_cases as A
from form_cases import BAD_ID, causal, check, on_gpu
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

KV = ["bf16", "e4m3", "fp4"]


def make(kv, groups, own, r, hq, hkv, d, seed):
    """groups: (sequences, prefix tokens) each; own: tokens behind the prefix of each sequence in turn (at least r)."""
    lens, starts, prefixes, at = [], [0], [], 0
    for n, p in groups:
        for _ in range(n):
            lens.append(p // 16 * 16 + max(own[at % len(own)], r))
            at += 1
        starts.append(at)
        prefixes.append(p)
    c = A.make(kv, lens, [r] * len(lens), hq, hkv, d, seed)
    # the sequences of a group look the prefix up in its first row: theirs is the definition's table, the call gets BAD_ID
    # where nothing may be read (blocks that only other rows had stay in the pool, unowned)
    call = c["table"].clone()
    for (n, p), s in zip(groups, starts):
        m = p // 16
        for b in range(s + 1, s + n):
            c["table"][b, :m] = c["table"][s, :m]
            call[b, :m] = BAD_ID
    c["starts"], c["prefixes"], c["call_table"] = starts, prefixes, call
    return c


def run(c, expect=None, as_verify=False, **kw):
    (q, k, v, _, lens), scales = on_gpu(c)
    fn = pa.decode if c["rows"][0] == 1 and not as_verify else pa.verify
    i32 = dict(dtype=torch.int32, device="cuda")
    got = fn(q, k, v, c["call_table"].cuda(), lens, c["scale"], group_starts=torch.tensor(c["starts"], **i32),
             prefix_lens=torch.tensor(c["prefixes"], **i32), **scales, **kw)
    assert pa.check_device_errors() == (expect or pa.PA_OK)
    return got


def hold(c, **kw):
    got = run(c, **kw)
    check(c, got, causal(c["lens"], c["rows"][0]), tiles=True)
    return got


GROUPS = [(3, 64), (1, 160), (5, 0), (2, 16), (7, 400)]
OWN = [1, 5, 16, 17, 40, 130, 33, 300, 64]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 2, 128), (8, 2, 64), (16, 2, 128), (6, 2, 64), (7, 1, 128), (32, 2, 64),
                                      (40, 8, 128), (64, 1, 128)])
def test_decode_head_groups(kv, hq, hkv, d):
    hold(make(kv, GROUPS, OWN, 1, hq, hkv, d, seed=hq))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r,hq,hkv,d", [(1, 8, 2, 64), (2, 8, 2, 128), (5, 8, 2, 128), (9, 16, 2, 128), (16, 8, 1, 64), (9, 28, 4, 64),
                                        (3, 40, 8, 128)])
def test_verify_rows(kv, r, hq, hkv, d):
    hold(make(kv, GROUPS, OWN, r, hq, hkv, d, seed=r + hq), as_verify=True)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("groups", [[(1, 16)], [(40, 33)], [(33, 1000), (1, 16)], [(1, 15), (2, 31)], [(0, 64), (3, 48), (0, 0), (2, 64)],
                                    [(1, 16 * i) for i in range(1, 71)]])
def test_group_shapes(kv, groups):
    # (70 groups: more than a warp looks through at once; prefixes that end inside a block: the rest is each row's own)
    c = make(kv, groups, OWN, 1, 8, 2, 64, seed=len(groups))
    hold(c)
    hold(make(kv, groups, OWN, 3, 8, 2, 64, seed=len(groups)), max_prefix_len=max(p for _, p in groups),
         max_own_len=300)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("parts", [1, 2, 5, 100])
@pytest.mark.parametrize("r", [1, 4, 16])
def test_forced_splits(kv, parts, r):
    pa.set_max_partitions(parts)
    try:
        hold(make(kv, [(3, 500), (2, 64)], [300, 20, 100], r, 8, 2, 128, seed=parts))
    finally:
        pa.set_max_partitions(0)


def test_sequences_outside_every_group_share_nothing():
    c = make("bf16", [(2, 0), (3, 64), (2, 0)], OWN, 1, 8, 2, 64, seed=3)
    c["starts"], c["prefixes"] = [2, 5], [64]
    hold(c)
    c["starts"], c["prefixes"] = [5], []  # no group at all
    c["call_table"] = c["table"]
    hold(c)


def test_a_large_batch_of_one_group():
    hold(make("bf16", [(300, 320)], OWN, 1, 32, 8, 128, seed=4), max_prefix_len=320, max_own_len=300)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r", [1, 3, 12])
def test_sequences_that_do_not_fit_are_zeros(kv, r):
    c = make(kv, [(4, 64), (2, 48)], [40, 50, 60, 70, 33, 44], r, 8, 2, 64, seed=5)
    lens = list(c["lens"])
    c["lens"] = lens[:1] + [64 + r - 1] + lens[2:4] + [0, -7]
    got = run(c, pa.PA_ERR_DEVICE_BOUNDS)
    assert all((got[b] == 0).all() for b in (1, 4, 5))
    c["lens"] = lens
    ref = run(c)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2:4], ref[2:4])
    # more of its own than the bound
    got = run(c, pa.PA_ERR_DEVICE_BOUNDS, max_own_len=60)
    assert (got[3] == 0).all() and all((got[b] != 0).any() for b in (0, 1, 2, 4, 5))


def test_a_prefix_past_its_bound_is_cut():
    c = make("bf16", [(2, 128)], [20, 30], 1, 8, 2, 64, seed=6)
    c["call_table"] = c["table"]  # the rest is looked up in each row
    got = run(c, pa.PA_ERR_DEVICE_BOUNDS, max_prefix_len=70)
    check(c, got, causal(c["lens"], 1), tiles=True)


@pytest.mark.parametrize("starts", [[0, 9], [-1, 2], [3, 1], [2 ** 31 - 1, -2 ** 31]])
def test_group_offsets_that_do_not_fit(starts):
    c = make("bf16", [(2, 64), (2, 0)], [20, 30], 1, 8, 2, 64, seed=7)
    c["starts"], c["prefixes"], c["call_table"] = starts, [64], c["table"]
    got = run(c, pa.PA_ERR_DEVICE_BOUNDS)  # the group shares nothing: every row reads its own table
    check(c, got, causal(c["lens"], 1), tiles=True)


def test_negative_prefixes_share_nothing():
    c = make("bf16", [(2, 0), (2, 64)], [20, 30], 1, 8, 2, 64, seed=8)
    c["prefixes"] = [-2 ** 31, 64]
    hold(c)


@pytest.mark.parametrize("kv", KV)
def test_a_bad_block_of_the_prefix_is_skipped_and_flagged(kv):
    c = make(kv, [(3, 96)], [20, 30], 1, 8, 2, 64, seed=9)
    c["call_table"][0, 2] = 1 << 29
    c["table"][:, 2] = 1 << 29
    got = run(c, pa.PA_ERR_DEVICE_BOUNDS)
    check(c, got, causal(c["lens"], 1), tiles=True)


def test_refusals():
    c = make("bf16", [(2, 64)], [20, 30], 1, 8, 2, 64, seed=10)
    (q, k, v, t, lens), _ = on_gpu(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    g, p = torch.tensor([0, 2], **i32), torch.tensor([64], **i32)
    with pytest.raises(ValueError):
        pa.decode(q, k, v, t, lens, 0.1, group_starts=g, prefix_lens=p.repeat(2))
    with pytest.raises(ValueError, match="need group_starts"):
        pa.decode(q, k, v, t, lens, 0.1, blocks=torch.zeros(2, 2, 1, **i32), prefix_lens=p)
    with pytest.raises(ValueError, match="need group_starts"):
        pa.decode(q, k, v, t, lens, 0.1, max_own_len=5)
    with pytest.raises(TypeError):
        pa.decode(q, k, v, t, lens, 0.1, group_starts=g)
    for kw in ({"max_prefix_len": -1}, {"max_own_len": -1}, {"max_prefix_len": 10 ** 9}):
        with pytest.raises(pa.PagedAttnError):
            pa.decode(q, k, v, t, lens, 0.1, group_starts=g, prefix_lens=p, **kw)
    with pytest.raises(ValueError):
        pa.tree_verify(q, k, v, t, lens, torch.ones(2, 1, **i32), 0.1, group_starts=g, prefix_lens=p)
