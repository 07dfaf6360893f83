"""Attention over listed blocks on the GPU against the definition in fp64: lists in any order with holes, of every cache
type and head group, blocks that no list names given back, splits, lists that leave a row nothing, and refusals."""

import numpy as np
import pytest
import torch

import attn_cases as A
from form_cases import BAD_ID, check, on_gpu
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

KV = ["bf16", "e4m3", "fp4"]
LENS = [1, 5, 16, 17, 40, 130, 333, 700, 64]


def _lists(c, hkv, count, seed, empty=()):
    """Random lists: up to count of a context's blocks, shuffled, holes of -1 (and worse) between them."""
    rng = np.random.default_rng(seed)
    out = np.full((len(c["lens"]), hkv, count), -1, np.int32)
    for b, n in enumerate(c["lens"]):
        nb = (n + 15) // 16
        for g in range(hkv):
            if (b, g) in empty:
                continue
            m = min(nb, int(rng.integers(1, count + 1)))
            cols = rng.permutation(nb)[:m]
            at = np.sort(rng.permutation(count)[:m])
            out[b, g, at] = cols
    out[out == -1] = np.where(rng.random((out == -1).sum()) < 0.5, -1, -2 ** 31)
    named = np.zeros((len(c["lens"]), c["table"].shape[1]), bool)
    for b in range(len(c["lens"])):
        for col in out[b][out[b] >= 0]:
            named[b, col] = True
    c["table"][torch.from_numpy(~named)] = BAD_ID  # not looked up
    return out


def _see(c, lists):
    r = c["rows"][0]

    def see(b, hkv):
        n = c["lens"][b]
        j = np.arange(n)
        own = n - r + np.arange(r)
        listed = np.stack([np.isin(j // 16, lists[b, g]) for g in range(hkv)])
        return listed[:, None] & (j[None] <= own[:, None])[None]
    return see


def _run(c, lists, expect=None, as_verify=False, **kw):
    args, scales = on_gpu(c)
    fn = pa.decode if c["rows"][0] == 1 and not as_verify else pa.verify
    got = fn(*args, c["scale"], blocks=torch.from_numpy(lists).cuda(), **scales, **kw)
    assert pa.check_device_errors() == (expect or pa.PA_OK)
    check(c, got, _see(c, lists), tiles=False)
    return got


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 2, 128), (8, 2, 64), (16, 2, 128), (6, 2, 64), (7, 1, 128), (32, 2, 64),
                                      (40, 8, 128), (32, 1, 128)])
def test_decode_head_groups(kv, hq, hkv, d):
    c = A.make(kv, LENS, [1] * len(LENS), hq, hkv, d, seed=hq)
    _run(c, _lists(c, hkv, 20, hq))


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r,hq,hkv,d", [(1, 8, 2, 64), (2, 8, 2, 128), (5, 8, 2, 128), (16, 4, 2, 64), (8, 16, 4, 128), (3, 7, 1, 64)])
def test_verify_rows(kv, r, hq, hkv, d):
    lens = [max(n, r) for n in LENS]
    c = A.make(kv, lens, [r] * len(lens), hq, hkv, d, seed=r + hq)
    _run(c, _lists(c, hkv, 24, r), as_verify=True)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r", [1, 4])
@pytest.mark.parametrize("parts", [1, 2, 7, 300])
def test_forced_splits(kv, r, parts):
    c = A.make(kv, [700, 20, 333], [r] * 3, 8, 2, 128, seed=parts)
    lists = _lists(c, 2, 150, parts)  # (ids beyond the first two windows of 32 a warp)
    pa.set_max_partitions(parts)
    try:
        _run(c, lists)
    finally:
        pa.set_max_partitions(0)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r", [1, 3])
def test_long_lists_in_one_partition(kv, r):
    c = A.make(kv, [8000], [r], 4, 1, 64, seed=r)
    lists = _lists(c, 1, 500, 3)
    pa.set_max_partitions(1)
    try:
        _run(c, lists)
    finally:
        pa.set_max_partitions(0)


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("r", [1, 3])
@pytest.mark.parametrize("parts", [0, 3])
def test_lists_that_leave_nothing_give_zeros(kv, r, parts):
    c = A.make(kv, [700, 20, 333], [r] * 3, 8, 2, 128, seed=5)
    lists = _lists(c, 2, 12, 6, empty={(0, 0), (1, 0), (1, 1)})
    pa.set_max_partitions(parts)
    try:
        got = _run(c, lists)
    finally:
        pa.set_max_partitions(0)
    assert (got[0, :, :4] == 0).all() and (got[1] == 0).all() and not (got[0, :, 4:] == 0).all()


def test_a_row_sees_no_later_token_of_a_listed_block():
    c = A.make("bf16", [37], [6], 4, 2, 64, seed=7)
    _run(c, np.array([[[2], [1]]], np.int32))


@pytest.mark.parametrize("kv", KV)
def test_columns_past_the_context_are_skipped_and_flagged(kv):
    c = A.make(kv, [40, 33], [1, 1], 8, 2, 64, seed=8)
    lists = np.array([[[0, 3, 2, 2 ** 31 - 1], [1, -1, 2, -1]]] * 2, np.int32)
    args, scales = on_gpu(c)
    got = pa.decode(*args, c["scale"], blocks=torch.from_numpy(lists).cuda(), **scales)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    lists = np.where(lists > 2, -1, lists)
    check(c, got, _see(c, lists), tiles=False)


@pytest.mark.parametrize("kv", KV)
def test_bad_block_ids_are_skipped_and_flagged(kv):
    c = A.make(kv, [40, 33], [1, 1], 8, 2, 64, seed=9)
    lists = np.array([[[0, 1, 2], [1, 0, 2]]] * 2, np.int32)
    for bad in (-2 ** 31, -1, 1 << 28):
        c["table"][1, 1] = bad
        args, scales = on_gpu(c)
        got = pa.decode(*args, c["scale"], blocks=torch.from_numpy(lists).cuda(), **scales)
        assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
        check(c, got, _see(c, lists), tiles=False)


def test_empty_contexts():
    c = A.make("bf16", [40, 16], [1, 1], 8, 2, 64, seed=10)
    args, _ = on_gpu(c)
    lists = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    args[4][1] = 0
    got = pa.decode(*args, c["scale"], blocks=lists)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert (got[1] == 0).all() and (got[0] != 0).any()


def test_refusals():
    c = A.make("bf16", [40, 16], [1, 1], 8, 2, 64, seed=11)
    args, _ = on_gpu(c)
    lists = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pa.decode(*args, 0.1, blocks=lists[:, :1].contiguous())
    with pytest.raises(TypeError):
        pa.decode(*args, 0.1, blocks=lists.long())
    with pytest.raises(ValueError, match="one of"):
        pa.decode(*args, 0.1, blocks=lists, window=5)
    with pytest.raises(pa.PagedAttnError):
        pa.decode(*args, 0.1, blocks=lists[..., :0])
    with pytest.raises(ValueError):
        pa.tree_verify(*args, torch.ones(2, 1, dtype=torch.int32, device="cuda"), 0.1, blocks=lists)
    q = args[0].repeat(1, 9, 1, 1)  # 36 rows a kv head
    with pytest.raises(pa.PagedAttnError):
        pa.verify(q, *args[1:], 0.1, blocks=lists)
