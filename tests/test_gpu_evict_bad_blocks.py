"""Eviction around block ids that are not there, on the GPU: the whole pools and sums against an expected state, bit for bit.
Tokens of a lost block count as sum 0 and move as zeros with a sum of 0; a page of the new table that is not there is
left out, and nothing else changes.  Few and many (sequence, head) pairs."""

import pytest
import torch

import attn_cases as A
from form_cases import on_gpu
from oracle import forms, plain
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

LENS = [100, 64, 40]
KEEP = 32  # two pages of each sequence; the last has fewer tokens than that to lose
LOST = [(1, 1), (0, 4)]  # (sequence, column) of the blocks that are not there


def _rows(kv, d, cache):
    """The parts of a cache that a token's row is: views [NB, Hkv, 16, ...]."""
    if kv != "fp4":
        return [cache]
    flat = cache.view(*cache.shape[:2], -1)
    return [flat[..., : 8 * d].unflatten(-1, (16, -1)), flat[..., 8 * d:].unflatten(-1, (16, -1))]


def _move(c, caches, sums, scales, table, fresh, sinks, recent):
    """The expected caches, sums and scales, in place."""
    kv, hkv, d, nb = c["kv"], sums.shape[1], c["d"], len(sums)
    before = [[r.clone() for r in _rows(kv, d, x)] for x in caches]
    old = sums.clone()
    scale0 = [s.clone() for s in scales]
    for b, n in enumerate(c["lens"]):
        for h in range(hkv):
            at = [(int(table[b, j // 16]), h, j % 16) for j in range(n)]
            there = [0 <= a[0] < nb for a in at]
            sum_of = [float(old[a]) if ok else 0.0 for a, ok in zip(at, there)]
            kept = forms.evict_positions(sum_of, KEEP, sinks, recent).tolist()
            for page in range(0, len(kept), 16):
                dst = int(fresh[b, page // 16])
                if not 0 <= dst < nb:
                    continue
                part = kept[page: page + 16]
                for i, j in enumerate(part):
                    sums[dst, h, i] = sum_of[j]
                for x, (cache, rows) in enumerate(zip(caches, before)):
                    if kv != "e4m3":
                        for new, src in zip(_rows(kv, d, cache), rows):
                            for i, j in enumerate(part):
                                new[dst, h, i] = src[at[j]] if there[j] else 0
                        continue
                    # fp32 values times the old pages' scales; amax / 448; to nearest even (torch's conversion)
                    v = torch.stack([rows[0][at[j]].view(torch.float8_e4m3fn).float() * scale0[x][at[j][:2]] if there[j]
                                     else torch.zeros(d) for j in part])
                    amax = v.abs().max()
                    s = amax / 448 if amax > 0 else torch.tensor(1.0)
                    cache[dst, h, : len(part)] = (v / s).to(torch.float8_e4m3fn).view(torch.uint8)
                    scales[x][dst, h] = s


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("hkv", [2, 20])  # 6 and 60 (sequence, head) pairs
def test_lost_tokens_are_zeros_and_lost_pages_left_out(kv, hkv):
    c = A.make(kv, LENS, [1] * 3, hkv, hkv, 64, seed=hkv, junk=False)
    nb = c["k"].shape[0]
    pool = nb + 6
    g = torch.Generator().manual_seed(hkv)

    def grown(t, fill):
        return None if t is None else torch.cat((t, torch.full((pool - nb, *t.shape[1:]), fill, dtype=t.dtype)))
    caches = [grown(c["k"], 0x31), grown(c["v"], 0x32)]
    sums = -torch.rand(pool, hkv, 16, generator=g) - 0.5  # below 0: what counts as 0 stands above all of them
    fresh = torch.arange(nb, pool, dtype=torch.int32).view(3, 2)
    fresh[0, 0], fresh[2, 1] = -3, pool
    table = c["table"].clone()
    for b, col in LOST:
        table[b, col] = 1 << 29 if b else -5
    scales = [grown(c["k_scale"], 0.5), grown(c["v_scale"], 0.25)] if kv == "e4m3" else []
    (_, k, v, table_d, lens), _ = on_gpu({**c, "k": caches[0], "v": caches[1], "table": table, "k_scale": None, "v_scale": None,
                                          "q": torch.zeros(3, hkv, 64, dtype=torch.bfloat16)})
    w = sums.cuda()
    given = {"k_scale": scales[0].cuda(), "v_scale": scales[1].cuda()} if scales else {}
    got = pa.evict(k, v, w, table_d, lens, fresh.cuda(), KEEP, sinks=1, recent=3, head_dim=64, **given)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert got.tolist() == [KEEP] * 3
    _move(c, caches, sums, scales, table, fresh, 1, 3)
    for now, want in ((k, caches[0]), (v, caches[1]), (w, sums), *zip(given.values(), scales)):
        assert torch.equal(now.cpu().view(torch.uint8), want.view(torch.uint8))
    # the lost block's sixteen tokens of sequence 1 are all there, as zeros
    if kv == "bf16":
        moved = k[fresh[1].long().cuda()].transpose(1, 2).flatten(0, 1)  # [32, Hkv, d]
        assert ((moved == 0).all(-1).sum(0) == 16).all()
    if kv == "fp4":
        codes = plain.fp4_unpack(k[fresh[1].long().cuda()].cpu().numpy(), 64)[0]
        assert codes.shape[0] == 2 and ((codes == 0).all(-1).sum((0, 2)) == 16).all()
