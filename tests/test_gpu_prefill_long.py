"""Prefill of one sequence with more than 32768 tiles of new rows: the tile's number fills its half of the
work item."""

import pytest
import torch

import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_more_than_32768_tiles_of_one_sequence(kv):
    hq, d, window, sinks, prefix, guard = 8, 64, 90, 4, 24, 64  # groups of 8: 16 new tokens a tile
    rows = 32768 * 16 + 37
    n = prefix + rows
    g = torch.Generator(device="cuda").manual_seed(7)
    nb = (n + 15) // 16
    table = torch.randperm(nb, generator=g, device="cuda").int()[None].contiguous()
    k = torch.randn(nb, 1, 16, d, generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn(nb, 1, 16, d, generator=g, device="cuda", dtype=torch.bfloat16)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    if kv == "fp4":
        caches = [torch.zeros(nb, 1, 16, 9 * d // 16, dtype=torch.uint8, device="cuda") for _ in "kv"]
        order = table[0].long()
        rowsof = [x[order].transpose(1, 2).reshape(1, nb * 16, 1, d)[:, :n].contiguous() for x in (k, v)]
        pa.append_kv(*rowsof, *caches, table, lens)
        kf, vf = (x[0, :, 0].double() for x in pa.read_kv(*caches, table, lens, n))
    else:
        caches = [k, v]
        kf, vf = (x[table[0].long()].reshape(nb * 16, d)[:n].double() for x in (k, v))
    # rows in front of and behind the sequence's own, which no write may reach
    q_all = torch.randn(rows + 2 * guard, hq, d, generator=g, device="cuda", dtype=torch.bfloat16)
    out_all = torch.full_like(q_all, 3.0)
    q, out = q_all[guard: guard + rows], out_all[guard: guard + rows]
    out.fill_(float("nan"))
    starts = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    pa.prefill(q, *caches, table, lens, starts, d ** -0.5, max_q_len=rows, window=window, sinks=sinks, out=out)
    assert pa.check_device_errors() == pa.PA_OK
    assert (out_all[:guard] == 3).all() and (out_all[guard + rows:] == 3).all()
    assert bool(torch.isfinite(out).all())
    tile = 16
    for i in [0, 1, 15, 16, 200, 32767 * tile - 1, 32767 * tile, 32768 * tile - 1, 32768 * tile, 32768 * tile + 21, rows - 1]:
        own = prefix + i
        seen = torch.tensor(sorted(set(range(min(sinks, own + 1))) | set(range(max(0, own + 1 - window), own + 1))),
                            device="cuda")
        x = q[i].double() @ kf[seen].T * d ** -0.5
        p = torch.softmax(x, -1)
        want = p @ vf[seen]
        # rounding of the output 2^-8, of the weights and of the sum that divides them 2^-8 each (bf16), 2^-11 (f16);
        # scores: 64 products in fp32
        score = 2 * d * 2.0 ** -24 * float((q[i].double().abs() @ kf[seen].abs().T).max()) * d ** -0.5
        bound = 2.0 ** -8 * want.abs() + ((2.0 ** -7 if kv == "bf16" else 2.0 ** -11) + 2 * score) * (p @ vf[seen].abs())
        floor = len(seen) * 2.0 ** -25 * vf[seen].abs().max()  # f16 weights below 2^-14
        over = (out[i].double() - want).abs() - bound - floor
        assert float(over.max()) <= 0, (i, float(over.max()))
