"""Calls with no sequence, no row and no token: nothing to do, and no error."""

import pytest
import torch

import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

CACHES = {"bf16": (torch.bfloat16, 128), "e4m3": (torch.uint8, 128), "fp4": (torch.uint8, 72)}


@pytest.mark.parametrize("window", [None, 100])
@pytest.mark.parametrize("kv", CACHES)
def test_attention_and_cache(kv, window):
    dtype, last = CACHES[kv]
    k, v = (torch.zeros(3, 2, 16, last, dtype=dtype, device="cuda") for _ in "kv")
    kw = {}
    if kv == "e4m3":
        kw = {n: torch.ones(3, 2, device="cuda") for n in ("k_scale", "v_scale")}
    win = {} if window is None else {"window": window, "sinks": 4}

    def ints(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device="cuda")

    def rows(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")

    assert pa.decode(rows(0, 1, 8, 128), k, v, ints(0, 4), ints(0), 0.1, **kw, **win).shape == (0, 1, 8, 128)
    assert pa.verify(rows(0, 5, 8, 128), k, v, ints(0, 4), ints(0), 0.1, **kw, **win).shape == (0, 5, 8, 128)
    if window is None:
        assert pa.tree_verify(rows(0, 5, 8, 128), k, v, ints(0, 4), ints(0), ints(0, 5), 0.1, **kw).shape == (0, 5, 8, 128)
    assert pa.prefill(rows(0, 8, 128), k, v, ints(0, 4), ints(0), ints(1), 0.1, **kw, **win).shape == (0, 8, 128)
    # sequences without rows, and rows behind no sequence
    assert pa.prefill(rows(0, 8, 128), k, v, ints(2, 4), ints(2), ints(3), 0.1, **kw, **win).shape == (0, 8, 128)
    out = rows(3, 8, 128) + 5
    assert (pa.prefill(rows(3, 8, 128), k, v, ints(0, 4), ints(0), ints(1), 0.1, out=out, **kw, **win) == 5).all()
    pa.append_kv(rows(0, 3, 2, 128), rows(0, 3, 2, 128), k, v, ints(0, 4), ints(0), **kw)
    pa.append_kv(rows(2, 0, 2, 128), rows(2, 0, 2, 128), k, v, ints(2, 4), ints(2), **kw)
    assert pa.read_kv(k, v, ints(0, 4), ints(0), 3, **kw)[0].shape == (0, 3, 2, 128)
    assert pa.read_kv(k, v, ints(2, 4), ints(2), 0, **kw)[1].shape == (2, 0, 2, 128)
    assert (k == 0).all() and (v == 0).all() and pa.check_device_errors() == pa.PA_OK


def test_norm_rotation_and_acceptance():
    q, k = (torch.zeros(0, h, 128, dtype=torch.bfloat16, device="cuda") for h in (8, 2))
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    got = pa.qk_norm_rope(q, k, w, w, torch.ones(4, 128, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"))
    assert got[0].shape == q.shape and got[1].shape == k.shape
    empty = [torch.zeros(*s, dtype=t, device="cuda") for s, t in (((0, 4, 50), torch.float32), ((0, 3, 50), torch.float32),
                                                                  ((0, 3), torch.int32), ((0, 3), torch.float32), ((0,), torch.int32))]
    accepted, tokens = pa.spec_accept(*empty)
    assert accepted.shape == (0,) and tokens.shape == (0, 4)
    assert pa.check_device_errors() == pa.PA_OK
