"""Every form gives the same bits again: nothing depends on the order in which CTAs run."""

import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("window", [None, 700])
@pytest.mark.parametrize("form,hq,hkv,rows", [("decode", 8, 2, [1] * 5), ("decode", 6, 2, [1] * 5), ("verify", 8, 2, [5] * 5),
                                              ("verify", 16, 2, [9] * 5), ("prefill", 8, 2, [300, 40, 1, 700, 129])])
def test_the_same_bits_again(form, hq, hkv, rows, window, kv):
    lens = [n + r for n, r in zip([3000, 1, 17, 900, 2000], rows)]
    c = A.make(kv, lens, rows, hq, hkv, 128, seed=hq, window=window, sinks=4 if window else 0)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    want = A.call(dev, form)
    for _ in range(20):
        assert torch.equal(A.call(dev, form), want)
    assert pa.check_device_errors() == pa.PA_OK
