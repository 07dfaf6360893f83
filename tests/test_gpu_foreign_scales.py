"""E4M3 caches in which every block that no row sees holds non-finite scales and codes, block 0 among them:
blocks never used, or owned by a request whose values overflowed.  No form may take anything from them."""

import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def foreign(c, scale):
    """The case with a block 0 that nobody owns in front, and `scale` as both scales of every block that
    the table does not name."""
    nb, hkv = c["k"].shape[:2]
    named = torch.zeros(nb, dtype=torch.bool)
    named[c["table"][c["table"] != A.BAD_ID].long()] = True
    out = {**c, "table": torch.where(c["table"] == A.BAD_ID, c["table"], c["table"] + 1)}
    for n in "kv":
        out[n] = torch.cat((torch.full_like(c[n][:1], 0x7F), c[n]))
        s = torch.where(named[:, None], c[n + "_scale"], torch.tensor(scale))
        out[n + "_scale"] = torch.cat((torch.full((1, hkv), scale), s))
        out[n + "f"] = torch.cat((torch.zeros_like(torch.from_numpy(c[n + "f"][:1])), torch.from_numpy(c[n + "f"]))).numpy()
    return out


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("form,hq,hkv,rows,window", [
    ("decode", 8, 2, [1] * 4, None), ("decode", 6, 2, [1] * 4, None),         # warp-level kernel; 64-row tiles
    ("decode", 8, 2, [1] * 4, 50), ("decode", 6, 2, [1] * 4, 50),             # with a window
    ("verify", 8, 2, [5] * 4, None), ("verify", 16, 2, [9] * 4, None),        # 64-row tiles; split 128-row tiles
    ("verify", 8, 2, [5] * 4, 50), ("verify", 16, 2, [9] * 4, 50),            # rows kernel; split 128-row tiles
    ("prefill", 8, 2, [20, 1, 9, 130], None), ("prefill", 8, 1, [20, 1, 9, 130], 50),
])
def test_a_scale_that_no_row_sees_reaches_no_row(form, hq, hkv, rows, window, d, scale):
    lens = [n + r for n, r in zip([300, 700, 17, 129], rows)]
    c = foreign(A.make("e4m3", lens, rows, hq, hkv, d, seed=hq + d, window=window, sinks=4 if window else 0), scale)
    got = A.call(c, form)
    assert pa.check_device_errors() == pa.PA_OK
    A.check(c, form, got)
