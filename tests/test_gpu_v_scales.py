"""E4M3 caches with small, large, mixed and (2^-200 in fp32) zero value scales: the result is right relative to
the values, whatever their size.  The bound is the common one, proportional to the values that a row sees."""

import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

FORMS = [
    # on the warp-level instruction: decode, decode with a window, other groups and verify with a window
    ("decode", 8, 2, [1] * 4, None), ("decode", 8, 2, [1] * 4, 200),
    ("decode", 6, 2, [1] * 4, 200), ("verify", 8, 2, [5] * 4, 200), ("verify", 8, 1, [4] * 4, 200),
    # 64-row tiles: verify, decode of other groups
    ("verify", 8, 2, [5] * 4, None), ("decode", 6, 2, [1] * 4, None),
    # 128-row tiles: split verify and prefill, without and with a window
    ("verify", 16, 2, [9] * 4, None), ("verify", 16, 2, [9] * 4, 200),
    ("prefill", 8, 2, [20, 1, 9, 130], None), ("prefill", 8, 1, [20, 1, 9, 130], 200),
]


def _scaled(form, hq, hkv, rows, window, d, factors):
    """A case whose value scales are multiplied by powers of two, factors[i] for block i modulo their number."""
    lens = [n + r for n, r in zip([300, 1500, 17, 700], rows)]
    c = A.make("e4m3", lens, rows, hq, hkv, d, seed=hq + d, window=window, sinks=4 if window else 0)
    f = torch.tensor([2.0 ** e for e in factors], dtype=torch.float64)[torch.arange(c["v"].shape[0]) % len(factors)]
    c["v_scale"] = (c["v_scale"].double() * f[:, None]).float()
    c["vf"] = c["vf"] * f.numpy()[:, None, None, None]
    return c


@pytest.mark.parametrize("e", [-10, -14, -20, -30, -50, -90, 14, 30, 90])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("form,hq,hkv,rows,window", FORMS)
def test_values_of_any_size(form, hq, hkv, rows, window, d, e):
    c = _scaled(form, hq, hkv, rows, window, d, [e])
    got = A.call(c, form)
    assert pa.check_device_errors() == pa.PA_OK
    A.check(c, form, got)


@pytest.mark.parametrize("parts", [0, 1])  # split as planned, and not at all
@pytest.mark.parametrize("factors", [(0, -20), (-14, -20, -26), (0, 3, -3), (-40, -41, -20), (-200, 0), (-200, -200, 40),
                                     (60, -200, -60)])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("form,hq,hkv,rows,window", FORMS)
def test_pages_of_different_sizes(form, hq, hkv, rows, window, d, factors, parts):
    c = _scaled(form, hq, hkv, rows, window, d, factors)
    pa.set_max_partitions(parts)
    try:
        got = A.call(c, form)
    finally:
        pa.set_max_partitions(0)
    assert pa.check_device_errors() == pa.PA_OK
    A.check(c, form, got)
