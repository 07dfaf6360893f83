"""The rows kernel (a few rows per kv head: windowed verify, windowed decode of other groups, 4-bit decode and
verify) at the precision that it has of its own, not the tile kernels'."""

import numpy as np
import pytest

import attn_cases as A
from oracle import plain
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def check_rows(c, form, got):
    """The bound, element by element:
      2^-8 |out|            the output's rounding to bf16;
      w sum p |v|           the weights: bf16 pages take a weight as two bf16 parts, the second's rounding 2^-8 of a
                            rounding of 2^-8, 2^-16; byte pages take f16 weights, 2^-11; for both the exponential and
                            the log2 of a page's scale are good to 2^-20;
      2 score sum p |v|     twice the error of a score: fp32 sums of d products of keys and a q that f16 holds exactly
                            (bf16 has 8 bits; after the row's power of two f16 keeps 8 bits over 2^29 below its
                            largest, and 2^-39 of it below that), d 2^-24 sum |q k|, doubled for the exponent's;
      n 2^-25 max |v|       f16 weights below 2^-14 lose absolute 2^-25, n of them."""
    ref, spread, dots = plain.attend(c["q"], c["kf"], c["vf"], c["table"].numpy(), c["lens"], c["rows"], c["scale"],
                                     c["window"], c["sinks"], sizes=True)
    byte = c["kv"] != "bf16"
    w = (2.0 ** -11 if byte else 2.0 ** -16) + 2.0 ** -20
    score = (2 * c["d"] * 2.0 ** -24 + 2.0 ** -38) * dots
    floor = max(c["lens"]) * 2.0 ** -25 * np.abs(c["vf"][np.isfinite(c["vf"])]).max() if byte else 0
    got = plain.to_f64(got)
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + (w + 2 * score) * spread + floor + 1e-30)
    assert (over <= 0).all(), (form, over.max(), int((over > 0).sum()))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("form,hq,hkv,r", [("verify", 8, 2, 4), ("verify", 8, 2, 2), ("verify", 4, 4, 9), ("decode", 6, 2, 1),
                                           ("decode", 10, 2, 1), ("verify", 8, 2, 8), ("verify", 8, 1, 3)])
@pytest.mark.parametrize("window,sinks", [(40, 4), (1500, 0)])
def test_windowed_rows(kv, d, form, hq, hkv, r, window, sinks):
    if kv == "bf16" and r * hq // hkv > 16:
        pytest.skip("bf16 pages take the tile kernel beyond 16 rows")
    lens = [n + r for n in (0, 17, 333, 2000)]
    c = A.make(kv, lens, [r] * 4, hq, hkv, d, seed=hq + r + d, window=window, sinks=sinks, k_mag=2.0)
    got = A.call(c, form)
    assert pa.check_device_errors() == pa.PA_OK
    check_rows(c, form, got)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("form,hq,hkv,r", [("decode", 8, 2, 1), ("decode", 5, 1, 1), ("verify", 8, 2, 5), ("verify", 16, 2, 4)])
def test_4_bit_rows(d, form, hq, hkv, r):
    lens = [n + r for n in (0, 17, 333, 2000)]
    c = A.make("fp4", lens, [r] * 4, hq, hkv, d, seed=hq + r + d, k_mag=2.0)
    got = A.call(c, form)
    assert pa.check_device_errors() == pa.PA_OK
    check_rows(c, form, got)
