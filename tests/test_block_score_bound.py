"""What a block's score says of its keys: never less than the rounded row's product with any of them, and at most half a code of
the row for each dim, times the key, below the row's own.  Whole numbers and powers of two: no tolerance.  Host code only."""

import os

import numpy as np
import pytest

from oracle import forms, plain

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bf16(x):
    import torch

    return plain.to_f64(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16))


def _score(row, keys):
    codes, scale = forms.block_bounds(keys)
    return forms.scores(row[None], codes[None], np.array([scale]))[0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(20))
def test_the_score_bounds_the_rounded_rows_products(d, seed):
    rng = np.random.default_rng(seed)
    keys = _bf16(rng.standard_normal((16, d)) * np.exp(rng.standard_normal(d)))
    row = _bf16(rng.standard_normal(d) * 2.0 ** rng.integers(-8, 8))
    step = 2.0 ** forms.code_exp(np.abs(row).max())
    rounded = np.rint(row / step) * step
    score = _score(row, keys)
    assert (keys @ rounded <= score + 2.0 ** -40 * np.abs(keys).sum(1)).all()  # (the right side: fp64 sums of the test's own)
    assert (keys @ row <= score + 0.5 * step * np.abs(keys).sum(1) * (1 + 2.0 ** -40)).all()


def test_the_score_can_lie_below_the_rows_own_product():
    # codes of 127 and zeros: 63 dims of 7/16 each are rounded away
    row = np.array([127.0] + [0.4375] * 63)
    keys = np.tile(np.array([0.0] + [1.0] * 63), (16, 1))
    assert _score(row, keys) == 0 < 63 * 0.4375 == (keys @ row)[0]


def test_the_header_says_so():
    text = open(os.path.join(ROOT, "include", "paged_attn.h"), encoding="utf-8").read()
    at = text.index("int paged_attn_select_blocks(")
    note = " ".join(text[text.rindex("/*", 0, at): at].replace("\n *", " ").split())
    assert "upper bound of their scores" not in note
    assert "half a code" in note
