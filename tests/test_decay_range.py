"""paged_attn_weighted_decode takes every finite decay and no other; no call here reaches a GPU."""

import pytest

import paged_kv_gqa_attn_gb300 as pa
from test_sparse_operator_checks import FAKE, _attn

MOST = (2 - 2.0 ** -23) * 2.0 ** 127


@pytest.mark.parametrize("decay,status", [
    (MOST, pa.PA_OK), (-MOST, pa.PA_OK), (2.0 ** -149, pa.PA_OK), (-0.0, pa.PA_OK),
    (float("inf"), pa.PA_ERR_INVALID_ARG), (float("-inf"), pa.PA_ERR_INVALID_ARG), (float("nan"), pa.PA_ERR_INVALID_ARG),
    (2.0 ** 128, pa.PA_ERR_INVALID_ARG),  # (an infinity as an fp32 number)
])
def test_every_finite_decay(decay, status):
    assert _attn("weighted_decode", lead=(FAKE,), tail=(decay,)) == status
