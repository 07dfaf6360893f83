"""paged_attn_plan answers for what it can know: 4-bit decode, and not 4-bit verify."""

import pytest

import paged_kv_gqa_attn_gb300 as pa


@pytest.mark.parametrize("parts", [0, 3])
def test_4_bit_verify_is_refused(parts):
    pa.set_max_partitions(parts)
    try:
        for q_len in (2, 5, 16):
            with pytest.raises(pa.PagedAttnError) as e:
                pa.plan(152, 32, 8, 8192, q_len=q_len, kv_dtype=pa.PA_KV_FP4_E2M1)
            assert e.value.status == pa.PA_ERR_UNSUPPORTED
    finally:
        pa.set_max_partitions(0)


def test_decode_plans_are_as_they_were():
    for shape, want in (((152, 1, 8, 8208), 513), ((152, 64, 8, 32768), 2048), ((152, 512, 8, 2048), 128)):
        per, parts = pa.plan(*shape, kv_dtype=pa.PA_KV_FP4_E2M1)
        # sqrt(pages * 4 CTAs of each SM / (38 * units)), at least 1 and at most 64
        units, P = shape[1] * shape[2], 1
        while (P + 1) ** 2 <= want * 152 * 4 / (38 * units) and P < 64:
            P += 1
        assert per == -(-want // P) and parts == -(-want // per)
    assert pa.plan(152, 64, 8, 2048, q_len=5) == pa.plan(152, 64, 8, 2048)
