"""Selection flags a block id that is not there whatever the context's length: where every block is taken, and none is scored,
as where the highest are."""

import pytest
import torch

import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def _select(lens, bad, count, seqs=1):
    """The lists of `seqs` copies of the lengths, over a table whose entry `bad` of the first row is not there."""
    g = torch.Generator().manual_seed(1)
    width, nb, hkv, d = -(-max(lens) // 16), 40, 2, 64
    table = torch.randint(0, nb, (len(lens) * seqs, width), generator=g).int()
    if bad is not None:
        table[0, bad[0]] = bad[1]
    q = torch.randn(len(table), 1, 4, d, generator=g).to(torch.bfloat16)
    codes = torch.randint(-127, 128, (nb, hkv, 2, d), generator=g).to(torch.int8)
    codes[:, :, 0] = torch.maximum(codes[:, :, 0], codes[:, :, 1])
    return pa.select_blocks(q.cuda(), codes.cuda(), torch.ones(nb, hkv, device="cuda"), table.cuda(),
                            torch.tensor(lens * seqs, dtype=torch.int32, device="cuda"), count).cpu()


@pytest.mark.parametrize("seqs", [1, 200])  # few lists: one kernel; many of long contexts: two
@pytest.mark.parametrize("bad", [(0, -1), (1, 40), (2, 1 << 29), (2, -2 ** 31)])
def test_a_short_context(bad, seqs):
    lens = [40, 100] if seqs == 1 else [40, 17000]
    got = _select(lens, bad, 8 if seqs == 1 else 1100, seqs)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert got[0, 0].tolist()[:5] == [0, 1, 2, -1, -1]
    assert torch.equal(got, _select(lens, None, got.shape[2], seqs))
    assert pa.check_device_errors() == pa.PA_OK


def test_entries_past_the_context_are_not_looked_at():
    for last in (3, 6):
        _select([40, 100], (last, -7), 8)
        assert pa.check_device_errors() == pa.PA_OK
