"""E4M3 pages of the smallest numbers, on the GPU: where amax / 448 is no fp32 number but zero, the rows that an append or an
eviction re-encodes keep their values.  Every value here is a code times 2^-149, which its new page holds exactly."""

import pytest
import torch

import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -149
CODES = torch.tensor([0.0, 1.0, -1.0, 2.0, -3.0]).to(torch.float8_e4m3fn).view(torch.uint8)


def _pages(n, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    codes = CODES[torch.randint(0, 5, (n, hkv, 16, d), generator=g)]
    codes[..., 0] = CODES[1]  # (no page of zeros)
    return codes, torch.full((n, hkv), TINY)


def _values(codes, scale):
    """Multiples of 2^-149, whole numbers in fp64."""
    return codes.cpu().view(torch.float8_e4m3fn).double() * (scale.cpu().double() / TINY)[..., None, None]


@pytest.mark.parametrize("hkv", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_evicted_pages(hkv, d):
    k, ks = _pages(6, hkv, d, 1)
    v, vs = _pages(6, hkv, d, 2)
    table = torch.tensor([[2, 0, 4]], dtype=torch.int32)
    args = [t.cuda() for t in (k, v, torch.zeros(6, hkv, 16), table, torch.tensor([48], dtype=torch.int32))]
    scales = {"k_scale": ks.cuda(), "v_scale": vs.cuda()}
    got = pa.evict(*args, torch.tensor([[5, 1]], dtype=torch.int32).cuda(), 32, recent=32, **scales)
    assert got.tolist() == [32] and pa.check_device_errors() == pa.PA_OK
    for new, old, scale, before in ((args[0], k, scales["k_scale"], ks), (args[1], v, scales["v_scale"], vs)):
        assert torch.equal(_values(new, scale)[[5, 1]], _values(old, before)[[0, 4]])


@pytest.mark.parametrize("d", [64, 128])
def test_an_appended_row_of_zeros(d):
    k, ks = _pages(2, 2, d, 3)
    v, vs = _pages(2, 2, d, 4)
    dev = [t.cuda() for t in (k, v)]
    scales = {"k_scale": ks.cuda(), "v_scale": vs.cuda()}
    zeros = torch.zeros(1, 1, 2, d, dtype=torch.bfloat16, device="cuda")
    pa.append_kv(zeros, zeros, *dev, torch.tensor([[1]], dtype=torch.int32).cuda(),
                 torch.tensor([9], dtype=torch.int32).cuda(), **scales)
    assert pa.check_device_errors() == pa.PA_OK
    for new, old, scale, before in ((dev[0], k, scales["k_scale"], ks), (dev[1], v, scales["v_scale"], vs)):
        now, was = _values(new, scale)[1], _values(old, before)[1]
        assert torch.equal(now[:, :8], was[:, :8]) and (now[:, 8] == 0).all()
