"""The 4-bit cache on the GPU: append_kv bit for bit against the plain form (codes and scales), read_kv
for every cache type, untouched slots, bad tables, side streams and graphs."""

import numpy as np
import pytest
import torch

from oracle import plain
import paged_kv_gqa_attn_gb300 as pa
from paged_kv_gqa_attn_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def _rows(lens, n, hkv, d, seed, mag=1.0):
    g = torch.Generator().manual_seed(seed)
    table, nb = W.allocate_block_tables(lens, 16, seed=seed)
    k = (torch.randn(len(lens), n, hkv, d, generator=g) * mag).to(torch.bfloat16)
    v = (torch.randn(len(lens), n, hkv, d, generator=g) * mag).to(torch.bfloat16)
    return k, v, table, nb, torch.tensor(lens, dtype=torch.int32)


def _stored(cache, new, table, lens, s, d):
    """The plain form of the append: cache bytes after it."""
    codes, scales = plain.fp4_unpack(cache.numpy(), d)
    codes, scales = codes.copy(), scales.copy()
    c, sc = plain.fp4_encode(new.float().numpy(), s)
    for b, n_all in enumerate(lens.tolist()):
        for t in range(new.shape[1]):
            j = n_all - new.shape[1] + t
            blk = int(table[b, j // 16])
            codes[blk, :, j % 16], scales[blk, :, j % 16] = c[b, t], sc[b, t]
    return plain.fp4_pack(codes, scales)


@pytest.mark.parametrize("lens,n,hkv,d", [
    ([1], 1, 1, 64),
    ([20, 33, 16, 1], 1, 2, 128),
    ([37, 64, 18, 5, 100], 5, 4, 128),
    ([40, 32, 17], 16, 2, 64),
    ([300, 77, 65], 65, 8, 128),
    ([200, 130], 130, 1, 64),
])
@pytest.mark.parametrize("scales", ["none", "powers", "any"])
def test_append_bit_for_bit_and_read_back(lens, n, hkv, d, scales):
    k, v, table, nb, cl = _rows(lens, n, hkv, d, seed=n + d)
    g = torch.Generator().manual_seed(d)
    s = {"none": None, "powers": 2.0 ** torch.randint(-9, -4, (hkv,), generator=g).float(),
         "any": 0.001 + 0.02 * torch.rand(hkv, generator=g)}[scales]
    ref_s = np.ones(hkv, np.float32) if s is None else s.numpy()
    start = torch.randint(0, 256, (nb, hkv, 16, 9 * d // 16), generator=g, dtype=torch.uint8)
    kc, vc = start.cuda(), start.flip(0).cuda()
    more = {} if s is None else {"k_scale": s.cuda(), "v_scale": s.cuda()}
    pa.append_kv(k.cuda(), v.cuda(), kc, vc, table.cuda(), cl.cuda(), **more)
    assert pa.check_device_errors() == pa.PA_OK
    assert np.array_equal(kc.cpu().numpy(), _stored(start, k, table, cl, ref_s, d))
    assert np.array_equal(vc.cpu().numpy(), _stored(start.flip(0), v, table, cl, ref_s, d))
    rk, rv = pa.read_kv(kc, vc, table.cuda(), cl.cuda(), n, **more)
    assert pa.check_device_errors() == pa.PA_OK
    for got, new in ((rk, k), (rv, v)):
        c, sc = plain.fp4_encode(new.float().numpy(), ref_s)
        val = plain.E2M1_MAGNITUDES[c & 7] * np.where(c & 8, -1, 1) * np.repeat(plain.E4M3_VALUES[sc], 16, -1)
        want = torch.from_numpy((val.astype(np.float32) * ref_s[:, None]).astype(np.float32)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)


def test_append_extremes():
    hkv, d = 2, 64
    x = torch.zeros(1, 6, hkv, d)
    x[0, 0] = 1e-30                                  # scale underflows: zeros
    x[0, 1] = 1e30                                   # scale and codes saturate
    x[0, 2, :, ::3] = float("inf")
    x[0, 3, :, 5] = float("nan")
    x[0, 4] = torch.linspace(-6, 6, d) * 448          # the format's full range with s = 1
    x[0, 5, :, :16] = -torch.tensor([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6])  # ties
    x = x.to(torch.bfloat16)
    kc = torch.zeros(1, hkv, 16, 9 * d // 16, dtype=torch.uint8).cuda()
    vc = kc.clone()
    table, lens = torch.zeros(1, 1, dtype=torch.int32).cuda(), torch.tensor([6], dtype=torch.int32).cuda()
    pa.append_kv(x.cuda(), x.flip(1).cuda(), kc, vc, table, lens)
    assert pa.check_device_errors() == pa.PA_OK
    c, sc = plain.fp4_encode(x.float().numpy(), np.ones(hkv, np.float32))
    codes, scales = plain.fp4_unpack(kc.cpu().numpy(), d)
    assert np.array_equal(codes[0, :, :6], np.swapaxes(c[0], 0, 1))
    assert np.array_equal(scales[0, :, :6], np.swapaxes(sc[0], 0, 1))
    assert not codes[0, :, 6:].any() and not scales[0, :, 6:].any()


def test_short_contexts_and_bad_blocks_are_skipped_and_flagged():
    hkv, d, n = 2, 128, 3
    k, v, table, nb, _ = _rows([40, 40, 40, 40], n, hkv, d, seed=4)
    table = table.clone()
    table[1, 2] = nb
    table[2, 2] = -1
    cl = torch.tensor([40, 40, 40, 2], dtype=torch.int32)
    kc = torch.full((nb, hkv, 16, 9 * d // 16), 7, dtype=torch.uint8).cuda()
    vc = kc.clone()
    pa.append_kv(k.cuda(), v.cuda(), kc, vc, table.cuda(), cl.cuda())
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    ref = _stored(torch.full((nb, hkv, 16, 9 * d // 16), 7, dtype=torch.uint8), k[:1], table[:1], cl[:1],
                  np.ones(hkv, np.float32), d)
    assert np.array_equal(kc.cpu().numpy(), ref)
    rk, rv = pa.read_kv(kc, vc, table.cuda(), cl.cuda(), n)
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert rk[0].any() and not rk[1:3].any() and not rv[1:3].any() and not rk[3, 0].any()
    assert rk[3, 1:].any()  # the two tokens that the short sequence has


@pytest.mark.parametrize("kv", ["bf16", W.KV_FP8_E4M3])
@pytest.mark.parametrize("lens,n,hkv,d", [([1], 1, 1, 64), ([20, 33, 16], 1, 2, 128), ([300, 77, 65], 65, 8, 128),
                                          ([40, 32, 17], 16, 3, 64)])
def test_read_other_caches(kv, lens, n, hkv, d):
    p = W.make_problem(lens, hkv, hkv, d, kv_dtype=kv, seed=n + d, tail_fill="nan")
    g = p.to("cuda")
    more = {} if kv == "bf16" else {"k_scale": g.k_scale, "v_scale": g.v_scale}
    got = pa.read_kv(g.k_cache, g.v_cache, g.block_table, g.context_lens, n, **more)
    assert pa.check_device_errors() == pa.PA_OK
    for out, cache, scale in zip(got, (p.k_cache, p.v_cache), (p.k_scale, p.v_scale)):
        for b, L in enumerate(lens):
            j = torch.arange(L - n, L)
            blk = p.block_table[b].long()[j // 16]
            rows = cache[blk, :, j % 16]
            if kv != "bf16":
                rows = (rows.view(torch.float8_e4m3fn).float() * scale[blk][:, :, None]).to(torch.bfloat16)
            assert torch.equal(out[b].cpu(), rows)


def test_side_stream_and_graph():
    k, v, table, nb, cl = (t.cuda() if torch.is_tensor(t) else t for t in _rows([50, 21], 5, 4, 128, seed=8))
    kc = torch.zeros(nb, 4, 16, 72, dtype=torch.uint8, device="cuda")
    vc = kc.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pa.append_kv(k, v, kc, vc, table, cl, stream=s)
    want = pa.read_kv(kc, vc, table, cl, 5, stream=s)
    s.synchronize()
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.append_kv(k, v, kc, vc, table, cl)
        pa.read_kv(kc, vc, table, cl, 5, k_out=out[0], v_out=out[1])
    k.copy_(-k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], -want[0]) and torch.equal(out[1], want[1])


def test_refusals():
    k, v, table, nb, cl = (t.cuda() if torch.is_tensor(t) else t for t in _rows([50, 21], 5, 4, 128, seed=8))
    kc = torch.zeros(nb, 4, 16, 72, dtype=torch.uint8, device="cuda")
    s = torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        pa.append_kv(k, v, kc, kc.clone(), table, cl, k_scale=torch.ones(nb, 4, device="cuda"), v_scale=s)
    with pytest.raises(TypeError):
        pa.append_kv(k, v, kc, kc.clone(), table, cl, k_scale=s.double(), v_scale=s)
    with pytest.raises(ValueError):
        pa.append_kv(k, v, kc[:, :3].contiguous(), kc[:, :3].contiguous(), table, cl)
    with pytest.raises(ValueError):
        pa.read_kv(kc, kc.clone(), table, cl, -1)
    with pytest.raises(pa.PagedAttnError):
        pa.read_kv(kc, kc.clone(), table, cl, table.shape[1] * 16 + 1)
    with pytest.raises(ValueError):
        pa.read_kv(kc, kc.clone(), table, cl, 2, k_out=torch.empty(2, 2, 4, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        pa.read_kv(kc, kc.clone(), table, cl[:1], 2)
