"""qk_norm_rope on the GPU against the plain fp64 form: head counts, both head dims, partial and
interleaved rotation, strided and in-place rows, far positions, bad positions, streams and graphs.

Tolerance.  The result is rounded to bf16 once: at most half a step, 2^-8 of the value.  Before it,
fp32: the sum of d <= 128 squares (error at most 7 + 8 roundings of positive terms), its root
(2 units), two products, then two products and a sum for the rotation: under 32 roundings of 2^-24
of the pair's size |y_a| + |y_b|, 2^-18.6 with a factor of 1.3 to spare."""

import numpy as np
import pytest
import torch

from oracle import plain
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def _table(positions, rotary, base=10000.0):
    ang = np.arange(positions)[:, None] * base ** (-np.arange(0, rotary, 2) / rotary)
    return torch.from_numpy(np.concatenate((np.cos(ang), np.sin(ang)), 1)).float()


def _make(T, hq, hkv, d, rotary, seed, positions=512, mag=3.0):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(T, hq, d, generator=g) * mag).to(torch.bfloat16)
    k = (torch.randn(T, hkv, d, generator=g) * mag).to(torch.bfloat16)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, positions, (T,), generator=g, dtype=torch.int32)
    return q, k, w[0], w[1], _table(positions, rotary), pos


def _bound(x, w, rotary, interleaved, ref, eps):
    """2^-8 of the value plus 2^-18.6 of the pair's size."""
    y = np.abs(plain.norm_rope(x, w, torch.tensor([[1.0] * (rotary // 2) + [0.0] * (rotary // 2)]),
                               np.zeros(len(x), int), eps, interleaved))
    size = y.copy()
    if interleaved:
        size[..., :rotary] = np.repeat(y[..., 0:rotary:2] + y[..., 1:rotary:2], 2, -1)
    else:
        both = y[..., : rotary // 2] + y[..., rotary // 2: rotary]
        size[..., :rotary] = np.concatenate((both, both), -1)
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -18.6 * size + 1e-38


def _check(args, eps=1e-6, interleaved=False, got=None):
    q, k, qw, kw, cs, pos = args
    if got is None:
        got = pa.qk_norm_rope(*(t.cuda() for t in args), eps=eps, interleaved=interleaved)
        assert pa.check_device_errors() == pa.PA_OK
    for x, w, y in ((q, qw, got[0]), (k, kw, got[1])):
        ref = plain.norm_rope(x, w, cs, pos.numpy(), eps, interleaved)
        off = np.abs(plain.to_f64(y) - ref)
        bound = _bound(x, w, cs.shape[1], interleaved, ref, eps)
        assert (off <= bound).all(), (off - bound).max()


@pytest.mark.parametrize("T", [1, 2, 7, 129])
@pytest.mark.parametrize("hq,hkv,d,rotary", [(32, 8, 128, 128), (8, 1, 64, 64), (28, 4, 128, 64), (1, 1, 64, 16),
                                             (64, 8, 128, 112), (5, 5, 64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_matches_the_definition(T, hq, hkv, d, rotary, interleaved):
    _check(_make(T, hq, hkv, d, rotary, seed=T + hq + d), interleaved=interleaved)


def test_tiny_large_and_zero_rows():
    q, k, qw, kw, cs, pos = _make(6, 4, 2, 128, 128, seed=5)
    q[0] *= 1e-18
    q[1] *= 1e15
    q[2] = 0
    k[3] = 0
    _check((q, k, qw, kw, cs, pos))
    _check((q[2:], k[2:], qw, kw, cs, pos[2:]), eps=1e-3)


def test_strided_rows_and_in_place():
    T, hq, hkv, d = 9, 8, 2, 128
    args = _make(T, hq, hkv, d, 128, seed=6)
    packed = torch.cat((args[0].flatten(1), args[1].flatten(1), torch.zeros(T, hkv * d, dtype=torch.bfloat16)), 1).cuda()
    keep = packed.clone()
    q = packed[:, : hq * d].unflatten(1, (hq, d))
    k = packed[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d))
    rest = [t.cuda() for t in args[2:]]
    plain_out = pa.qk_norm_rope(q, k, *rest)
    assert torch.equal(packed, keep)
    _check(args, got=plain_out)
    out = pa.qk_norm_rope(q, k, *rest, q_out=q, k_out=k)
    assert out[0].data_ptr() == q.data_ptr()
    assert torch.equal(out[0], plain_out[0]) and torch.equal(out[1], plain_out[1])
    assert torch.equal(packed[:, (hq + hkv) * d:], keep[:, (hq + hkv) * d:])


def test_bad_positions_are_zeroed_and_flagged():
    args = list(_make(4, 4, 2, 64, 64, seed=7, positions=100))
    args[5] = torch.tensor([3, -1, 100, 99], dtype=torch.int32)
    q, k = pa.qk_norm_rope(*(t.cuda() for t in args))
    assert pa.check_device_errors() == pa.PA_ERR_DEVICE_BOUNDS
    assert not q[1:3].any() and not k[1:3].any()
    good = [args[0][[0, 3]], args[1][[0, 3]], *args[2:5], args[5][[0, 3]]]
    _check(good, got=(q[[0, 3]], k[[0, 3]]))
    assert pa.check_device_errors() == pa.PA_OK


def test_non_finite_rows_stay_in_their_row():
    args = list(_make(3, 4, 2, 128, 128, seed=8))
    args[0][1, 2, 5] = float("nan")
    args[1][2, 0, 7] = float("inf")
    q, k = pa.qk_norm_rope(*(t.cuda() for t in args))
    assert torch.isnan(q[1, 2]).all() and not torch.isnan(k[2, 1]).any()
    keep = torch.ones(3, 4, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.isfinite(q.cpu()[keep]).all()


def test_no_tokens_and_a_side_stream_and_a_graph():
    args = [t.cuda() for t in _make(33, 32, 8, 128, 128, seed=9)]
    empty = pa.qk_norm_rope(args[0][:0], args[1][:0], *args[2:5], args[5][:0])
    assert empty[0].shape == (0, 32, 128)
    want = pa.qk_norm_rope(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = pa.qk_norm_rope(*args, stream=s)
    s.synchronize()
    assert torch.equal(side[0], want[0]) and torch.equal(side[1], want[1])
    out = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.qk_norm_rope(*args, q_out=out[0], k_out=out[1])
    args[0].copy_(args[0].flip(0))
    args[5].copy_(args[5].flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0].flip(0))


def test_refusals():
    q, k, qw, kw, cs, pos = (t.cuda() for t in _make(4, 4, 2, 64, 64, seed=10))
    with pytest.raises(TypeError):
        pa.qk_norm_rope(q.float(), k, qw, kw, cs, pos)
    with pytest.raises(TypeError):
        pa.qk_norm_rope(q, k, qw.float(), kw, cs, pos)
    with pytest.raises(TypeError):
        pa.qk_norm_rope(q, k, qw, kw, cs, pos.long())
    with pytest.raises(TypeError):
        pa.qk_norm_rope(q, k.cpu(), qw, kw, cs, pos)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(q, k[:3], qw, kw, cs, pos)
    with pytest.raises(ValueError):
        pa.qk_norm_rope(q.transpose(1, 2), k, qw, kw, cs, pos)
    with pytest.raises(pa.PagedAttnError):
        pa.qk_norm_rope(q, k, qw, kw, cs[:, :24].contiguous(), pos)  # rotary_dim 24
    with pytest.raises(pa.PagedAttnError):
        pa.qk_norm_rope(q, k, qw, kw, cs, pos, eps=-1.0)
    with pytest.raises(pa.PagedAttnError):
        pa.qk_norm_rope(  # head_dim 32
            q[..., :32].contiguous(), k[..., :32].contiguous(), qw[:32], kw[:32], cs[:, :32].contiguous(), pos)
