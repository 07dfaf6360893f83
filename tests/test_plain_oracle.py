"""Pins of the plain fp64 forms (4-bit format, window visibility, norm and rotation) on the CPU:
against the OCP tables through torch's casts, brute force, closed forms and the C oracle."""

import numpy as np
import pytest
import torch

import oracle
from oracle import plain
from paged_kv_gqa_attn_gb300 import workloads as W


def test_e4m3_table_is_torchs():
    bytes_ = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(bytes_.view(torch.float8_e4m3fn).double().numpy(), plain.E4M3_VALUES)


def test_nearest_index_rounds_ties_to_the_even_code():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.2500001, 100.0, 0.0])
    want = np.array([0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.5, 6.0, 0.0])
    assert np.array_equal(plain.E2M1_MAGNITUDES[plain.nearest_index(x, plain.E2M1_MAGNITUDES)], want)
    y = torch.rand(4096, dtype=torch.float64, generator=torch.Generator().manual_seed(1)).numpy() * 500
    got = plain.nearest_index(y.astype(np.float32).astype(np.float64), plain.E4M3_VALUES)
    ref = torch.from_numpy(np.minimum(y.astype(np.float32), 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("d", [64, 128])
def test_fp4_round_trip_and_error_bound(d):
    g = torch.Generator().manual_seed(d)
    x = torch.randn(3, 2, 16, d, generator=g).to(torch.bfloat16).double().numpy()
    s = np.array([2.0 ** -8, 2.0 ** -6], np.float32)
    cache = plain.fp4_pages(x, s)
    assert cache.shape == (3, 2, 16, 9 * d // 16)
    codes, scales = plain.fp4_unpack(cache, d)
    assert np.array_equal(plain.fp4_pack(codes, scales), cache)
    v = plain.fp4_values(cache, d, s)
    # spacing of the codes is at most 2 steps (between 4 and 6): off by one step, plus what the
    # scale's own rounding (half a step of E4M3, 2^-4 relative) can cut off the largest
    step = np.repeat(plain.E4M3_VALUES[scales] * s[None, :, None, None], 16, axis=-1)
    assert (np.abs(v - x) <= step * (1 + 6 * 2.0 ** -4)).all()
    # values that are codes already are stored exactly
    again = plain.fp4_values(plain.fp4_pages(v, s), d, s)
    assert np.abs(again - v).max() <= np.abs(v).max() * 2.0 ** -3
    zero = plain.fp4_pages(np.zeros((1, 2, 16, d)), s)
    assert not zero.any()


def test_window_visibility_by_brute_force():
    for n in (1, 5, 40):
        for window in (1, 3, 40, 100):
            for sinks in (0, 1, 4, 60):
                got = plain.sees(n, np.arange(64), window, sinks)
                want = [j < n and (n - 1 - j < window or j < sinks) for j in range(64)]
                assert got.tolist() == want


@pytest.mark.parametrize("q_len", [1, 5])
def test_attend_without_a_window_is_the_c_oracle(q_len):
    p = W.make_problem([q_len, 40, 130], 8, 2, 64, q_len=q_len, seed=11)
    ref = oracle.attention_problem(p)
    got = plain.attend(p.q.flatten(0, 1), plain.to_f64(p.k_cache), plain.to_f64(p.v_cache), p.block_table.numpy(),
                       p.context_lens.tolist(), [q_len] * 3, p.scale)
    assert np.abs(got.reshape(ref.shape) - ref).max() < 1e-12
    wide = plain.attend(p.q.flatten(0, 1), plain.to_f64(p.k_cache), plain.to_f64(p.v_cache), p.block_table.numpy(),
                        p.context_lens.tolist(), [q_len] * 3, p.scale, window=130, sinks=2)
    assert np.array_equal(wide, got)


def test_attend_window_of_one_is_the_tokens_own_value():
    p = W.make_problem([7, 33], 4, 2, 64, seed=12)
    v = plain.to_f64(p.v_cache)
    got = plain.attend(p.q[:, 0], plain.to_f64(p.k_cache), v, p.block_table.numpy(), [7, 33], [1, 1], p.scale, window=1)
    for b, n in enumerate((7, 33)):
        own = v[int(p.block_table[b, (n - 1) // 16]), :, (n - 1) % 16]
        assert np.allclose(got[b].reshape(2, 2, 64), own[:, None], rtol=0, atol=0)


def test_norm_rope_rotates_by_the_angle_and_keeps_the_norm():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 2, 64, generator=g, dtype=torch.float64)
    pos = np.array([0, 1, 7, 100, 3])
    for inter in (False, True):
        freq = 100.0 ** (-np.arange(0, 32, 2) / 32)
        ang = np.arange(128)[:, None] * freq
        cs = np.concatenate((np.cos(ang), np.sin(ang)), 1)
        y = plain.norm_rope(x, np.ones(64), cs, pos, 0.0, inter)
        assert np.allclose((y * y).mean(-1), 1)  # the norm's own scale, kept by the rotation
        base = plain.norm_rope(x, np.ones(64), cs, np.zeros(5, int), 0.0, inter)
        assert np.array_equal(base[0], y[0]) and np.array_equal(base[..., 32:], y[..., 32:])
        a, b = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if inter else (np.arange(16), np.arange(16, 32))
        z0, z1 = base[..., a] + 1j * base[..., b], y[..., a] + 1j * y[..., b]
        assert np.allclose(z1, z0 * np.exp(1j * ang[pos])[:, None])
