"""Plain fp64 forms of the window attention, the 4-bit cache and the norm and rotation (numpy).

TEST INFRASTRUCTURE ONLY, as the rest of this package.  Everything is written from the definitions:
attention row by row over an explicit visibility mask, the 4-bit format by nearest-value search in the
OCP value tables.  The roundings that the format fixes (fp32 quotients before each search) are taken in
fp32; everything else is fp64.
"""

from __future__ import annotations

import numpy as np

BLOCK = 16
E2M1_MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _e4m3_table():
    """Values of the bytes 0 .. 126 (the finite non-negative ones), from the OCP definition."""
    out = []
    for byte in range(127):
        e, m = byte >> 3, byte & 7
        out.append((m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(out)


E4M3_VALUES = _e4m3_table()


def to_f64(t):
    """torch tensor (any float type) or array -> fp64 numpy."""
    if hasattr(t, "detach"):
        t = t.detach().cpu().double().numpy()
    return np.asarray(t, dtype=np.float64)


def nearest_index(x, table):
    """Index of the nearest table value (ascending), ties to the even index, saturating at the last."""
    x = np.minimum(x, table[-1])
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    up, down = table[hi] - x, x - table[lo]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)


def fp4_encode(x, s):
    """x [..., Hkv, d] (values exactly representable in fp32), s [Hkv] fp32 -> (codes [..., Hkv, d]
    in 0..15, scale bytes [..., Hkv, d / 16])."""
    x = np.asarray(x, dtype=np.float32)
    xb = x.reshape(*x.shape[:-1], -1, 16)
    s = np.asarray(s, dtype=np.float32)[:, None]
    with np.errstate(all="ignore"):
        amax = np.nanmax(np.where(np.isnan(xb), 0, np.abs(xb)), axis=-1).astype(np.float32)
        want = (amax / (np.float32(6) * s)).astype(np.float32)
        scale = nearest_index(want.astype(np.float64), E4M3_VALUES)
        step = (E4M3_VALUES[scale].astype(np.float32) * s).astype(np.float32)[..., None]
        y = np.where(step > 0, xb / np.where(step > 0, step, 1), 0).astype(np.float32)
    nan = np.isnan(y)
    mag = nearest_index(np.where(nan, 6, np.abs(y)).astype(np.float64), E2M1_MAGNITUDES)
    sign = np.signbit(y) & ~nan & (step > 0)
    return (mag + 8 * sign).reshape(x.shape).astype(np.uint8), scale.astype(np.uint8)


def fp4_pages(values, s):
    """values [NB, Hkv, 16, d] -> 4-bit cache bytes [NB, Hkv, 16, 9 d / 16]."""
    nb, hkv, bs, d = values.shape
    codes, scales = fp4_encode(np.swapaxes(np.asarray(values, np.float32), 1, 2), s)
    return fp4_pack(np.swapaxes(codes, 1, 2), np.swapaxes(scales, 1, 2))


def fp4_pack(codes, scales):
    """codes [NB, Hkv, 16, d], scale bytes [NB, Hkv, 16, d / 16] -> cache bytes."""
    nb, hkv, bs, d = codes.shape
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    flat = np.concatenate((packed.reshape(nb, hkv, -1), scales.reshape(nb, hkv, -1)), axis=-1)
    return np.ascontiguousarray(flat.reshape(nb, hkv, bs, d * 9 // 16))


def fp4_unpack(cache, d):
    """Cache bytes -> (codes [NB, Hkv, 16, d], scale bytes [NB, Hkv, 16, d / 16])."""
    cache = np.asarray(cache, dtype=np.uint8)
    nb, hkv = cache.shape[:2]
    flat = cache.reshape(nb, hkv, -1)
    packed = flat[..., : BLOCK * d // 2].reshape(nb, hkv, BLOCK, d // 2)
    codes = np.stack((packed & 15, packed >> 4), axis=-1).reshape(nb, hkv, BLOCK, d)
    return codes, flat[..., BLOCK * d // 2:].reshape(nb, hkv, BLOCK, d // 16)


def fp4_values(cache, d, s):
    """Cache bytes -> fp64 values [NB, Hkv, 16, d]."""
    codes, scales = fp4_unpack(cache, d)
    mag = E2M1_MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    table = np.concatenate((E4M3_VALUES, [np.nan], -E4M3_VALUES, [np.nan]))
    step = np.repeat(table[scales], 16, axis=-1)
    return mag * step * np.asarray(s, np.float64)[None, :, None, None]


def e4m3_values(cache, scale):
    """E4M3 cache bytes [NB, Hkv, 16, d] and scales [NB, Hkv] -> fp64 values."""
    table = np.concatenate((E4M3_VALUES, [np.nan], -E4M3_VALUES, [np.nan]))
    return table[np.asarray(cache, np.uint8)] * np.asarray(scale, np.float64)[:, :, None, None]


def sees(n, j, window=None, sinks=0):
    """Whether a row whose own position is n - 1 sees token j."""
    return (j < n) & (True if window is None else ((j >= n - window) | (j < sinks)))


def attend(q, keys, values, table, lens, rows, scale, window=None, sinks=0, masks=None, sizes=False):
    """Attention of packed rows.  q [total, Hq, d]; keys, values [NB, Hkv, 16, d] fp64; rows[b] new rows
    of sequence b, the last of its lens[b] tokens; masks: optional ancestor bitmasks [total] over the new
    tokens.  A row that sees nothing is zeros; blocks outside the pool are left out.  fp64 [total, Hq, d].
    With sizes=True also sum_j p_j |v_j| [total, Hq, d] and max_j sum |q k_j| scale [total, Hq, 1] over the
    tokens each row sees: what the rounding errors of an evaluation are proportional to."""
    q = to_f64(q)
    hkv, d = keys.shape[1], keys.shape[3]
    group = q.shape[1] // hkv
    out = np.zeros(q.shape)
    spread, dots = np.zeros(q.shape), np.zeros((*q.shape[:2], 1))
    first = 0
    for b, r in enumerate(rows):
        n_all = int(lens[b])
        j = np.arange(max(n_all, 0))
        block = np.asarray(table[b], np.int64)[j // BLOCK] if n_all > 0 else j
        good = (block >= 0) & (block < keys.shape[0])
        own = n_all - r + np.arange(r)
        see = sees(own[:, None] + 1, j[None, :], window, sinks)
        if masks is not None:
            new = j - (n_all - r)
            bit = (np.asarray(masks, np.int64)[first: first + r, None] >> np.clip(new, 0, 31)[None]) & 1
            see = np.where(new[None] >= 0, bit == 1, True)
        see = see & good[None]
        used = see.any(0)
        jj, blk = j[used], block[used]
        k, v = keys[blk, :, jj % BLOCK], values[blk, :, jj % BLOCK]  # [P, Hkv, d]
        x = np.einsum("rhgd,phd->rhgp", q[first: first + r].reshape(r, hkv, group, d), k) * scale
        x = np.where(see[:, used][:, None, None], x, -np.inf)
        any_seen = see.any(1)[:, None, None, None]
        top = np.where(any_seen, x.max(-1, keepdims=True, initial=-np.inf), 0)
        p = np.where(np.isneginf(x), 0, np.exp(x - top))
        # a token that a row does not see gives it nothing, whatever is stored there
        # (callers store non-finite values only where no row sees them)
        v = np.where(np.isnan(v) | np.isinf(v), 0, v) if not np.isfinite(v).all() else v
        o = np.einsum("rhgp,phd->rhgd", p, v) / np.maximum(p.sum(-1, keepdims=True), 1e-300)
        out[first: first + r] = np.where(any_seen, o, 0).reshape(r, -1, d)
        if sizes:
            a = np.einsum("rhgp,phd->rhgd", p, np.abs(v)) / np.maximum(p.sum(-1, keepdims=True), 1e-300)
            spread[first: first + r] = np.where(any_seen, a, 0).reshape(r, -1, d)
            k0 = np.where(np.isfinite(k), np.abs(k), 0)
            y = np.einsum("rhgd,phd->rhgp", np.abs(q[first: first + r]).reshape(r, hkv, group, d), k0) * abs(scale)
            y = np.where(see[:, used][:, None, None], y, 0)
            dots[first: first + r] = y.max(-1, keepdims=True, initial=0).reshape(r, -1, 1)
        first += r
    return (out, spread, dots) if sizes else out


def norm_rope(x, weight, cos_sin, positions, eps, interleaved=False):
    """x [T, heads, d] -> normed and rotated rows, fp64."""
    x, weight, cos_sin = to_f64(x), to_f64(weight), to_f64(cos_sin)
    rotary = cos_sin.shape[1]
    half = rotary // 2
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    cos, sin = cos_sin[positions][:, None, :half], cos_sin[positions][:, None, half:]
    a_at, b_at = (np.arange(0, rotary, 2), np.arange(1, rotary, 2)) if interleaved else \
        (np.arange(half), np.arange(half, rotary))
    out = y.copy()
    out[..., a_at] = y[..., a_at] * cos - y[..., b_at] * sin
    out[..., b_at] = y[..., b_at] * cos + y[..., a_at] * sin
    return out
