"""Plain forms of block selection, attention over any set of tokens, and eviction (numpy, fp64 or exact whole numbers).

TEST INFRASTRUCTURE ONLY, as the rest of this package.  Written from the definitions: bounds and scores in fp64 and
Python integers, selection and eviction by sorting, attention row by row over an explicit visibility array.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def code_exp(amax):
    """The smallest e with amax 2^-e <= 127, at least -126; 0 for amax 0."""
    if amax == 0:
        return 0
    e = math.frexp(amax)[1] - 7
    if math.ldexp(amax, -e) > 127:
        e += 1
    return max(e, -126)


def block_bounds(keys):
    """keys [T, d] fp64 (fp32 values) of one (block, head) -> codes [2, d] int8 and the scale 2^e."""
    e = code_exp(float(np.abs(keys).max()))
    step = math.ldexp(1.0, e)
    return np.stack((np.ceil(keys.max(0) / step), np.floor(keys.min(0) / step))).astype(np.int8), np.float32(step)


def scores(rows, codes, scale):
    """rows [R, d] fp64 (bf16 values), codes [N, 2, d] int8, scale [N] -> the blocks' scores [N], each the exact value."""
    best = np.full(len(codes), -np.inf)
    c64 = codes.astype(np.int64)
    for row in rows:
        f = code_exp(float(np.abs(row).max()))
        q = np.rint(np.ldexp(row, -f)).astype(np.int64)
        whole = np.maximum(q * c64[:, 0], q * c64[:, 1]).sum(-1)
        best = np.maximum(best, whole * math.ldexp(1.0, f))
    return best * np.asarray(scale, np.float64)


def pick(score, count, sinks, recent):
    """The columns taken of len(score) blocks, ascending."""
    n = len(score)
    s = np.array(score, np.float64)
    s[:sinks] = np.inf
    s[max(0, n - recent):] = np.inf
    return np.sort(np.argsort(-s, kind="stable")[:count])


def evict_positions(sums, keep, sinks, recent):
    """Positions that one (sequence, kv head) keeps of len(sums) tokens, ascending.  The first and the last stand above
    every sum; a NaN stands below every number."""
    n = len(sums)
    always = (np.arange(n) < sinks) | (np.arange(n) >= n - recent)
    order = sorted(range(n), key=lambda i: (not always[i], bool(np.isnan(sums[i])), -sums[i] if sums[i] == sums[i] else 0.0, i))
    return np.sort(np.array(order[:keep], np.int64))


def attend(q, keys, values, table, lens, scale, see):
    """q [B, R, Hq, d]; keys, values [NB, Hkv, 16, d] fp64; see(b) -> bool [Hkv, R, lens[b]].  Returns the outputs
    [B, R, Hq, d], what their errors are proportional to -- sum_j p_j |v_j| [B, R, Hq, d], max_j sum |q k_j| scale
    [B, R, Hq, 1] -- and each sequence's weights [Hkv, R, G, lens[b]].  A row that sees nothing is zeros."""
    B, R, Hq, d = q.shape
    hkv = keys.shape[1]
    g = Hq // hkv
    out, spread, dots, probs = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, R, Hq, 1)), []
    for b in range(B):
        n = max(int(lens[b]), 0)
        j = np.arange(n)
        block = np.asarray(table[b], np.int64)[j // BLOCK] if n else j
        good = (block >= 0) & (block < keys.shape[0])
        block = np.where(good, block, 0)
        p_all = np.zeros((hkv, R, g, n))
        vis = see(b)
        for h in range(hkv):
            s = vis[h] & good[None]
            if not s.any():
                continue
            used = s.any(0)
            k, v = keys[block[used], h, j[used] % BLOCK], values[block[used], h, j[used] % BLOCK]
            s = s[:, used]
            rows = q[b, :, h * g: (h + 1) * g]
            x = np.einsum("rgd,pd->rgp", rows, k) * scale
            x = np.where(s[:, None], x, -np.inf)
            some = s.any(1)[:, None, None]
            top = np.where(some, x.max(-1, keepdims=True), 0)
            p = np.where(np.isneginf(x), 0, np.exp(x - top))
            p = p / np.maximum(p.sum(-1, keepdims=True), 1e-300)
            at = slice(h * g, (h + 1) * g)
            out[b, :, at] = p @ v
            spread[b, :, at] = p @ np.abs(v)
            y = np.einsum("rgd,pd->rgp", np.abs(rows), np.abs(k)) * abs(scale)
            dots[b, :, at, 0] = np.where(s[:, None], y, 0).max(-1)
            p_all[h][:, :, used] = p
        probs.append(p_all)
    return out, spread, dots, probs
