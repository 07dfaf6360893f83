"""Cases of the tests of listed blocks, shared prefixes and kept weights: the caches of attn_cases, and the bounds that
results are held to."""

import numpy as np
import torch

import attn_cases as A
from oracle import forms, plain

BAD_ID = A.BAD_ID


def causal(lens, r):
    """see(b) of ordinary decode and verify."""
    def see(b, hkv):
        n = lens[b]
        own = n - r + np.arange(r)
        return np.broadcast_to(np.arange(n)[None] <= own[:, None], (hkv, r, n))
    return see


def reference(c, see):
    """oracle.forms.attend of an attn_cases case whose sequences have the same rows."""
    r, hkv = c["rows"][0], c["kf"].shape[1]
    q = plain.to_f64(c["q"]).reshape(len(c["lens"]), r, *c["q"].shape[1:])
    return forms.attend(q, c["kf"], c["vf"], c["table"].numpy(), c["lens"], c["scale"], lambda b: see(b, hkv))


def check(c, got, see, tiles):
    """Hold [B, R, Hq, d] outputs to the definition; the bound is that of attn_cases.check: the output's rounding to
    bf16, the weights' rounding (tiles: bf16 weights 2^-8, twice; else a bf16 pair, 2^-14; f16 weights 2^-11), twice the
    error of a score, and f16 weights below 2^-14."""
    ref, spread, dots, probs = reference(c, see)
    d = c["d"]
    w = {"bf16": 2.0 ** -7 if tiles else 2.0 ** -14, "e4m3": 2.0 ** -11, "fp4": 2.0 ** -11}[c["kv"]]
    score = 2 * d * 2.0 ** -24 + (2.0 ** -8 if c["kv"] == "e4m3" and d == 128 and tiles else 0)
    floor = 0 if c["kv"] == "bf16" else max(c["lens"]) * 2.0 ** -25 * np.abs(c["vf"][np.isfinite(c["vf"])]).max()
    bound = 2.0 ** -8 * np.abs(ref) + (w + 2 * score * dots) * spread + floor + 1e-30
    got = plain.to_f64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:4].tolist()
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), (over.max(), np.argwhere(over > 0)[:4].tolist(), int((over > 0).sum()))
    return ref, dots, probs


def on_gpu(c):
    """(q [B, R, Hq, d], k, v, table, lens) on the GPU, and the scales."""
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    q = dev["q"].view(len(c["lens"]), c["rows"][0], *dev["q"].shape[1:])
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    return (q, dev["k"], dev["v"], dev["table"], lens), {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"]}
