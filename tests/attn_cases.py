"""Cases of the window and 4-bit attention tests: random paged caches of every type with their fp64
values, junk wherever no row looks, and the error bound that a result is held to."""

import numpy as np
import torch

from oracle import plain
import paged_kv_gqa_attn_gb300 as pa

BAD_ID = 1 << 30  # a block id that a lookup would flag


def make(kv, lens, rows, hq, hkv, d, seed, window=None, sinks=0, junk=True, k_mag=1.0, head_scales=True):
    """One batch: rows[b] new rows of sequence b, packed.  Blocks that no row sees have BAD_ID in the
    table, and tokens that no row sees (in visible blocks and in blocks nobody owns) hold NaN."""
    g = torch.Generator().manual_seed(seed)
    width = max(max((n + 15) // 16 for n in lens), 1)
    seen_token = np.zeros((len(lens), width * 16), bool)
    for b, (n, r) in enumerate(zip(lens, rows)):
        for i in range(r):
            if n - r + i + 1 > 0:
                seen_token[b, :n] |= plain.sees(n - r + i + 1, np.arange(n), window, sinks)
    used = seen_token.reshape(len(lens), width, 16).any(-1)
    nb = int(used.sum()) + 3
    perm = torch.randperm(nb, generator=g).numpy()
    table = np.full((len(lens), width), BAD_ID, np.int32)
    table[used] = perm[: int(used.sum())]
    k = (torch.randn(nb, hkv, 16, d, generator=g) * k_mag).to(torch.bfloat16)
    v = torch.randn(nb, hkv, 16, d, generator=g).to(torch.bfloat16)
    dead = np.ones((nb, 16), bool)
    for b in range(len(lens)):
        for j in np.nonzero(seen_token[b])[0]:
            dead[table[b, j // 16], j % 16] = False
    dead = torch.from_numpy(dead)[:, None, :, None].expand(nb, hkv, 16, d)
    c = {"kv": kv, "d": d, "lens": lens, "rows": rows, "window": window, "sinks": sinks,
         "q": torch.randn(sum(rows), hq, d, generator=g).to(torch.bfloat16), "table": torch.from_numpy(table),
         "scale": 1 / d ** 0.5, "k_scale": None, "v_scale": None}
    if kv == "bf16":
        if junk:
            k, v = k.masked_fill(dead, float("nan")), v.masked_fill(dead, float("nan"))
        c["k"], c["v"], c["kf"], c["vf"] = k, v, plain.to_f64(k), plain.to_f64(v)
    elif kv == "e4m3":
        for n, x in (("k", k.float()), ("v", v.float())):
            s = (x.abs().amax((2, 3)) / 448).contiguous()
            code = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            c[n] = code.masked_fill(dead, 0x7F) if junk else code
            c[n + "_scale"] = s
            c[n + "f"] = plain.e4m3_values(c[n].numpy(), s.numpy())
    else:
        for n, x in (("k", k), ("v", v)):
            s = 0.001 + 0.01 * torch.rand(hkv, generator=g) if head_scales else None
            sf = np.ones(hkv, np.float32) if s is None else s.numpy()
            codes, scales = plain.fp4_unpack(plain.fp4_pages(x.float().numpy(), sf), d)
            if junk:
                codes = np.where(dead.numpy(), 15, codes).astype(np.uint8)
                scales = np.where(dead.numpy()[..., :: 16], 0x7F, scales).astype(np.uint8)
            c[n] = torch.from_numpy(plain.fp4_pack(codes, scales))
            c[n + "_scale"] = s
            c[n + "f"] = plain.fp4_values(c[n].numpy(), d, sf)
    return c


def call(c, form, device="cuda", **more):
    """Run the case through decode, verify or prefill; packed rows [total, Hq, d]."""
    dev = {n: (t.to(device) if torch.is_tensor(t) else t) for n, t in c.items()}
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=device)
    kw = {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"], **more}
    if c["window"] is not None:
        kw |= {"window": c["window"], "sinks": c["sinks"]}
    if form == "prefill":
        starts = torch.tensor(np.concatenate(([0], np.cumsum(c["rows"]))), dtype=torch.int32, device=device)
        return pa.prefill(dev["q"], dev["k"], dev["v"], dev["table"], lens, starts, c["scale"], **kw)
    q = dev["q"].view(len(c["lens"]), c["rows"][0], *dev["q"].shape[1:])
    fn = pa.decode if form == "decode" else pa.verify
    return fn(q, dev["k"], dev["v"], dev["table"], lens, c["scale"], **kw).flatten(0, 1)


def check(c, form, got):
    """Hold a result to the plain form.  The bound, element by element:
      2^-8 |out|                 the output's rounding to bf16;
      w sum p |v|                the weights' rounding w: bf16 weights 2^-8 (and the sum that divides
                                 them takes the rounded ones: once more), f16 weights 2^-11, and twice the
                                 error of a score: fp32 sums of d products, d 2^-24 sum |q k|, a factor
                                 of 2 for the exponent's own rounding; E4M3 keys at d = 128 in the tile
                                 kernels take q as two E4M3 terms, off by 2^-8 of |q|;
      n 2^-25 max |v|            f16 weights below 2^-14 lose absolute 2^-25, n of them."""
    ref, spread, dots = plain.attend(c["q"], c["kf"], c["vf"], c["table"].numpy(), c["lens"], c["rows"], c["scale"],
                                     c["window"], c["sinks"], masks=c.get("masks"), sizes=True)
    group = c["q"].shape[1] // c["kf"].shape[1]
    tiles = form != "decode" or group not in (1, 2, 4, 8)
    d = c["d"]
    w = {"bf16": 2.0 ** -7 if tiles else 2.0 ** -14, "e4m3": 2.0 ** -11, "fp4": 2.0 ** -11}[c["kv"]]
    score = 2 * d * 2.0 ** -24 + (2.0 ** -8 if c["kv"] == "e4m3" and d == 128 and tiles else 0)
    vf = c["vf"][np.isfinite(c["vf"])]
    floor = 0 if c["kv"] == "bf16" else max(c["lens"]) * 2.0 ** -25 * np.abs(vf).max()
    bound = 2.0 ** -8 * np.abs(ref) + (w + 2 * score * dots) * spread + floor + 1e-30
    got = plain.to_f64(got)
    assert np.isfinite(got).all(), np.argwhere(~np.isfinite(got))[:4].tolist()
    over = np.abs(got - ref) - bound
    assert (over <= 0).all(), (form, over.max(), np.argwhere(over > 0)[:4].tolist(), int((over > 0).sum()))
    return ref
