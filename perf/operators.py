"""Cases of the sliding-window, 4-bit-cache and norm-and-rotation operators, with their plain forms.

``run`` makes one pass: the plain form in elementary torch operations (32-bit, rounded once at the
end), or, where ``own`` is true, the calls that a serving program makes of the package.  ``exact``
gives the same outputs from the definitions in 64 bits, written apart from the plain form.

Definitions.
  Window attention.  A row whose own position is n - 1 sees token j when j < n and (j >= n - window
  or j < sinks).  Query heads share K/V heads in contiguous groups; out = softmax(scale q.k) v.
  Blocks of the table that no row sees are never read and hold -1 here, as in a program that has
  given them back to its pool.
  4-bit cache.  Each 16 consecutive dims of one token's head row are 16 E2M1 codes (two a byte, the
  lower dim in the low nibble) and one E4M3 scale; the value is code * scale * s with one fp32 s for
  each kv head.  A (block, head) page of uint8 holds the codes of its 16 tokens, then their scales.
  Storing x: scale = e4m3(min(amax|x| / (6 s), 448)), code = e2m1(x / (scale * s)), both to nearest
  even in fp32 arithmetic; a zero scale stores zeros.
  Norm and rotation.  Each head row of q and k: y = x / sqrt(mean(x^2) + eps) * weight, then the first
  `rotary` dims are rotated in pairs (i, i + rotary / 2) by the row of the position's cosines and
  sines.
"""

import math

import torch

own = False

BLOCK = 16
EPS = 1e-6
MAX_POSITION = 32768
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ------------------------------------------------------------------------------------

def _attn(name, kv, batch, rows, ctx_min, ctx_max, hq, hkv, d, window=0, sinks=0, packed=False):
    c = {"op": "attention", "kv": kv, "batch": batch, "rows": rows, "ctx_min": ctx_min, "ctx_max": ctx_max,
         "hq": hq, "hkv": hkv, "d": d, "window": window, "sinks": sinks, "packed": packed}
    return {"name": name, **c} if name else c


def _append(name, batch, rows, ctx_min, ctx_max, hkv, d):
    c = {"op": "append", "kv": "fp4", "batch": batch, "rows": rows, "ctx_min": ctx_min, "ctx_max": ctx_max,
         "hkv": hkv, "d": d}
    return {"name": name, **c} if name else c


def _rope(name, tokens, hq, hkv, d, rotary):
    c = {"op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rotary": rotary}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a handful of chats, one token each: latency counts
        _attn("window_decode_chat", "bf16", 8, 1, 37, 8192, 32, 8, 128, 1024, 4),
        # a full continuous batch of long conversations that keep only a window and the first tokens
        _attn("window_decode_batch", "bf16", 256, 1, 100, 32768, 64, 8, 128, 4096, 4),
        # four drafts and the bonus row verified against an 8-bit windowed cache
        _attn("window_verify_e4m3", "e4m3", 32, 5, 41, 16001, 32, 8, 128, 2048, 16),
        # chunked prefill of several prompts in one call, ragged, most of the context out of the window
        _attn("window_prefill", "bf16", 4, 2048, 2100, 12011, 32, 8, 128, 4096, 4, True),
        # one decode step of a batch stored in the 4-bit cache and read back
        _append("fp4_append_step", 64, 1, 1, 8192, 8, 128),
        # prompt chunks stored in the 4-bit cache
        _append("fp4_append_chunk", 4, 2048, 2048, 8200, 8, 128),
        # one user, one token, a context that ends inside a block
        _attn("fp4_decode_single", "fp4", 1, 1, 8193, 8193, 32, 8, 128),
        # the case the 4-bit cache is for: many long contexts at once
        _attn("fp4_decode_batch", "fp4", 64, 1, 1000, 32768, 32, 8, 128),
        # four drafts and the bonus row against 4-bit contexts
        _attn("fp4_verify", "fp4", 32, 5, 100, 8192, 32, 8, 128),
        # prompt chunks behind long 4-bit contexts
        _attn("fp4_prefill", "fp4", 2, 1024, 9001, 16384, 32, 8, 128, 0, 0, True),
        # the queries and keys of one decode step
        _rope("qk_norm_rope_step", 8, 32, 8, 128, 128),
        # the queries and keys of a long packed prompt
        _rope("qk_norm_rope_chunk", 16384, 32, 8, 128, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 8), (8, 8), (8, 1), (28, 4), (40, 8)])
    d = rng.choice([64, 128])
    kind = rng.choice(["decode", "decode", "verify", "prefill", "append", "rope"])
    if kind == "rope":
        return _rope(None, _log(rng, 1, 16384), hq, hkv, d, rng.choice([d, d, d // 2]))
    if kind == "append":
        rows = rng.choice([1, 1, _log(rng, 2, 2048)])
        batch = _log(rng, 1, max(1, min(128, 8192 // rows)))
        hi = rows + _log(rng, 1, 8192)
        return _append(None, batch, rows, rng.randint(rows, hi), hi, hkv, d)
    kv = rng.choice(["fp4", "fp4", "bf16", "e4m3"])
    window = _log(rng, 1, 8192) if kv != "fp4" or rng.random() < 0.3 else 0
    sinks = rng.choice([0, 1, 4, 16, 100]) if window else 0
    if kind == "prefill":
        if hq // hkv not in (1, 2, 4, 8):
            hq, hkv = 32, 8
        rows = _log(rng, 2, 2048)
        batch = _log(rng, 1, max(1, min(16, 4096 // rows)))
        hi = rows + _log(rng, 1, 12000)
        return _attn(None, kv, batch, rows, rng.randint(rows, hi), hi, hq, hkv, d, window, sinks, True)
    rows = 1 if kind == "decode" else rng.randint(2, 9)
    hi = rows + _log(rng, 1, 32768)
    seen = min(hi, window + sinks + rows) if window else hi
    batch = _log(rng, 1, max(1, min(256, 500000 // seen)))
    return _attn(None, kv, batch, rows, rng.randint(rows, hi), hi, hq, hkv, d, window, sinks)


def _lens(case):
    """The batch's context lengths: ctx_max first, the others spread over the range."""
    lo, hi = case["ctx_min"], case["ctx_max"]
    return [hi] + [lo + int((hi - lo) * ((b * 0.6180339887) % 1.0)) for b in range(1, case["batch"])]


def _rows(case):
    """New rows of each sequence: the same for a decode or verify step, ragged for packed chunks."""
    r = case["rows"]
    if not case.get("packed"):
        return [r] * case["batch"]
    return [r] + [1 + int((r - 1) * ((b * 0.7548776662) % 1.0)) for b in range(1, case["batch"])]


def _seen(case):
    """For each sequence the first window position that any row sees (0: the whole context)."""
    if case["op"] != "attention" or not case["window"]:
        return [0] * case["batch"]
    return [max(0, n - r + 1 - case["window"]) for n, r in zip(_lens(case), _rows(case))]


def work(case):
    """Bytes: queries, outputs and every visible cache row once; flops: two products per visible pair."""
    if case["op"] == "rope":
        t, h, d = case["tokens"], case["hq"] + case["hkv"], case["d"]
        return {"bytes": t * h * d * 4 + t * (case["rotary"] + 1) * 4, "flops": t * h * d * 8}
    hkv, d = case["hkv"], case["d"]
    row = {"bf16": 2 * d, "e4m3": d, "fp4": d * 9 // 16}[case["kv"]]
    if case["op"] == "append":
        t = case["batch"] * case["rows"] * hkv * 2
        return {"bytes": t * (2 * d + 2 * row + 2 * d), "flops": t * d * 4}
    w, s = case["window"], case["sinks"]
    total_bytes = flops = 0
    for n, r, lo in zip(_lens(case), _rows(case), _seen(case)):
        total_bytes += (n - lo + min(s, lo)) * hkv * row * 2 + r * case["hq"] * d * 4
        for i in range(r):
            end = n - r + i + 1
            first = max(0, end - w) if w else 0
            flops += 4 * d * case["hq"] * (end - first + min(s, first))
    return {"bytes": total_bytes, "flops": flops}


# ---- inputs -----------------------------------------------------------------------------------

def _codes_of(a):
    """E2M1 magnitude codes of a >= 0, to nearest, ties to the even code, saturating at 6."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _encode(x, s):
    """x [..., Hkv, d] bf16 and s [Hkv] fp32 -> E2M1 bytes [..., Hkv, d / 2], E4M3 scale bytes [..., Hkv, d / 16]."""
    xb = x.float().unflatten(-1, (-1, 16))
    s = s[:, None]
    amax = xb.abs().amax(-1)
    scale = torch.minimum(amax / (6.0 * s), torch.full_like(amax, 448.0)).to(torch.float8_e4m3fn)
    step = (scale.float() * s).unsqueeze(-1)
    y = torch.where(step > 0, xb / step, torch.zeros_like(xb))
    code = (_codes_of(y.abs()) + 8 * (torch.signbit(xb) & (step > 0)).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(codes, scales, s):
    """E2M1 bytes [..., Hkv, d / 2], E4M3 scale bytes [..., Hkv, d / 16] and s [Hkv] -> fp32 [..., Hkv, d]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = lut[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    step = scales.view(torch.float8_e4m3fn).float() * s[:, None]
    return (v.unflatten(-1, (-1, 16)) * step.unsqueeze(-1)).flatten(-2)


def _page_views(cache, d):
    """Code bytes [NB, Hkv, 16, d / 2] and scale bytes [NB, Hkv, 16, d / 16] of a 4-bit cache."""
    pages = cache.view(cache.shape[0], cache.shape[1], -1)
    codes, scales = pages[:, :, : BLOCK * d // 2], pages[:, :, BLOCK * d // 2:]
    return codes.unflatten(-1, (BLOCK, d // 2)), scales.unflatten(-1, (BLOCK, d // 16))


def _fp4_cache(x, s):
    """A 4-bit cache [NB, Hkv, 16, 9 d / 16] holding x [NB, Hkv, 16, d]."""
    nb, hkv, _, d = x.shape
    codes, scales = _encode(x.transpose(1, 2), s)
    codes, scales = codes.transpose(1, 2).reshape(nb, hkv, -1), scales.transpose(1, 2).reshape(nb, hkv, -1)
    return torch.cat((codes, scales), -1).view(nb, hkv, BLOCK, d * 9 // 16)


def _table(case, rng, dev):
    """A block table with random physical blocks for the blocks in use, and the pool's size."""
    lens, seen = _lens(case), _seen(case)
    width = max(-(-n // BLOCK) for n in lens)
    rows = torch.arange(width, device=dev)[None]
    n = torch.tensor([-(-x // BLOCK) for x in lens], device=dev)[:, None]
    lo = torch.tensor([x // BLOCK for x in seen], device=dev)[:, None]
    sink_blocks = -(-case.get("sinks", 0) // BLOCK)
    used = (rows < n) & ((rows >= lo) | (rows < sink_blocks))
    order = used.flatten().cumsum(0).view_as(used) - 1
    count = int(used.sum())
    pool = count + max(1, count // 8)
    perm = torch.randperm(pool, generator=rng, device=dev)
    table = torch.where(used, perm[order.clamp(min=0)], -torch.ones_like(order)).int()
    return table.contiguous(), pool


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=rng, device=dev, dtype=torch.bfloat16)

    d, hkv = case["d"], case["hkv"]
    if case["op"] == "rope":
        t, hq = case["tokens"], case["hq"]
        qkv = randn(t, (hq + 2 * hkv) * d) * 3  # the packed projection of one layer
        pos = torch.randint(0, MAX_POSITION, (t,), generator=rng, device=dev, dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, case["rotary"], 2, device=dev, dtype=torch.float64) / case["rotary"])
        angle = torch.arange(MAX_POSITION, device=dev, dtype=torch.float64)[:, None] * freq
        weights = [1 + 0.2 * randn(d) for _ in range(2)]
        return {"case": case, "q": qkv[:, : hq * d].unflatten(-1, (hq, d)),
                "k": qkv[:, hq * d: (hq + hkv) * d].unflatten(-1, (hkv, d)), "pos": pos, "qw": weights[0], "kw": weights[1],
                "cos_sin": torch.cat((angle.cos(), angle.sin()), -1).float().contiguous()}
    lens, rows = _lens(case), _rows(case)
    table, pool = _table(case, rng, dev)
    st = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "max_len": max(lens),
          "k_scale": None, "v_scale": None}
    gains = torch.exp(0.5 * randn(hkv, 1, d))  # some channels of the keys are larger than others
    if case["kv"] == "fp4":  # one scale for each head, a power of two near amax / (6 * 448)
        st["k_scale"] = torch.exp2(torch.randint(-8, -5, (hkv,), generator=rng, device=dev).float())
        st["v_scale"] = torch.exp2(torch.randint(-8, -5, (hkv,), generator=rng, device=dev).float())
    if case["op"] == "append":
        st["k_new"] = randn(case["batch"], case["rows"], hkv, d) * gains.view(hkv, d)
        st["v_new"] = randn(case["batch"], case["rows"], hkv, d)
        shape = (pool, hkv, BLOCK, d * 9 // 16)
        st["k"], st["v"] = (torch.zeros(shape, dtype=torch.uint8, device=dev) for _ in range(2))
        return st
    k, v = randn(pool, hkv, BLOCK, d) * gains, randn(pool, hkv, BLOCK, d)
    if case["kv"] == "bf16":
        st["k"], st["v"] = k, v
    elif case["kv"] == "fp4":
        st["k"], st["v"] = _fp4_cache(k, st["k_scale"]), _fp4_cache(v, st["v_scale"])
    else:
        for n, x in (("k", k.float()), ("v", v.float())):
            st[n + "_scale"] = (x.abs().amax((2, 3)) / 448).clamp(min=1e-12)
            st[n] = (x / st[n + "_scale"][:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if case["packed"]:
        st["q"] = randn(sum(rows), case["hq"], d)
        st["starts"] = torch.tensor([0] + rows, device=dev).cumsum(0).int()
        st["row_seq"] = torch.repeat_interleave(torch.arange(len(rows), device=dev), torch.tensor(rows, device=dev))
        st["row_at"] = torch.arange(sum(rows), device=dev) - st["starts"][st["row_seq"]]
        st["max_rows"] = max(rows)
    else:
        st["q"] = randn(case["batch"], case["rows"], case["hq"], d)
    return st


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"attention": _plain_attention, "append": _plain_append, "rope": _plain_rope}[state["case"]["op"]](state)


def _run_own(st):
    import paged_kv_gqa_attn_gb300 as pa

    c = st["case"]
    if c["op"] == "rope":
        return pa.qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["cos_sin"], st["pos"], eps=EPS)
    scales = {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if c["op"] == "append":
        pa.append_kv(st["k_new"], st["v_new"], st["k"], st["v"], st["table"], st["lens"], **scales)
        return pa.read_kv(st["k"], st["v"], st["table"], st["lens"], c["rows"], **scales)
    scale = 1 / math.sqrt(c["d"])
    more = {"max_context_len": st["max_len"], **scales}
    if c["window"]:
        more |= {"window": c["window"], "sinks": c["sinks"]}
    lead = (st["q"], st["k"], st["v"], st["table"], st["lens"])
    if c["packed"]:
        return pa.prefill(*lead, st["starts"], scale, max_q_len=st["max_rows"], **more)
    return (pa.decode if c["rows"] == 1 else pa.verify)(*lead, scale, **more)


def _gather(st, cache, scale, pos):
    """Cache rows [B, P, Hkv, d] in fp32 of the positions pos [B, P]."""
    c = st["case"]
    block = st["table"].long().gather(1, pos // BLOCK).clamp(min=0)
    at = pos % BLOCK
    if c["kv"] == "fp4":
        codes, scales = _page_views(cache, c["d"])
        return _values(codes[block, :, at], scales[block, :, at], scale)
    if c["kv"] == "e4m3":
        return cache.view(torch.float8_e4m3fn)[block, :, at].float() * scale[block][..., None]
    return cache[block, :, at].float()


def _plain_attention(st):
    c = st["case"]
    dev, w, s = st["q"].device, c["window"], c["sinks"]
    n = st["lens"].long()
    if c["packed"]:  # rows padded to [B, R]
        r = st["starts"].long().diff()
        pad = c["rows"]
        q = st["q"][(st["starts"][:-1, None] + torch.arange(pad, device=dev)).clamp(max=st["q"].shape[0] - 1)]
    else:
        r = torch.full_like(n, c["rows"])
        pad = c["rows"]
        q = st["q"]
    ends = (n - r)[:, None] + torch.arange(pad, device=dev) + 1  # [B, R]: tokens that each row sees without a window
    if w and s + w + pad - 1 < st["max_len"]:
        low = (n - r + 1 - w).clamp(min=s)  # the first tokens, then the window of the first row to the last token
        tail = low[:, None] + torch.arange(w + pad - 1, device=dev)
        pos = torch.cat((torch.arange(s, device=dev).expand(len(n), s), tail), 1)
    else:
        pos = torch.arange(st["max_len"], device=dev).expand(len(n), -1)
    seen = (pos[:, None] < ends[..., None])
    if w:
        seen = seen & ((pos[:, None] >= ends[..., None] - w) | (pos[:, None] < s))
    pos = torch.minimum(pos, n[:, None] - 1)
    k = _gather(st, st["k"], st["k_scale"], pos)
    v = _gather(st, st["v"], st["v_scale"], pos)
    qf = q.float().unflatten(2, (c["hkv"], -1))  # [B, R, Hkv, G, d]
    x = torch.einsum("brhgd,bphd->bhgrp", qf, k) * (1 / math.sqrt(c["d"]))
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.einsum("bhgrp,bphd->brhgd", p / p.sum(-1, keepdim=True), v).flatten(2, 3).to(torch.bfloat16)
    return o[st["row_seq"], st["row_at"]] if c["packed"] else o


def _plain_append(st):
    c = st["case"]
    pos = (st["lens"].long() - c["rows"])[:, None] + torch.arange(c["rows"], device=st["lens"].device)
    block, at = st["table"].long().gather(1, pos // BLOCK), pos % BLOCK
    out = []
    for new, cache, scale in ((st["k_new"], st["k"], st["k_scale"]), (st["v_new"], st["v"], st["v_scale"])):
        codes, scales = _page_views(cache, c["d"])
        codes[block, :, at], scales[block, :, at] = _encode(new, scale)
        out.append(_values(codes[block, :, at], scales[block, :, at], scale).to(torch.bfloat16))
    return tuple(out)


def _plain_rope(st):
    half = st["case"]["rotary"] // 2
    cs = st["cos_sin"][st["pos"].long()][:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    out = []
    for x, weight in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        y = x.float()
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
        a, b, rest = y[..., :half], y[..., half: 2 * half], y[..., 2 * half:]
        out.append(torch.cat((a * cos - b * sin, b * cos + a * sin, rest), -1).to(torch.bfloat16))
    return tuple(out)


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "rope": _exact_rope}[case["op"]](case, st)


def _exact_rows(case, st, name, b, idx):
    """Values [P, Hkv, d] in fp64 of the positions idx of sequence b."""
    pages, scale, d = st[name], st[name + "_scale"], case["d"]
    block, at = st["table"][b].long()[idx // BLOCK], idx % BLOCK
    if case["kv"] == "bf16":
        return pages[block, :, at].double()
    if case["kv"] == "e4m3":
        return pages[block, :, at].view(torch.float8_e4m3fn).double() * scale[block].double()[:, :, None]
    flat = pages.view(pages.shape[0], pages.shape[1], -1)
    dims = torch.arange(d, device=flat.device)
    byte = flat[block[:, None], :, (at[:, None] * (d // 2) + dims // 2)].transpose(1, 2).int()  # [P, Hkv, d]
    code = torch.where(dims % 2 == 0, byte & 15, byte >> 4)
    e, m = (code >> 1) & 3, code & 1
    mag = torch.where(e == 0, m * 0.5, torch.ldexp(1 + m.double() * 0.5, e - 1))
    sc = flat[block[:, None], :, (BLOCK * d // 2 + at[:, None] * (d // 16) + dims // 16)].transpose(1, 2).contiguous()
    return torch.where(code >= 8, -mag, mag) * sc.view(torch.float8_e4m3fn).double() * scale.double()[:, None]


def _exact_attention(case, st):
    dev, hkv, g, d = st["q"].device, case["hkv"], case["hq"] // case["hkv"], case["d"]
    lens, rows, outs, first = _lens(case), _rows(case), [], 0
    for b, (n, r) in enumerate(zip(lens, rows)):
        q = (st["q"][first: first + r] if case["packed"] else st["q"][b]).double()
        first += r
        own_pos = torch.arange(n - r, n, device=dev)[:, None]
        j = torch.arange(n, device=dev)
        see = j <= own_pos
        if case["window"]:
            see &= (own_pos - j < case["window"]) | (j < case["sinks"])
        idx = see.any(0).nonzero().flatten()
        see = see[:, idx].repeat_interleave(g, 0)
        k, v = _exact_rows(case, st, "k", b, idx), _exact_rows(case, st, "v", b, idx)
        out = torch.empty(r, hkv, g, d, dtype=torch.float64, device=dev)
        for h in range(hkv):
            qh = q[:, h * g: (h + 1) * g].reshape(r * g, d)
            x = qh @ k[:, h].T / d ** 0.5
            x[~see] = -math.inf
            out[:, h] = (torch.softmax(x, -1) @ v[:, h]).view(r, g, d)
        outs.append(out.flatten(1, 2))
    return torch.cat(outs) if case["packed"] else torch.stack(outs)


def _exact_append(case, st):
    grid = torch.tensor(E2M1, dtype=torch.float64, device=st["k"].device)
    # every E4M3 value that a scale can take
    e4m3 = torch.arange(127, dtype=torch.uint8, device=grid.device).view(torch.float8_e4m3fn).double()

    def nearest(x, table):
        hi = torch.searchsorted(table, x.contiguous()).clamp(1, len(table) - 1)
        lo = hi - 1
        up, down = table[hi] - x, x - table[lo]
        return table[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)]

    out = []
    for new, s in ((st["k_new"], st["k_scale"]), (st["v_new"], st["v_scale"])):
        x = new.double().unflatten(-1, (-1, 16))
        s = s.double()[:, None]
        step = (nearest((x.abs().amax(-1) / 6 / s).clamp(max=448), e4m3) * s)[..., None]
        y = nearest((x.abs() / step.clamp(min=1e-300)).clamp(max=6), grid)
        out.append((torch.sign(x) * y * step).flatten(-2))
    return tuple(out)


def _exact_rope(case, st):
    half = case["rotary"] // 2
    turn = st["cos_sin"].double()[st["pos"].long()]
    turn = torch.complex(turn[:, :half], turn[:, half:])[:, None]
    out = []
    for x, weight in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        y = x.double()
        y = y * (y.square().mean(-1, keepdim=True) + EPS).rsqrt() * weight.double()
        z = torch.complex(y[..., :half].contiguous(), y[..., half: 2 * half].contiguous()) * turn
        y[..., :half], y[..., half: 2 * half] = z.real, z.imag
        out.append(y)
    return tuple(out)
