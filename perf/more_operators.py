"""Cases of block-sparse attention, shared-prefix attention and eviction by attention weight, with their plain forms.

``run`` makes one pass: the plain form in elementary torch operations (32-bit, rounded once at the end), or, where
``own`` is true, the calls that a serving program makes of the package.  ``exact`` gives the same outputs from the
definitions in 64 bits, written apart from the plain form.

Definitions (blocks of 16 tokens, caches and tables as in ordinary paged attention).
  Block bounds.  For each (block, kv head): the largest and the smallest of every dim over the block's stored tokens, as
  int8 codes times one power of two 2^e, rounded away from the keys (ceil and floor); e is the smallest integer with
  max|k| 2^-e <= 127 (at least -126; 0 for keys of zero).  A key of an E4M3 or 4-bit cache is its fp32 value.
  Selection.  Each query row is rounded to int8 codes times a power of two by the same rule; a block's score for it is the
  sum over dims of max(q hi, q lo), an upper bound of q.k, and its score for a kv head the largest over that head's rows.
  The first sink_blocks and last recent_blocks blocks are always taken, then the highest scores, ties to the lowest block;
  `count` blocks in ascending order, -1 where there are fewer.  Every sum is a whole number below 2^22 times a power of two.
  Sparse attention.  softmax(scale q.k) v over the tokens of the selected blocks that the row sees.
  Shared prefix.  The sequences of a group have their first prefix tokens in the same blocks; the outputs are those of
  ordinary attention over the whole context.
  Weighted decode.  Ordinary decode that also folds the step's softmax weights, summed over the query heads of a kv head,
  into fp32 sums kept for every cached token: sum = decay * sum + weight; the new token's sum starts with its weight.
  Eviction.  Each kv head keeps of its n tokens the first `sinks`, the last `recent` and, up to `keep` in all, those of
  the largest sums (ties to the earliest); they move in order, with their sums, to the blocks of another table.
"""

import math

import torch

own = False

BLOCK = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases ------------------------------------------------------------------------------------

def _case(name, **c):
    return {"name": name, **c} if name else c


def _bounds(name, kv, batch, rows, ctx_min, ctx_max, hkv, d):
    return _case(name, op="bounds", kv=kv, batch=batch, rows=rows, ctx_min=ctx_min, ctx_max=ctx_max, hkv=hkv, d=d)


def _sparse(name, kv, batch, rows, ctx_min, ctx_max, hq, hkv, d, count, sinks=1, recent=2):
    return _case(name, op="sparse", kv=kv, batch=batch, rows=rows, ctx_min=ctx_min, ctx_max=ctx_max, hq=hq, hkv=hkv, d=d,
                 count=count, sinks=sinks, recent=recent)


def _prefix(name, kv, groups, batch, rows, prefix_min, prefix_max, own_min, own_max, hq, hkv, d):
    return _case(name, op="prefix", kv=kv, groups=groups, batch=batch, rows=rows, prefix_min=prefix_min,
                 prefix_max=prefix_max, own_min=own_min, own_max=own_max, hq=hq, hkv=hkv, d=d)


def _weighted(name, kv, batch, ctx_min, ctx_max, hq, hkv, d, decay):
    return _case(name, op="weighted", kv=kv, batch=batch, rows=1, ctx_min=ctx_min, ctx_max=ctx_max, hq=hq, hkv=hkv, d=d,
                 decay=decay)


def _evict(name, kv, batch, ctx_min, ctx_max, hkv, d, keep, sinks, recent):
    return _case(name, op="evict", kv=kv, batch=batch, rows=1, ctx_min=ctx_min, ctx_max=ctx_max, hkv=hkv, d=d, keep=keep,
                 sinks=sinks, recent=recent)


def listed():
    return [
        # the bounds of one decode step's blocks
        _bounds("bounds_step", "bf16", 64, 1, 100, 32768, 8, 128),
        # the bounds of several long prompts, made once after their prefill
        _bounds("bounds_prompts", "e4m3", 8, 32768, 9001, 32768, 8, 128),
        # a few chats over long documents: bounds of the new token, selection, attention; latency counts
        _sparse("sparse_step_chat", "bf16", 4, 1, 1000, 16384, 32, 8, 128, 64),
        # a full batch of long contexts, a sixteenth of the longest read
        _sparse("sparse_step_batch", "bf16", 64, 1, 8000, 32768, 32, 8, 128, 128),
        # four drafts and the bonus row verified over the selected blocks of 8-bit caches
        _sparse("sparse_verify_e4m3", "e4m3", 16, 5, 3000, 16384, 32, 8, 128, 96),
        # a batch behind one long system prompt
        _prefix("prefix_decode_batch", "bf16", 1, 64, 1, 8192, 8192, 17, 1000, 32, 8, 128),
        # several prompts shared by groups of different sizes, 8-bit caches
        _prefix("prefix_decode_groups", "e4m3", 5, 128, 1, 2000, 16384, 5, 2048, 32, 8, 128),
        # drafts verified for a small group behind a short shared prompt, 4-bit caches: latency counts
        _prefix("prefix_verify_fp4", "fp4", 1, 8, 5, 2048, 2048, 100, 700, 32, 8, 128),
        # a handful of chats whose sums are kept; latency counts
        _weighted("weighted_decode_chat", "bf16", 8, 37, 4096, 32, 8, 128, 1.0),
        # a batch of long contexts whose sums fade
        _weighted("weighted_decode_batch", "bf16", 64, 1000, 16384, 32, 8, 128, 0.98),
        # a few chats halved
        _evict("evict_chat", "bf16", 4, 2100, 4096, 8, 128, 2048, 4, 256),
        # long contexts brought down to a budget
        _evict("evict_batch", "bf16", 16, 9000, 32768, 8, 128, 4096, 16, 1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 8), (8, 8), (8, 1), (28, 4), (40, 8)])
    d = rng.choice([64, 128])
    kv = rng.choice(["bf16", "bf16", "e4m3", "fp4"])
    kind = rng.choice(["bounds", "sparse", "sparse", "prefix", "prefix", "weighted", "evict"])
    if kind == "bounds":
        hi = _log(rng, 1, 32768)
        rows = rng.choice([1, 1, _log(rng, 2, 2048), hi])
        batch = _log(rng, 1, max(1, min(256, 250000 // hi)))
        return _bounds(None, kv, batch, min(rows, hi), rng.randint(1, hi), hi, hkv, d)
    if kind == "sparse":
        rows = rng.choice([1, 1, rng.randint(2, max(2, min(9, 32 * hkv // hq)))])
        hi = rows + _log(rng, 1, 32768)
        sinks, recent = rng.choice([(0, 1), (1, 2), (1, 4), (4, 8)])
        count = _log(rng, max(1, sinks + recent), 256)
        batch = _log(rng, 1, max(1, min(128, 1000000 // hi, 8192 // count)))
        return _sparse(None, kv, batch, rows, rng.randint(rows, hi), hi, hq, hkv, d, count, sinks, recent)
    if kind == "prefix":
        rows = rng.choice([1, 1, rng.randint(2, 9)])
        prefix = BLOCK * _log(rng, 1, 1024)
        own_max = rows + _log(rng, 1, 2048)
        batch = _log(rng, 1, max(1, min(128, 130000 // own_max)))
        groups = _log(rng, 1, min(batch, max(1, 40000 // prefix)))
        lo = BLOCK * rng.randint(0, prefix // BLOCK)
        return _prefix(None, kv, groups, batch, rows, lo, prefix, rng.randint(rows, own_max), own_max, hq, hkv, d)
    hi = _log(rng, 1, 32768)
    batch = _log(rng, 1, max(1, min(128, 500000 // hi)))
    lo = rng.randint(1, hi)
    if kind == "weighted":
        return _weighted(None, kv, batch, lo, hi, hq, hkv, d, rng.choice([0.0, 0.9, 1.0]))
    batch = min(batch, max(1, 300000 // hi))
    keep = _log(rng, 1, min(8192, 2 * hi))
    sinks = rng.choice([0, min(4, keep - 1)])
    return _evict(None, kv, batch, lo, hi, hkv, d, keep, sinks, rng.randint(0, keep - sinks))


def _spread(n, lo, hi, step=0.6180339887):
    """n whole numbers: hi first, the others over [lo, hi]."""
    return [hi] + [lo + int((hi - lo) * ((b * step) % 1.0)) for b in range(1, n)]


def _starts(case):
    """First sequence of each group of a prefix case, and the batch's size at the end."""
    g, b = case["groups"], case["batch"]
    shares = [1.0 + 2.0 * ((i * 0.7548776662) % 1.0) for i in range(g)]
    edges = [0]
    for i in range(g):
        left = b - edges[-1] - (g - 1 - i)
        edges.append(edges[-1] + (left if i == g - 1 else max(1, min(left, round(b * shares[i] / sum(shares))))))
    return edges


def _prefixes(case):
    """Shared tokens of each group (whole blocks) and of each sequence."""
    each = [p // BLOCK * BLOCK for p in _spread(case["groups"], case["prefix_min"], case["prefix_max"])]
    starts = _starts(case)
    return each, [each[i] for i in range(case["groups"]) for _ in range(starts[i + 1] - starts[i])]


def _lens(case):
    if case["op"] == "prefix":
        return [p + n for p, n in zip(_prefixes(case)[1], _spread(case["batch"], case["own_min"], case["own_max"]))]
    return _spread(case["batch"], case["ctx_min"], case["ctx_max"])


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    """Bytes: every input that counts read once, every output written once; flops: two products per visible pair."""
    hkv, d, lens, rows = case["hkv"], case["d"], _lens(case), case["rows"]
    row = {"bf16": 2 * d, "e4m3": d, "fp4": d * 9 // 16}[case["kv"]]
    bound = 2 * d + 4
    if case["op"] == "bounds":
        tokens = sum(n - max(0, n - rows) // BLOCK * BLOCK for n in lens)
        blocks = sum(_blocks(n) - max(0, n - rows) // BLOCK for n in lens)
        return {"bytes": hkv * (tokens * row + blocks * bound), "flops": tokens * hkv * d * 2}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": hkv * (sum(lens) * 4 + kept * (4 * row + 4)), "flops": sum(lens) * hkv}
    hq = case["hq"]
    io = case["batch"] * rows * hq * d * 4
    if case["op"] == "sparse":
        read = [min(n, case["count"] * BLOCK) for n in lens]
        scored = sum(_blocks(n) for n in lens)
        return {"bytes": io + hkv * (scored * bound + sum(read) * 2 * row) + case["batch"] * hkv * case["count"] * 8,
                "flops": 4 * d * hq * rows * sum(read) + scored * hq * rows * 4 * d}
    if case["op"] == "prefix":
        each, of = _prefixes(case)
        tokens = sum(each) + sum(n - p for n, p in zip(lens, of))
        return {"bytes": io + hkv * tokens * 2 * row, "flops": 4 * d * hq * rows * sum(lens)}
    return {"bytes": io + hkv * sum(lens) * (2 * row + 8), "flops": 4 * d * hq * sum(lens)}


# ---- inputs -----------------------------------------------------------------------------------

def _codes_of(a):
    """E2M1 magnitude codes of a >= 0, to nearest, ties to the even code, saturating at 6."""
    return ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))


def _fp4_cache(x, s):
    """A 4-bit cache [NB, Hkv, 16, 9 d / 16] holding x [NB, Hkv, 16, d]: codes, then E4M3 scales, for each (block, head)."""
    nb, hkv, _, d = x.shape
    cache = torch.empty(nb, hkv, BLOCK * d * 9 // 16, dtype=torch.uint8, device=x.device)
    for i in range(0, nb, 4096):  # (a slice of the pool at a time: the temporaries are many)
        xb = x[i: i + 4096].float().unflatten(-1, (-1, 16))
        amax = xb.abs().amax(-1)
        scale = torch.minimum(amax / (6.0 * s[:, None, None]), torch.full_like(amax, 448.0)).to(torch.float8_e4m3fn)
        step = (scale.float() * s[:, None, None]).unsqueeze(-1)
        y = torch.where(step > 0, xb / step, torch.zeros_like(xb))
        code = (_codes_of(y.abs()) + 8 * (torch.signbit(xb) & (step > 0)).to(torch.uint8)).flatten(-2)
        codes = code[..., 0::2] | (code[..., 1::2] << 4)
        cache[i: i + 4096] = torch.cat((codes.flatten(2), scale.view(torch.uint8).flatten(2)), -1)
    return cache.view(nb, hkv, BLOCK, d * 9 // 16)


def _page_values(case, pages, scale, ids):
    """Keys or values [*ids.shape, Hkv, 16, d] in fp32 of the blocks ids."""
    d, hkv = case["d"], case["hkv"]
    x = pages[ids]
    if case["kv"] == "bf16":
        return x.float()
    if case["kv"] == "e4m3":
        return x.view(torch.float8_e4m3fn).float() * scale[ids][..., None, None]
    x = x.reshape(*ids.shape, hkv, -1)
    codes, scales = x[..., : BLOCK * d // 2].contiguous(), x[..., BLOCK * d // 2:].contiguous()
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=x.device)
    v = lut[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()].unflatten(-1, (BLOCK, d // 16, 16))
    step = scales.view(torch.float8_e4m3fn).float().unflatten(-1, (BLOCK, d // 16)).unsqueeze(-1)
    return (v * step).flatten(-2) * scale[:, None, None]


def _exponents(amax):
    """The smallest e with amax 2^-e <= 127, at least -126; 0 for amax 0."""
    m, e = torch.frexp(amax)
    e = e - 7 + (m * 128 > 127).to(e.dtype)
    return torch.where(amax > 0, e.clamp(min=-126), torch.zeros_like(e))


def _exp2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _bound_codes(k, seen):
    """Keys k [..., Hkv, 16, d] fp32 with the tokens seen [..., 16] -> int8 codes [..., Hkv, 2, d], scales [..., Hkv]."""
    none = ~seen[..., None, :, None]
    hi = k.masked_fill(none, -math.inf).amax(-2)
    lo = k.masked_fill(none, math.inf).amin(-2)
    e = _exponents(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    down = _exp2(-e)[..., None]
    return torch.stack((torch.ceil(hi * down), torch.floor(lo * down)), -2).to(torch.int8), _exp2(e)


def _all_bounds(case, st):
    """Bounds of every block in use."""
    shape = (st["k"].shape[0], case["hkv"])
    codes = torch.zeros(*shape, 2, case["d"], dtype=torch.int8, device=st["k"].device)
    scale = torch.ones(shape, device=codes.device)
    at = torch.arange(BLOCK, device=codes.device)
    for b, n in enumerate(_lens(case)):
        nb = _blocks(n)
        ids = st["table"][b, :nb].long()
        seen = torch.arange(nb, device=codes.device)[:, None] * BLOCK + at < n
        codes[ids], scale[ids] = _bound_codes(_page_values(case, st["k"], st["k_scale"], ids), seen)
    return codes, scale


def _table(case, rng, dev):
    """A block table with random physical blocks (a group's shared ones once), and the pool's size."""
    lens = _lens(case)
    width = max(_blocks(n) for n in lens)
    column = torch.arange(width, device=dev)[None]
    used = column < torch.tensor([_blocks(n) for n in lens], device=dev)[:, None]
    first = torch.arange(len(lens), device=dev)[:, None].expand(-1, width)
    if case["op"] == "prefix":  # the row that holds each entry first
        starts, (each, of) = _starts(case), _prefixes(case)
        lead = torch.tensor([starts[i] for i in range(len(each)) for _ in range(starts[i + 1] - starts[i])], device=dev)
        shared = column < torch.tensor([p // BLOCK for p in of], device=dev)[:, None]
        first = torch.where(shared, lead[:, None], first)
    owns = used & (first == torch.arange(len(lens), device=dev)[:, None])
    order = owns.flatten().cumsum(0).view_as(owns) - 1
    order = order.gather(0, first)
    count = int(owns.sum())
    extra = case["batch"] * _blocks(case["keep"]) if case["op"] == "evict" else 0
    pool = count + extra + max(1, count // 8)
    perm = torch.randperm(pool, generator=rng, device=dev)
    table = torch.where(used, perm[order.clamp(min=0)], -torch.ones_like(order)).int().contiguous()
    fresh = perm[count: count + extra].view(case["batch"], -1).int().contiguous() if extra else None
    return table, pool, fresh


def prepare(case, seed):
    dev = torch.device("cuda")
    rng = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=rng, device=dev, dtype=torch.bfloat16)

    d, hkv = case["d"], case["hkv"]
    table, pool, fresh = _table(case, rng, dev)
    lens = _lens(case)
    st = {"case": case, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "max_len": max(lens),
          "k_scale": None, "v_scale": None}
    # some channels of the keys are larger than others, and what a block is about moves its keys together
    k = randn(pool, hkv, BLOCK, d).add_(randn(pool, hkv, 1, d), alpha=0.7).mul_(torch.exp(0.5 * randn(hkv, 1, d)))
    v = randn(pool, hkv, BLOCK, d)
    if case["kv"] == "bf16":
        st["k"], st["v"] = k, v
    elif case["kv"] == "fp4":  # one scale for each head, a power of two near amax / (6 * 448)
        for n, x in (("k", k), ("v", v)):
            st[n + "_scale"] = torch.exp2(torch.randint(-8, -5, (hkv,), generator=rng, device=dev).float())
            st[n] = _fp4_cache(x, st[n + "_scale"])
    else:
        for n, x in (("k", k), ("v", v)):
            scale = (x.abs().amax((2, 3)).float() / 448).clamp(min=1e-12)
            st[n + "_scale"] = scale
            st[n] = (x.float() / scale[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    del k, v
    if "hq" in case:
        st["q"] = randn(case["batch"], case["rows"], case["hq"], d)
    if case["op"] in ("bounds", "sparse"):
        st["bounds"], st["bound_scale"] = _all_bounds(case, st)
        if case["op"] == "bounds":  # not made yet
            st["bounds"].zero_()
            st["bound_scale"].fill_(1.0)
    elif case["op"] == "prefix":
        st["starts"] = torch.tensor(_starts(case), dtype=torch.int32, device=dev)
        st["prefix_lens"] = torch.tensor(_prefixes(case)[0], dtype=torch.int32, device=dev)
        st["max_prefix"], st["max_own"] = max(_prefixes(case)[0]), case["own_max"]
    else:  # sums of a few hundred steps: a few tokens have most of the weight
        st["weights"] = torch.exp(2.0 * torch.randn(pool, hkv, BLOCK, generator=rng, device=dev))
        if case["op"] == "evict":
            st["fresh"] = fresh
    return st


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"bounds": _plain_bounds, "sparse": _plain_sparse, "prefix": _plain_prefix, "weighted": _plain_weighted,
            "evict": _plain_evict}[state["case"]["op"]](state)


def _sums(st):
    """The sums that a weighted pass updates: a copy where it reads them, so that a pass can be made again."""
    return st["weights"] if st["case"]["decay"] == 0 else st["weights"].clone()


def _run_own(st):
    import paged_kv_gqa_attn_gb300 as pa

    c = st["case"]
    scales = {"k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if c["op"] in ("bounds", "sparse"):
        pa.block_bounds(st["k"], st["table"], st["lens"], c["rows"], st["bounds"], st["bound_scale"], k_scale=st["k_scale"])
        if c["op"] == "bounds":
            return st["bounds"], st["bound_scale"]
    if c["op"] == "evict":
        lens = pa.evict(st["k"], st["v"], st["weights"], st["table"], st["lens"], st["fresh"], c["keep"], sinks=c["sinks"],
                        recent=c["recent"], max_context_len=st["max_len"], **scales)
        if c["kv"] == "bf16":
            return lens, st["weights"], st["k"], st["v"]
        count = min(c["keep"], *_lens(c))  # the tokens that every sequence has, read back from its end
        return lens, st["weights"], *pa.read_kv(st["k"], st["v"], st["fresh"], lens, count, head_dim=c["d"], **scales)
    scale = 1 / math.sqrt(c["d"])
    more = {"max_context_len": st["max_len"], **scales}
    out = ()
    if c["op"] == "sparse":
        blocks = pa.select_blocks(st["q"], st["bounds"], st["bound_scale"], st["table"], st["lens"], c["count"],
                                  sink_blocks=c["sinks"], recent_blocks=c["recent"], max_context_len=st["max_len"])
        more["blocks"] = blocks
        out = (blocks,)
    elif c["op"] == "prefix":
        more |= {"group_starts": st["starts"], "prefix_lens": st["prefix_lens"], "max_prefix_len": st["max_prefix"],
                 "max_own_len": st["max_own"]}
    else:
        more |= {"weights": _sums(st), "decay": c["decay"]}
        out = (more["weights"],)
    fn = pa.decode if c["rows"] == 1 else pa.verify
    return (fn(st["q"], st["k"], st["v"], st["table"], st["lens"], scale, **more), *out)


def _plain_bounds(st):
    c = st["case"]
    n = st["lens"].long()
    first = (n - c["rows"]).clamp(min=0) // BLOCK
    most = int(_blocks(c["rows"])) + 1
    blocks = first[:, None] + torch.arange(min(most, st["table"].shape[1]), device=n.device)
    ok = blocks * BLOCK < n[:, None]
    ids = st["table"].long().gather(1, blocks.clamp(max=st["table"].shape[1] - 1))[ok]
    at = blocks[ok][:, None] * BLOCK + torch.arange(BLOCK, device=n.device)
    seen = at < n[:, None].expand_as(blocks)[ok][:, None]
    st["bounds"][ids], st["bound_scale"][ids] = _bound_codes(_page_values(c, st["k"], st["k_scale"], ids), seen)
    return st["bounds"], st["bound_scale"]


def _plain_select(st):
    c = st["case"]
    n = st["lens"].long()
    nb = -(-n // BLOCK)
    q = st["q"].float().unflatten(2, (c["hkv"], -1))  # [B, R, Hkv, G, d]
    f = _exponents(q.abs().amax(-1))
    code = torch.round(q * _exp2(-f)[..., None])
    ids = st["table"].long().clamp(min=0)
    bounds = st["bounds"][ids].float()  # [B, N, Hkv, 2, d]
    s = torch.einsum("brhgd,bnhd->brhgn", code.clamp(min=0), bounds[:, :, :, 0])
    s += torch.einsum("brhgd,bnhd->brhgn", code.clamp(max=0), bounds[:, :, :, 1])
    s = (s * _exp2(f)[..., None]).amax((1, 3)) * st["bound_scale"][ids].transpose(1, 2)  # [B, Hkv, N]
    j = torch.arange(ids.shape[1], device=ids.device)
    forced = (j < c["sinks"]) | (j >= nb[:, None] - c["recent"])
    s = s.masked_fill(forced[:, None], math.inf).masked_fill((j >= nb[:, None])[:, None], -math.inf)
    best = torch.sort(s, dim=-1, descending=True, stable=True).indices[..., : c["count"]]
    best = best.masked_fill(best >= nb[:, None, None], ids.shape[1]).sort(-1).values
    best = best.masked_fill(best == ids.shape[1], -1).int()
    return torch.nn.functional.pad(best, (0, c["count"] - best.shape[-1]), value=-1)


def _plain_sparse(st):
    c = st["case"]
    _plain_bounds(st)
    blocks = _plain_select(st)
    n, dev = st["lens"].long(), st["q"].device
    b, h = torch.arange(c["batch"], device=dev)[:, None, None], torch.arange(c["hkv"], device=dev)[None, :, None]
    ids = st["table"].long()[b, blocks.long().clamp(min=0)].clamp(min=0)  # [B, Hkv, K]

    def tokens(name):
        """[B, Hkv, K * 16, d] of the selected blocks, a sequence at a time."""
        scale = st[name + "_scale"]
        out = []
        for i in range(c["batch"]):
            x = st[name][ids[i], h[0]]  # [Hkv, K, 16, bytes or dims] of each head's own blocks
            if c["kv"] == "e4m3":
                x = x.view(torch.float8_e4m3fn).float() * scale[ids[i], h[0]][..., None, None]
            elif c["kv"] == "fp4":
                x = x.reshape(*x.shape[:2], -1)
                lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=dev)
                codes, steps = x[..., : BLOCK * c["d"] // 2], x[..., BLOCK * c["d"] // 2:].contiguous()
                x = lut[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()].unflatten(-1, (BLOCK, -1, 16))
                x = x * steps.view(torch.float8_e4m3fn).float().unflatten(-1, (BLOCK, -1)).unsqueeze(-1)
                x = x.flatten(-2) * scale[:, None, None, None]
            out.append(x.float().flatten(1, 2))
        return torch.stack(out)

    pos = (blocks.long()[..., None] * BLOCK + torch.arange(BLOCK, device=dev)).flatten(2)  # [B, Hkv, K * 16]
    ends = (n - c["rows"])[:, None] + torch.arange(c["rows"], device=dev) + 1
    seen = (pos[:, :, None] >= 0) & (pos[:, :, None] < ends[:, None, :, None])  # [B, Hkv, R, P]
    q = st["q"].float().unflatten(2, (c["hkv"], -1))
    x = torch.einsum("brhgd,bhpd->bhgrp", q, tokens("k")) * (1 / math.sqrt(c["d"]))
    x = x.masked_fill(~seen[:, :, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    o = torch.einsum("bhgrp,bhpd->brhgd", p / p.sum(-1, keepdim=True), tokens("v"))
    return o.flatten(2, 3).to(torch.bfloat16), blocks


def _rows_of(st, name, seqs, columns):
    """Cache rows [S, C * 16, Hkv, d] in fp32 of the table columns [S, C] of the sequences seqs [S]."""
    ids = st["table"].long()[seqs[:, None], columns].clamp(min=0)
    x = _page_values(st["case"], st[name], st[name + "_scale"], ids)  # [S, C, Hkv, 16, d]
    return x.transpose(2, 3).flatten(1, 2)


def _plain_prefix(st):
    """Each group's shared tokens against all of its rows at once, beside every sequence's own."""
    c, dev = st["case"], st["q"].device
    edges, each = _starts(c), _prefixes(c)[0]
    n = st["lens"].long()
    q = st["q"].float().unflatten(2, (c["hkv"], -1)) * (1 / math.sqrt(c["d"]))
    out = []
    for i, p in enumerate(each):
        seqs = torch.arange(edges[i], edges[i + 1], device=dev)
        own_blocks = _blocks(c["own_max"])
        cols = (p // BLOCK + torch.arange(own_blocks, device=dev)).expand(len(seqs), -1)
        pos = (cols[..., None] * BLOCK + torch.arange(BLOCK, device=dev)).flatten(1)
        ends = (n[seqs] - c["rows"])[:, None] + torch.arange(c["rows"], device=dev) + 1
        hidden = pos[:, None] >= ends[..., None]  # [S, R, P]
        cols = cols.clamp(max=st["table"].shape[1] - 1)
        qg = q[seqs]
        x = torch.einsum("srhgd,sphd->shgrp", qg, _rows_of(st, "k", seqs, cols)).masked_fill(hidden[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        if p:
            shared = torch.arange(p // BLOCK, device=dev)[None]
            y = torch.einsum("srhgd,phd->shgrp", qg, _rows_of(st, "k", seqs[:1], shared)[0])
            top = torch.maximum(top, y.amax(-1, keepdim=True))
            y = torch.exp(y - top)
        x = torch.exp(x - top)
        total = x.sum(-1, keepdim=True)
        o = torch.einsum("shgrp,sphd->shgrd", x, _rows_of(st, "v", seqs, cols))
        if p:
            total = total + y.sum(-1, keepdim=True)
            o = o + torch.einsum("shgrp,phd->shgrd", y, _rows_of(st, "v", seqs[:1], shared)[0])
        out.append((o / total).permute(0, 3, 1, 2, 4).flatten(2, 3))
    return (torch.cat(out).to(torch.bfloat16),)


def _plain_weighted(st):
    c, dev = st["case"], st["q"].device
    n = st["lens"].long()
    sums = _sums(st)
    seqs = torch.arange(c["batch"], device=dev)
    cols = torch.arange(st["table"].shape[1], device=dev).expand(c["batch"], -1)
    pos = torch.arange(cols.shape[1] * BLOCK, device=dev)
    seen = pos < n[:, None]
    q = st["q"][:, 0].float().unflatten(1, (c["hkv"], -1))
    x = torch.einsum("bhgd,bphd->bhgp", q, _rows_of(st, "k", seqs, cols)) * (1 / math.sqrt(c["d"]))
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = torch.einsum("bhgp,bphd->bhgd", p, _rows_of(st, "v", seqs, cols)).flatten(1, 2)[:, None].to(torch.bfloat16)
    step = p.sum(2)  # [B, Hkv, P]
    b, j = seen.nonzero(as_tuple=True)
    ids, at = st["table"].long()[b, j // BLOCK], j % BLOCK
    old = sums[ids, :, at] * c["decay"] if c["decay"] else torch.zeros_like(sums[ids, :, at])
    old = torch.where((j == n[b] - 1)[:, None], torch.zeros_like(old), old)
    sums[ids, :, at] = old + step[b, :, j]
    return o, sums


def _plain_evict(st):
    c, dev = st["case"], st["k"].device
    n, keep = st["lens"].long(), c["keep"]
    width = st["table"].shape[1] * BLOCK
    ids = st["table"].long().clamp(min=0)
    w = st["weights"][ids].permute(0, 2, 1, 3).flatten(2)  # [B, Hkv, P]
    pos = torch.arange(width, device=dev)
    end = n[:, None, None]
    w = w.masked_fill((pos < c["sinks"]) | (pos >= end - c["recent"]), math.inf).masked_fill(pos >= end, -math.inf)
    kept = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    kept = torch.where(kept < end, kept, width).sort(-1).values  # [B, Hkv, keep], in order
    lens = torch.minimum(n, torch.full_like(n, keep))
    b, h, i = (kept < width).nonzero(as_tuple=True)
    src = kept[b, h, i]
    from_block, from_at = ids[b, src // BLOCK], src % BLOCK
    to_block, to_at = st["fresh"].long()[b, i // BLOCK], i % BLOCK
    st["weights"][to_block, h, to_at] = st["weights"][from_block, h, from_at]
    if c["kv"] == "bf16":
        for name in ("k", "v"):
            st[name][to_block, h, to_at] = st[name][from_block, h, from_at]
        return lens.int(), st["weights"], st["k"], st["v"]
    tail = []
    count = min(keep, *_lens(c))
    at = (lens - count)[:, None] + torch.arange(count, device=dev)
    for name in ("k", "v"):
        scale = st[name + "_scale"]
        blocks = _blocks(keep)
        x = torch.zeros(c["batch"], c["hkv"], blocks * BLOCK, c["d"], device=dev)
        if c["kv"] == "e4m3":
            rows = st[name].view(torch.float8_e4m3fn)[from_block, h, from_at].float() * scale[from_block, h][:, None]
            x[b, h, i] = rows
            x = x.unflatten(2, (blocks, BLOCK))
            amax = x.abs().amax((3, 4))
            new = torch.where(amax > 0, amax / 448, torch.ones_like(amax))[..., None, None]
            codes = (x / new).clamp(-448, 448).to(torch.float8_e4m3fn)
            used = torch.arange(blocks, device=dev) < (-(-lens // BLOCK))[:, None]
            bb, jj = used.nonzero(as_tuple=True)
            st[name][st["fresh"].long()[bb, jj]] = codes.view(torch.uint8)[bb, :, jj]
            scale[st["fresh"].long()[bb, jj]] = new[bb, :, jj, 0, 0]
            x = (codes.float() * new).flatten(2, 3)
        else:
            flat = st[name].view(st[name].shape[0], c["hkv"], -1)
            half, sc = c["d"] // 2, c["d"] // 16
            for size, base in ((half, 0), (sc, BLOCK * half)):
                k = torch.arange(size, device=dev)
                flat[to_block[:, None], h[:, None], base + to_at[:, None] * size + k] = \
                    flat[from_block[:, None], h[:, None], base + from_at[:, None] * size + k]
            x = _page_values(c, st[name], scale, st["fresh"].long()).transpose(1, 2).flatten(2, 3)
        at_ = at[:, None, :, None].expand(-1, c["hkv"], -1, c["d"])
        tail.append(x.gather(2, at_).transpose(1, 2).to(torch.bfloat16))
    return lens.int(), st["weights"], *tail


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "bounds":
        return _exact_bounds(case, st)
    if case["op"] == "evict":
        return _exact_evict(case, st)
    if case["op"] == "sparse":
        _exact_bounds(case, st)
        blocks = _exact_select(case, st)
        return _exact_attention(case, st, blocks)[0], blocks
    out, step = _exact_attention(case, st, None)
    if case["op"] == "prefix":
        return (out,)
    sums = st["weights"].double()
    for b, n in enumerate(_lens(case)):
        j = torch.arange(n, device=sums.device)
        ids = st["table"][b].long()[j // BLOCK]
        old = sums[ids, :, j % BLOCK] * case["decay"]
        old[n - 1] = 0
        sums[ids, :, j % BLOCK] = old + step[b].T
    return out, sums


def _exact_tokens(case, st, name, b, idx):
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


def _exact_step(amax):
    """2^e of the int8 codes of numbers up to amax, in 64 bits."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 127))
    e = torch.where(amax * torch.exp2(-e) > 127, e + 1, e)
    e = torch.where(amax * torch.exp2(1 - e) <= 127, e - 1, e)
    return torch.where(amax > 0, torch.exp2(e.clamp(min=-126)), torch.ones_like(amax))


def _exact_bounds(case, st):
    for b, n in enumerate(_lens(case)):
        first = max(0, n - case["rows"]) // BLOCK * BLOCK
        k = _exact_tokens(case, st, "k", b, torch.arange(first, n, device=st["k"].device))
        k = k.float().double()  # (a key of a scaled cache is an fp32 number)
        size = _blocks(n - first)
        pad = k[-1:].expand(size * BLOCK - len(k), -1, -1)  # the last token again: no bound moves
        k = torch.cat((k, pad)).unflatten(0, (size, BLOCK))
        ids = st["table"][b].long()[first // BLOCK: first // BLOCK + size]
        step = _exact_step(k.abs().amax((1, 3)))
        hi, lo = k.amax(1) / step[..., None], k.amin(1) / step[..., None]
        st["bounds"][ids] = torch.stack((hi.ceil(), lo.floor()), 2).to(torch.int8)
        st["bound_scale"][ids] = step.float()
    return st["bounds"], st["bound_scale"]


def _exact_select(case, st):
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    out = torch.full((case["batch"], hkv, case["count"]), -1, dtype=torch.int32, device=st["q"].device)
    q = st["q"].double()
    step = _exact_step(q.abs().amax(-1, keepdim=True))
    q = torch.round(q / step) * step
    for b, n in enumerate(_lens(case)):
        nb = _blocks(n)
        ids = st["table"][b, :nb].long()
        ends = st["bounds"][ids].double() * st["bound_scale"][ids].double()[..., None, None]  # [N, Hkv, 2, d]
        for h in range(hkv):
            rows = q[b, :, h * g: (h + 1) * g].reshape(-1, case["d"])
            s = torch.stack([torch.maximum(r * ends[:, h, 0], r * ends[:, h, 1]).sum(-1) for r in rows]).amax(0)
            s[: case["sinks"]] = math.inf
            s[max(0, nb - case["recent"]):] = math.inf
            top = torch.sort(-s, stable=True).indices[: case["count"]].sort().values
            out[b, h, : len(top)] = top.int()
    return out


def _exact_attention(case, st, blocks):
    """Outputs [B, R, Hq, d] in fp64, and each sequence's weights summed over the rows and heads of a kv head."""
    dev, hkv, g, d, r = st["q"].device, case["hkv"], case["hq"] // case["hkv"], case["d"], case["rows"]
    out = torch.zeros(case["batch"], r, hkv, g, d, dtype=torch.float64, device=dev)
    sums = []
    for b, n in enumerate(_lens(case)):
        q = st["q"][b].double().unflatten(1, (hkv, g)) / d ** 0.5
        every = torch.arange(n, device=dev)
        own_at = torch.arange(n - r, n, device=dev)
        k, v = _exact_tokens(case, st, "k", b, every), _exact_tokens(case, st, "v", b, every)
        total = torch.zeros(hkv, n, dtype=torch.float64, device=dev)
        for h in range(hkv):
            see = every <= own_at[:, None]
            if blocks is not None:
                see = see & torch.isin(every // BLOCK, blocks[b, h])
            x = (q[:, h] @ k[:, h].T).masked_fill(~see[:, None], -math.inf)
            p = torch.softmax(x, -1)
            out[b, :, h] = p @ v[:, h]
            total[h] = p.sum((0, 1))
        sums.append(total)
    return out.flatten(2, 3), sums


def _exact_evict(case, st):
    lens = _lens(case)
    keep, dev = case["keep"], st["k"].device
    kept_lens = [min(n, keep) for n in lens]
    sums = st["weights"].double()
    moved = {"k": st["k"], "v": st["v"]}
    if case["kv"] == "bf16":
        moved = {name: x.double() for name, x in moved.items()}
    tail = {"k": [], "v": []}
    count = min(kept_lens)
    for b, n in enumerate(lens):
        ids = st["table"][b].long()
        every = torch.arange(n, device=dev)
        w = sums[ids[every // BLOCK], :, every % BLOCK]  # [n, Hkv]
        left = max(0, min(n, keep) - min(n, case["sinks"]) - case["recent"])
        mid = torch.arange(min(n, case["sinks"]), max(min(n, case["sinks"]), n - case["recent"]), device=dev)
        choice = torch.zeros(n, case["hkv"], dtype=torch.bool, device=dev)
        choice[: case["sinks"]] = True
        choice[max(0, n - case["recent"]):] = True
        for h in range(case["hkv"]):
            choice[mid[torch.sort(-w[mid, h], stable=True).indices[:left]], h] = True
        if n <= keep:
            choice[:] = True
        rows = {name: _exact_tokens(case, st, name, b, every) for name in ("k", "v")}
        got = {name: torch.empty(kept_lens[b], case["hkv"], case["d"], dtype=torch.float64, device=dev) for name in rows}
        for h in range(case["hkv"]):
            src = choice[:, h].nonzero().flatten()
            to = torch.arange(len(src), device=dev)
            block, at = st["fresh"][b].long()[to // BLOCK], to % BLOCK
            sums[block, h, at] = w[src, h]
            for name in rows:
                got[name][:, h] = rows[name][src, h]
                if case["kv"] == "bf16":
                    moved[name][block, h, at] = rows[name][src, h]
        for name, x in got.items():
            if case["kv"] == "e4m3":  # each new block has a scale of its own
                for j in range(0, len(x), BLOCK):
                    y = x[j: j + BLOCK]
                    amax = y.abs().amax((0, 2), keepdim=True)
                    s = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
                    x[j: j + BLOCK] = (y / s).float().to(torch.float8_e4m3fn).double() * s
            tail[name].append(x[len(x) - count:])
    out = torch.tensor(kept_lens, dtype=torch.int32, device=dev)
    if case["kv"] == "bf16":
        return out, sums, moved["k"], moved["v"]
    return out, sums, torch.stack(tail["k"]), torch.stack(tail["v"])
