"""The largest batches and long contexts that the entry points admit, on values whose answer is known, and calls
from several host threads at once."""

import threading

import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def _cache(kv, blocks, d, gen):
    """A cache of one kv head with random keys and values, and its values as bf16 [blocks * 16, d]."""
    k, v = (torch.randn(blocks, 1, 16, d, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    if kv == "bf16":
        return k, v, {}, v.view(-1, d)
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([blocks * 16], dtype=torch.int32, device="cuda")
    if kv == "fp4":
        ck, cv = (torch.zeros(blocks, 1, 16, 9 * d // 16, dtype=torch.uint8, device="cuda") for _ in "kv")
        kw = {}
    else:
        ck, cv = (torch.zeros(blocks, 1, 16, d, dtype=torch.uint8, device="cuda") for _ in "kv")
        kw = {n: torch.ones(blocks, 1, device="cuda") for n in ("k_scale", "v_scale")}
    pa.append_kv(k.view(1, -1, 1, d), v.view(1, -1, 1, d), ck, cv, table, lens, **kw)
    return ck, cv, kw, pa.read_kv(ck, cv, table, lens, blocks * 16, **kw)[1].view(-1, d)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("window", [None, 1])
@pytest.mark.parametrize("form,B,r", [("decode", 65535, 1), ("verify", 65535, 2), ("prefill", 65536, 1)])
def test_the_largest_batch(form, B, r, window, kv):
    # every sequence sees one token (its first row none but for that): the answer is its value
    d, hq = 64, 2
    gen = torch.Generator(device="cuda").manual_seed(B + r)
    blocks = 4096
    k, v, kw, vf = _cache(kv, blocks, d, gen)
    table = torch.randint(0, blocks, (B, 1), generator=gen, device="cuda", dtype=torch.int32)
    lens = torch.full((B,), r, dtype=torch.int32, device="cuda")
    q = torch.randn(B, r, hq, d, generator=gen, device="cuda", dtype=torch.bfloat16)
    if window:
        kw = {**kw, "window": window}
    if form == "prefill":
        starts = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        out = pa.prefill(q[:, 0].contiguous(), k, v, table, lens, starts, d ** -0.5, max_q_len=1, **kw)[:, None]
    else:
        out = (pa.decode if form == "decode" else pa.verify)(q, k, v, table, lens, d ** -0.5, **kw)
    assert pa.check_device_errors() == pa.PA_OK
    rows = range(r) if window else [0]  # (without a window the second row sees two tokens)
    for i in rows:
        want = vf[table[:, 0].long() * 16 + i][:, None].float().expand(B, hq, d)
        got = out[:, i].float()
        # one rounding to bf16 of the kernel's and one of the value read back, 2^-8 each, and an f16 weight's, 2^-11
        assert ((got - want).abs() <= (2 * 2.0 ** -8 + 2.0 ** -11) * want.abs()).all()


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("form,r", [("decode", 1), ("verify", 5), ("verify", 16), ("prefill", 40)])
def test_a_context_of_millions(form, r, kv):
    # keys of zero weigh every token alike, and every token's value is the same: so is the answer
    d, hq, n = 64, 4, 3_000_017
    blocks = (n + 15) // 16
    kw = {}
    if kv == "bf16":
        k, v = torch.zeros(blocks, 1, 16, d, dtype=torch.bfloat16, device="cuda"), torch.full(
            (blocks, 1, 16, d), 1.5, dtype=torch.bfloat16, device="cuda")
    elif kv == "e4m3":
        k = torch.zeros(blocks, 1, 16, d, dtype=torch.uint8, device="cuda")
        v = torch.full((blocks, 1, 16, d), 0x3C, dtype=torch.uint8, device="cuda")  # 1.5
        kw = {n_: torch.ones(blocks, 1, device="cuda") for n_ in ("k_scale", "v_scale")}
    else:
        k = torch.zeros(blocks, 1, 16, 9 * d // 16, dtype=torch.uint8, device="cuda")
        v = torch.full_like(k, 0x33)  # codes of 1.5
        v.view(blocks, -1)[:, 8 * d:] = 0x38  # scales of 1
    table = torch.randperm(blocks, device="cuda").int()[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.randn(1, r, hq, d, device="cuda").bfloat16()
    if form == "prefill":
        starts = torch.tensor([0, r], dtype=torch.int32, device="cuda")
        out = pa.prefill(q[0], k, v, table, lens, starts, d ** -0.5, max_q_len=r, **kw)
    else:
        out = (pa.decode if form == "decode" else pa.verify)(q, k, v, table, lens, d ** -0.5, **kw)
    assert pa.check_device_errors() == pa.PA_OK
    # weights of 1, sums that are multiples of 0.5 below 2^23: exact in fp32 up to the division and the merge, a few
    # 2^-20; then the output's rounding
    assert ((out.float() - 1.5).abs() <= 1.5 * 2.0 ** -8).all()


def test_host_threads():
    cases = [("decode", "fp4"), ("verify", "e4m3"), ("prefill", "bf16"), ("decode", "bf16")]
    work = []
    for i, (form, kv) in enumerate(cases):
        rows = [1, 1] if form == "decode" else [5, 5]
        c = A.make(kv, [900, 70], rows, 8, 2, 128, seed=20 + i, window=300, sinks=4)
        dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
        more = {"max_q_len": 5} if form == "prefill" else {}
        work.append((form, dev, more, A.call(dev, form, **more)))
    torch.cuda.synchronize()
    wrong = []

    def run(form, dev, more, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got = A.call(dev, form, **more)
                torch.cuda.current_stream().synchronize()
                if not torch.equal(got, want):
                    wrong.append(form)

    threads = [threading.Thread(target=run, args=w) for w in work * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and pa.check_device_errors() == pa.PA_OK
