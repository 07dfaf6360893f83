"""The forms over listed blocks, shared prefixes and kept weights, selection and eviction: captured and replayed, on
other streams than the current one, from several host threads, and with outputs repeated bit for bit."""

import threading

import numpy as np
import pytest
import torch

import attn_cases as A
from form_cases import on_gpu
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


class Step:
    """One of each call, over buffers of its own."""

    def __init__(self, kv, seed, lens=(300, 40, 700, 129), hq=8, hkv=2, d=128):
        c = A.make(kv, list(lens), [1] * len(lens), hq, hkv, d, seed=seed, junk=False)
        (self.q, self.k, self.v, self.table, self.n), self.s = on_gpu(c)
        self.shared = self.table.clone()
        self.shared[1:, :2] = self.shared[0, :2]  # a shared prefix of 32 tokens (the sums' call shares no blocks)
        self.scale = c["scale"]
        B, nb = len(lens), len(self.k)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.codes = torch.zeros(nb, hkv, 2, d, dtype=torch.int8, device="cuda")
        self.bscale = torch.ones(nb, hkv, device="cuda")
        self.w = torch.zeros(nb, hkv, 16, device="cuda")
        self.starts, self.pre = torch.tensor([0, B], **i32), torch.tensor([32], **i32)
        self.blocks = torch.empty(B, hkv, 6, **i32)
        self.outs = [torch.empty_like(self.q) for _ in range(3)]
        self.new_lens = torch.empty(B, **i32)
        # the evicted tokens' new blocks: the pool grown at its end
        m = 3
        for name in ("k", "v"):
            x = getattr(self, name)
            setattr(self, name, torch.cat((x, torch.zeros(B * m, *x.shape[1:], dtype=x.dtype, device="cuda"))))
        if kv == "e4m3":
            self.s = {n: torch.cat((t, torch.zeros(B * m, hkv, device="cuda"))) for n, t in self.s.items()}
        self.codes = torch.zeros(nb + B * m, hkv, 2, d, dtype=torch.int8, device="cuda")
        self.bscale = torch.ones(nb + B * m, hkv, device="cuda")
        self.w = torch.zeros(nb + B * m, hkv, 16, device="cuda")
        self.fresh = (nb + torch.arange(B * m, **i32)).view(B, m).contiguous()
        self.d = d
        torch.cuda.synchronize()

    def run(self, stream=None):
        kw = {"stream": stream}
        pa.block_bounds(self.k, self.table, self.n, 10000, self.codes, self.bscale, k_scale=self.s["k_scale"], **kw)
        pa.select_blocks(self.q, self.codes, self.bscale, self.table, self.n, 6, out=self.blocks, **kw)
        a = (self.q, self.k, self.v, self.table, self.n, self.scale)
        pa.decode(*a, blocks=self.blocks, out=self.outs[0], **self.s, **kw)
        pa.decode(*a[:3], self.shared, *a[4:], group_starts=self.starts, prefix_lens=self.pre, max_prefix_len=32, out=self.outs[1], **self.s, **kw)
        pa.decode(*a, weights=self.w, decay=0.0, out=self.outs[2], **self.s, **kw)
        pa.evict(self.k, self.v, self.w, self.table, self.n, self.fresh, 40, sinks=2, recent=5, head_dim=self.d,
                 new_lens=self.new_lens, **self.s, **kw)

    def results(self):
        return [t.clone() for t in (self.codes, self.bscale, self.blocks, *self.outs, self.w, self.new_lens, self.k, self.v)]

    def scramble(self):
        for t in (self.blocks, self.new_lens, *self.outs):
            t.zero_()
        self.codes.zero_()
        self.bscale.fill_(1.0)  # (blocks that nobody owns keep it)
        self.k[self.fresh.flatten().long()] = 0
        self.v[self.fresh.flatten().long()] = 0


def _bits(t):
    return t.view({2: torch.int16, 4: torch.int32}.get(t.element_size(), t.dtype)) if t.is_floating_point() else t


def _same(a, b):
    return all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
def test_captured_and_replayed(kv):
    st, other = Step(kv, 1), Step(kv, 2)
    st.run()
    torch.cuda.synchronize()
    want = st.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    for _ in range(3):
        st.scramble()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(st.results(), want)
    # new inputs in the captured buffers
    other.run()
    torch.cuda.synchronize()
    want = other.results()
    if other.table.shape == st.table.shape and other.k.shape == st.k.shape:
        for name in ("q", "k", "v", "table", "shared", "n", "w"):
            getattr(st, name).copy_(getattr(other, name))
        for n, t in st.s.items():
            if t is not None:
                t.copy_(other.s[n])
        st.scramble()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(st.results(), want)
    assert pa.check_device_errors() == pa.PA_OK


def test_two_graphs_at_once():
    # scratch belongs to each captured call: replays that overlap do not meet
    steps = [Step("bf16", 3), Step("bf16", 4)]
    graphs, wants = [], []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        wants.append(st.results())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            st.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for st in steps:
            st.scramble()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(_same(st.results(), w) for st, w in zip(steps, wants))


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "fp4"])
def test_on_a_stream_of_its_own_and_bit_for_bit(kv):
    st = Step(kv, 5)
    st.run()
    torch.cuda.synchronize()
    want = st.results()
    side = torch.cuda.Stream()
    for _ in range(5):
        st.scramble()
        torch.cuda.synchronize()
        st.run(side)
        side.synchronize()
        assert _same(st.results(), want)
    # outputs that the calls make themselves
    made = pa.select_blocks(st.q, st.codes, st.bscale, st.table, st.n, 6, stream=side)
    lens = pa.evict(st.k, st.v, st.w, st.table, st.n, st.fresh, 40, sinks=2, recent=5, head_dim=st.d, **st.s, stream=side)
    side.synchronize()
    assert torch.equal(made, st.blocks) and torch.equal(lens, st.new_lens)


def test_from_several_host_threads():
    steps = [Step("bf16", 10 + i) for i in range(4)]
    wants = []
    for st in steps:
        st.run()
        torch.cuda.synchronize()
        wants.append(st.results())
        st.scramble()
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            steps[i].run(s)
        s.synchronize()
        if not _same(steps[i].results(), wants[i]):
            bad.append(i)
        torch.cuda.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert pa.check_device_errors() == pa.PA_OK


def test_caches_past_4_gib():
    # offsets of blocks, bounds and sums beyond 32 bits
    hkv, d = 8, 128
    nb = 140_000  # 140000 * 8 * 16 * 128 * 2 bytes = 4.6 GB a cache
    k = torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    ids = torch.tensor([[139_999, 3, 139_000, 70_000, 139_998]], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in ids[0].tolist():
        k[i] = torch.randn(hkv, 16, d, generator=g, device="cuda").to(torch.bfloat16)
        v[i] = torch.randn(hkv, 16, d, generator=g, device="cuda").to(torch.bfloat16)
    small = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    ks, vs = k[ids[0].long()].contiguous(), v[ids[0].long()].contiguous()
    n = torch.tensor([75], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 1, 32, d, generator=g, device="cuda").to(torch.bfloat16)
    res = []
    for kk, vv, table in ((k, v, ids), (ks, vs, small)):
        codes = torch.zeros(len(kk), hkv, 2, d, dtype=torch.int8, device="cuda")
        sc = torch.zeros(len(kk), hkv, device="cuda")
        w = torch.zeros(len(kk), hkv, 16, device="cuda")
        pa.block_bounds(kk, table, n, 75, codes, sc)
        blocks = pa.select_blocks(q, codes, sc, table, n, 3)
        i32 = dict(dtype=torch.int32, device="cuda")
        res.append([blocks, pa.decode(q, kk, vv, table, n, 0.1, blocks=blocks),
                    pa.decode(q, kk, vv, table, n, 0.1, group_starts=torch.tensor([0, 1], **i32),
                              prefix_lens=torch.tensor([64], **i32)),
                    pa.decode(q, kk, vv, table, n, 0.1, weights=w), w[table[0].long()], codes[table[0].long()]])
    assert _same(*res)
    fresh = torch.tensor([[139_997, 139_996]], dtype=torch.int32, device="cuda")
    w = torch.zeros(nb, hkv, 16, device="cuda")
    w[ids[0].long()] = torch.rand(5, hkv, 16, generator=g, device="cuda")
    pa.evict(k, v, w, ids, n, fresh, 20, recent=20)
    last = torch.cat([k[i] for i in ids[0].tolist()], 1)[:, 55:75]
    assert torch.equal(torch.cat([k[i] for i in fresh[0].tolist()], 1)[:, :20], last)
    assert pa.check_device_errors() == pa.PA_OK
