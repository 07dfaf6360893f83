"""Outputs that a call makes itself while it is given a stream: they lie in that stream's memory, so that no
block which work on the current stream may still use is written, and they hold the call's result."""

import pytest
import torch

import attn_cases as A
import paged_kv_gqa_attn_gb300 as pa

pytestmark = pytest.mark.gpu


def _stream_of(t):
    """The stream whose memory a tensor lies in, by the allocator's own account."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any segment")


def _calls():
    for form, kv in (("decode", "bf16"), ("verify", "e4m3"), ("prefill", "fp4")):
        r = [1, 1] if form == "decode" else [4, 4]
        c = A.make(kv, [300, 70], r, 8, 2, 128, seed=5, window=100, sinks=4)
        dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
        more = {"max_q_len": 4} if form == "prefill" else {}
        yield form, lambda dev=dev, form=form, more=more, **kw: [A.call(dev, form, **more, **kw)]
    c = A.make("fp4", [300, 70], [1, 1], 8, 2, 128, seed=6, window=None)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    scales = {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"]}
    yield "read_kv", lambda **kw: list(pa.read_kv(dev["k"], dev["v"], dev["table"], lens, 50, **scales, **kw))
    q, k = (torch.randn(7, h, 128, device="cuda").bfloat16() for h in (8, 2))
    w = torch.ones(128, device="cuda").bfloat16()
    turns = torch.rand(16, 128, device="cuda")
    pos = torch.arange(7, device="cuda", dtype=torch.int32)
    yield "qk_norm_rope", lambda **kw: list(pa.qk_norm_rope(q, k, w, w, turns, pos, **kw))
    p, d = (torch.softmax(torch.randn(3, n, 50, device="cuda"), -1) for n in (4, 3))
    draft = torch.zeros(3, 3, dtype=torch.int32, device="cuda")
    u = torch.rand(3, 3, device="cuda")
    words = torch.arange(3, dtype=torch.int32, device="cuda")
    yield "spec_accept", lambda **kw: list(pa.spec_accept(p, d, draft, u, words, **kw))


def test_outputs_lie_in_the_memory_of_the_stream_that_writes_them():
    here = torch.cuda.current_stream()
    for name, call in _calls():
        want = call()
        assert all(_stream_of(t) == here.cuda_stream for t in want), name
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = call(stream=side)
        here.wait_stream(side)
        assert all(_stream_of(t) == side.cuda_stream for t in got), name
        assert all(torch.equal(g, w) for g, w in zip(got, want)), name
        # handed to the current stream: dropped and made again while it still reads, nothing is overwritten
        copies = [t * 1 for t in got]
        del got
        again = call(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(copies, want)), name
        assert all(torch.equal(g, w) for g, w in zip(again, want)), name
    assert pa.check_device_errors() == pa.PA_OK


def test_a_given_stream_inside_a_capture():
    c = A.make("fp4", [900, 70], [5, 5], 8, 2, 128, seed=8)
    dev = {n: (t.cuda() if torch.is_tensor(t) else t) for n, t in c.items()}
    lens = torch.tensor(c["lens"], dtype=torch.int32, device="cuda")
    q = dev["q"].view(2, 5, 8, 128)
    kw = {"k_scale": dev["k_scale"], "v_scale": dev["v_scale"]}
    want = pa.verify(q, dev["k"], dev["v"], dev["table"], lens, c["scale"], **kw)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        out = pa.verify(q, dev["k"], dev["v"], dev["table"], lens, c["scale"], stream=side, **kw)
        here.wait_stream(side)
        after = out * 1
    for _ in range(5):
        out.zero_()
        after.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(after, want)
    assert pa.check_device_errors() == pa.PA_OK
