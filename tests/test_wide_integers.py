"""Integer arguments beyond 32 bits: a window, sinks or bounds of 2^32 + 5 are not 5.  The library is a stand-in
that records what it is called with; no GPU is reached."""

import ctypes

import pytest
import torch

import paged_kv_gqa_attn_gb300 as pa

BIG = (1 << 31) - 1


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            # as ctypes passes them: the low 32 bits of an int
            self.calls.append((name, [ctypes.c_int(a).value if type(a) is int and abs(a) >= 1 << 31 else a for a in args]))
            return pa.PA_OK
        return fn


@pytest.fixture
def library(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(pa, "load_library", lambda: rec)
    monkeypatch.setattr(pa, "_check_cuda", lambda name, t, dtypes: None)
    monkeypatch.setattr(pa, "_one_device", lambda *a, **k: pa._HERE)
    monkeypatch.setattr(pa, "_stream_handle", lambda s: None)
    return rec


def _caches():
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    return k, k.clone(), torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)


@pytest.mark.parametrize("wide", [(1 << 32) + 5, (1 << 31) + 5, 1 << 40])
def test_a_wide_window_hides_nothing(library, wide):
    k, v, table, lens = _caches()
    q = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    pa.decode(q, k, v, table, lens, 0.1, window=wide, sinks=wide)
    pa.verify(q, k, v, table, lens, 0.1, window=wide, sinks=0)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32)
    pa.prefill(q[:, 0], k, v, table, lens, starts, 0.1, max_q_len=1, window=wide, sinks=wide)
    names = [n for n, _ in library.calls]
    assert names == ["paged_attn_window_decode", "paged_attn_window_verify", "paged_attn_window_prefill"]
    assert library.calls[0][1][14:16] == [BIG, BIG]
    assert library.calls[1][1][14:16] == [BIG, 0]
    assert library.calls[2][1][16:18] == [BIG, BIG]


def test_negative_and_bounding_arguments_keep_their_side(library):
    k, v, table, lens = _caches()
    q = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    pa.decode(q, k, v, table, lens, 0.1, window=-(1 << 32) + 7, max_context_len=(1 << 32) + 16)
    args = library.calls[-1][1]
    assert args[14] < 0 and args[8] == BIG  # refused by the library, as any other
    starts = torch.tensor([0, 1, 2], dtype=torch.int32)
    pa.prefill(q[:, 0], k, v, table, lens, starts, 0.1, max_q_len=(1 << 32) + 1, max_context_len=1 << 33)
    args = library.calls[-1][1]
    assert args[8] == BIG and args[11] == BIG
    pa.set_max_partitions(1 << 32)
    assert library.calls[-1][1] == [BIG]


def test_the_library_refuses_what_is_too_large():
    with pytest.raises(pa.PagedAttnError):
        pa.set_max_partitions(1 << 32)  # (0 would be "automatic")
    with pytest.raises(pa.PagedAttnError):
        pa.plan(152, -(1 << 32) + 3, 8, 4096)  # (3 would be three sequences)
