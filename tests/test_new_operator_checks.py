"""Host-side argument checks of qk_norm_rope, read_kv and the 4-bit cache type through the C ABI: no
call here reaches a GPU."""

import ctypes

import pytest

import paged_kv_gqa_attn_gb300 as pa

FAKE = 1 << 20  # a 16-byte aligned non-null address that is never dereferenced


def _rope(**over):
    a = dict(q=FAKE, k=FAKE, qw=FAKE, kw=FAKE, cs=FAKE, pos=FAKE, T=0, Hq=8, Hkv=2, d=128, rot=128, inter=0,
             P=100, eps=1e-6, qs=1024, ks=256, qos=1024, kos=256, qo=FAKE, ko=FAKE)
    a.update(over)
    return pa.load_library().paged_attn_qk_norm_rope(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(), pa.PA_OK),
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(pos=None), pa.PA_ERR_INVALID_ARG),
    (dict(ko=None), pa.PA_ERR_INVALID_ARG),
    (dict(T=-1), pa.PA_ERR_INVALID_ARG),
    (dict(Hkv=0), pa.PA_ERR_INVALID_ARG),
    (dict(P=0), pa.PA_ERR_INVALID_ARG),
    (dict(eps=-1e-6), pa.PA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), pa.PA_ERR_INVALID_ARG),
    (dict(eps=float("inf")), pa.PA_ERR_INVALID_ARG),
    (dict(qs=1016), pa.PA_ERR_INVALID_ARG),
    (dict(kos=257), pa.PA_ERR_INVALID_ARG),
    (dict(q=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(cs=FAKE + 4), pa.PA_ERR_INVALID_ARG),
    (dict(d=96), pa.PA_ERR_UNSUPPORTED),
    (dict(rot=0), pa.PA_ERR_UNSUPPORTED),
    (dict(rot=24), pa.PA_ERR_UNSUPPORTED),
    (dict(rot=144), pa.PA_ERR_UNSUPPORTED),
])
def test_qk_norm_rope_checks(over, status):
    assert _rope(**over) == status


def _read(**over):
    a = dict(k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, B=0, n=1, M=4, NB=8, Hkv=2, d=128, bs=16, dt=2, ks=None, vs=None,
             ko=FAKE, vo=FAKE)
    a.update(over)
    return pa.load_library().paged_attn_read_kv(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(), pa.PA_OK),
    (dict(B=2, n=0), pa.PA_OK),
    (dict(k=None), pa.PA_ERR_INVALID_ARG),
    (dict(vo=None), pa.PA_ERR_INVALID_ARG),
    (dict(n=65), pa.PA_ERR_INVALID_ARG),
    (dict(n=-1), pa.PA_ERR_INVALID_ARG),
    (dict(dt=3), pa.PA_ERR_INVALID_ARG),
    (dict(dt=1), pa.PA_ERR_INVALID_ARG),
    (dict(ko=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(d=32), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
    (dict(B=65536), pa.PA_ERR_UNSUPPORTED),
])
def test_read_kv_checks(over, status):
    assert _read(**over) == status


def test_append_takes_the_4_bit_type_without_scales():
    fn = pa.load_library().paged_attn_append_kv
    lead = [FAKE] * 6
    assert fn(*lead, 0, 1, 4, 8, 2, 128, 16, 2, None, None, None) == pa.PA_OK
    assert fn(*lead, 0, 1, 4, 8, 2, 128, 16, 3, None, None, None) == pa.PA_ERR_INVALID_ARG
    assert fn(*lead, 0, 1, 4, 8, 2, 128, 16, 1, None, None, None) == pa.PA_ERR_INVALID_ARG


def _attn(name, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, B=0, M=4, NB=8, maxL=64, q_len=1, Hq=8, Hkv=2, d=128, bs=16,
             window=5, sinks=2, scale=0.1, dt=0, ks=None, vs=None, out=FAKE)
    a.update(over)
    if name in ("decode", "verify"):
        del a["window"], a["sinks"]
    return getattr(pa.load_library(), "paged_attn_" + name)(*a.values(), None)


@pytest.mark.parametrize("name", ["window_decode", "window_verify"])
@pytest.mark.parametrize("over,status", [
    (dict(), pa.PA_OK),
    (dict(window=0), pa.PA_ERR_INVALID_ARG),
    (dict(window=-4), pa.PA_ERR_INVALID_ARG),
    (dict(sinks=-1), pa.PA_ERR_INVALID_ARG),
    (dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), pa.PA_OK),
    (dict(maxL=2 ** 30 + 1, M=2 ** 27), pa.PA_ERR_UNSUPPORTED),
    (dict(out=None), pa.PA_ERR_INVALID_ARG),
    (dict(dt=1), pa.PA_ERR_INVALID_ARG),
    (dict(dt=2), pa.PA_OK),
    (dict(d=32), pa.PA_ERR_UNSUPPORTED),
])
def test_window_checks(name, over, status):
    assert _attn(name, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(dt=2), pa.PA_OK),
    (dict(dt=3), pa.PA_ERR_INVALID_ARG),
    (dict(dt=2, Hq=256), pa.PA_ERR_UNSUPPORTED),
    (dict(dt=2, k=FAKE + 8), pa.PA_ERR_INVALID_ARG),
])
def test_4_bit_decode_checks(over, status):
    assert _attn("decode", **over) == status


def test_static_scratch_decode_refuses_the_4_bit_type():
    fn = pa.load_library().paged_attn_decode_static_scratch
    P, I = ctypes.c_void_p, ctypes.c_int
    fn.restype, fn.argtypes = I, [P] * 5 + [I] * 9 + [ctypes.c_float, I] + [P] * 4
    a = [FAKE] * 5 + [2, 4, 8, 64, 1, 8, 2, 128, 16, 0.1]
    assert fn(*a, 2, None, None, FAKE, None) == pa.PA_ERR_UNSUPPORTED


def test_window_prefill_checks():
    fn = pa.load_library().paged_attn_window_prefill
    lead = [FAKE] * 6 + [0, 0, 1, 4, 8, 64, 8, 2, 128, 16]
    assert fn(*lead, 5, 2, 0.1, 2, None, None, FAKE, None) == pa.PA_OK
    assert fn(*lead, 0, 2, 0.1, 0, None, None, FAKE, None) == pa.PA_ERR_INVALID_ARG
    assert fn(*lead, 5, -2, 0.1, 0, None, None, FAKE, None) == pa.PA_ERR_INVALID_ARG
    assert fn(*lead, 5, 2, 0.1, 4, None, None, FAKE, None) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("kv", [0, 2])
def test_prefill_takes_at_most_65536_sequences(kv):
    # the planner packs a sequence and a tile into one word; no rows, so that no accepted call reaches a GPU
    lib = pa.load_library()
    for seqs, status in ((65536, pa.PA_OK), (65537, pa.PA_ERR_UNSUPPORTED)):
        lead = [FAKE] * 6 + [seqs, 0, 1, 4, 8, 64, 8, 2, 128, 16]
        assert lib.paged_attn_window_prefill(*lead, 5, 2, 0.1, kv, None, None, FAKE, None) == status
        assert lib.paged_attn_prefill(*lead, 0.1, kv, None, None, FAKE, None) == status


def test_plan_of_4_bit_pages():
    pa.set_max_partitions(0)
    for units_b, pages in ((1, 513), (16, 257), (64, 2048), (256, 100), (1, 1)):
        ppp, parts = pa.plan(152, units_b, 8, pages * 16, kv_dtype=pa.PA_KV_FP4_E2M1)
        assert ppp * parts >= pages and ppp * (parts - 1) < pages and parts <= 64
    # few contexts are cut finely, many coarsely
    assert pa.plan(152, 1, 8, 8208, kv_dtype=pa.PA_KV_FP4_E2M1)[1] > 16
    assert pa.plan(152, 512, 8, 2048, kv_dtype=pa.PA_KV_FP4_E2M1)[1] == 1


def test_an_e4m3_cache_takes_no_per_head_scales(monkeypatch):
    # the check of the scales' size alone: the tensors are on the host, where the device check would refuse
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(pa, "_check_cuda", lambda name, t, dtypes: None)
    cache = torch.zeros(5, 2, 16, 128, dtype=torch.uint8)
    per_page, per_head = torch.ones(5, 2), torch.ones(2)
    assert pa._kv_dtype(cache, cache, 128, per_page, per_page) == pa.PA_KV_FP8_E4M3
    for scales in ((per_head, per_head), (per_page, per_head), (per_head, per_page)):
        with pytest.raises(ValueError, match="num_blocks"):
            pa._kv_dtype(cache, cache, 128, *scales)
