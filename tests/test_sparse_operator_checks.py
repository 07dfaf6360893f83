"""Host-side argument checks of block bounds, selection, attention over listed blocks and behind shared prefixes, kept
weights and eviction through the C ABI, and their kernels' dependent launches: no call here reaches a GPU."""

import re

import pytest

import paged_kv_gqa_attn_gb300 as pa
from oracle import forms
from test_dependent_launches import WAIT, _all_sources, _body

FAKE = 1 << 20  # a 16-byte aligned non-null address that is never dereferenced


def _attn(name, *mid, lead=(), **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, lead=lead, B=0, M=4, NB=8, maxL=64, q_len=1, mid=mid, Hq=8, Hkv=2, d=128,
             bs=16, tail=(), scale=0.1, dt=0, ks=None, vs=None, out=FAKE)
    a.update(over)
    flat = []
    for v in a.values():
        flat += list(v) if isinstance(v, tuple) else [v]
    return getattr(pa.load_library(), "paged_attn_" + name)(*flat, None)


COMMON = [
    (dict(), pa.PA_OK),
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(out=None), pa.PA_ERR_INVALID_ARG),
    (dict(B=-1), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=9), pa.PA_ERR_INVALID_ARG),
    (dict(maxL=65), pa.PA_ERR_INVALID_ARG),
    (dict(dt=1), pa.PA_ERR_INVALID_ARG),
    (dict(dt=3), pa.PA_ERR_INVALID_ARG),
    (dict(dt=2), pa.PA_OK),
    (dict(d=32), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=32), pa.PA_ERR_UNSUPPORTED),
    (dict(q_len=17), pa.PA_ERR_INVALID_ARG),
    (dict(maxL=2 ** 30 + 1, M=2 ** 27), pa.PA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("name", ["sparse_decode", "sparse_verify"])
@pytest.mark.parametrize("over,status", COMMON + [
    (dict(lead=(None,)), pa.PA_ERR_INVALID_ARG),
    (dict(mid=(0,)), pa.PA_ERR_INVALID_ARG),
    (dict(mid=(-1,)), pa.PA_ERR_INVALID_ARG),
    (dict(mid=(1 << 26,)), pa.PA_OK),
    (dict(mid=((1 << 26) + 1,)), pa.PA_ERR_UNSUPPORTED),
    (dict(Hq=64), pa.PA_OK),
    (dict(Hq=66), pa.PA_ERR_UNSUPPORTED),
])
def test_sparse_checks(name, over, status):
    assert _attn(name, **{"lead": (FAKE,), "mid": (3,), **over}) == status


def test_sparse_and_prefix_verify_rows():
    assert _attn("sparse_verify", 3, lead=(FAKE,), q_len=8) == pa.PA_OK
    assert _attn("sparse_verify", 3, lead=(FAKE,), q_len=9) == pa.PA_ERR_UNSUPPORTED
    assert _attn("prefix_verify", 1, 64, 64, lead=(FAKE, FAKE), q_len=16) == pa.PA_OK
    assert _attn("prefix_verify", 1, 64, 64, lead=(FAKE, FAKE), q_len=16, Hq=18) == pa.PA_ERR_UNSUPPORTED
    assert _attn("sparse_decode", 3, lead=(FAKE,), q_len=2) == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["prefix_decode", "prefix_verify"])
@pytest.mark.parametrize("over,status", COMMON + [
    (dict(lead=(None, FAKE)), pa.PA_ERR_INVALID_ARG),
    (dict(lead=(FAKE, None)), pa.PA_ERR_INVALID_ARG),
    (dict(lead=(None, None), mid=(0, 64, 64)), pa.PA_OK),
    (dict(mid=(-1, 64, 64)), pa.PA_ERR_INVALID_ARG),
    (dict(mid=(1, -1, 64)), pa.PA_ERR_INVALID_ARG),
    (dict(mid=(1, 64, -1)), pa.PA_ERR_INVALID_ARG),
    (dict(mid=(1, 65, 64)), pa.PA_ERR_INVALID_ARG),
    (dict(mid=(1, 64, 2 ** 31 - 1)), pa.PA_OK),
    (dict(mid=(65535, 64, 64)), pa.PA_OK),
    (dict(mid=(65536, 64, 64)), pa.PA_ERR_UNSUPPORTED),
])
def test_prefix_checks(name, over, status):
    assert _attn(name, **{"lead": (FAKE, FAKE), "mid": (1, 64, 64), **over}) == status


def test_prefix_tiles_fit_a_grid_dimension():
    # 65535 sequences of 16 rows, groups of 8: 16 tokens a tile; the empty batch passes every check before it
    assert _attn("prefix_verify", 65535, 64, 64, lead=(FAKE, FAKE), q_len=16, Hq=16, B=0) == pa.PA_OK
    assert _attn("prefix_verify", 65535, 64, 64, lead=(FAKE, FAKE), q_len=16, Hq=16, B=65535) == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("over,status", COMMON + [
    (dict(lead=(None,)), pa.PA_ERR_INVALID_ARG),
    (dict(lead=(FAKE + 4,)), pa.PA_ERR_INVALID_ARG),
    (dict(tail=(float("nan"),)), pa.PA_ERR_INVALID_ARG),
    (dict(tail=(float("inf"),)), pa.PA_ERR_INVALID_ARG),
    (dict(tail=(-0.5,)), pa.PA_OK),
    (dict(Hq=64), pa.PA_OK),
    (dict(Hq=66), pa.PA_ERR_UNSUPPORTED),
    (dict(q_len=2), pa.PA_ERR_INVALID_ARG),
])
def test_weighted_checks(over, status):
    assert _attn("weighted_decode", **{"lead": (FAKE,), "tail": (0.9,), **over}) == status


def _bounds(**over):
    a = dict(k=FAKE, bt=FAKE, cl=FAKE, B=0, n=1, M=4, NB=8, Hkv=2, d=128, bs=16, dt=0, ks=None, bounds=FAKE, scale=FAKE)
    a.update(over)
    return pa.load_library().paged_attn_block_bounds(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(), pa.PA_OK),
    (dict(B=2, n=0), pa.PA_OK),
    (dict(n=2 ** 31 - 1), pa.PA_OK),
    (dict(k=None), pa.PA_ERR_INVALID_ARG),
    (dict(bounds=None), pa.PA_ERR_INVALID_ARG),
    (dict(scale=None), pa.PA_ERR_INVALID_ARG),
    (dict(n=-1), pa.PA_ERR_INVALID_ARG),
    (dict(dt=1), pa.PA_ERR_INVALID_ARG),
    (dict(dt=1, ks=FAKE), pa.PA_OK),
    (dict(dt=2), pa.PA_OK),
    (dict(dt=3), pa.PA_ERR_INVALID_ARG),
    (dict(k=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(bounds=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(d=96), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=32), pa.PA_ERR_UNSUPPORTED),
    (dict(B=65536), pa.PA_ERR_UNSUPPORTED),
    (dict(M=2 ** 27), pa.PA_ERR_UNSUPPORTED),
])
def test_bounds_checks(over, status):
    assert _bounds(**over) == status


def _select(**over):
    a = dict(q=FAKE, bounds=FAKE, scale=FAKE, bt=FAKE, cl=FAKE, B=0, M=4, NB=8, maxL=64, q_len=1, Hq=8, Hkv=2, d=128, bs=16,
             count=4, sinks=1, recent=2, out=FAKE)
    a.update(over)
    return pa.load_library().paged_attn_select_blocks(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(), pa.PA_OK),
    (dict(out=None), pa.PA_ERR_INVALID_ARG),
    (dict(scale=None), pa.PA_ERR_INVALID_ARG),
    (dict(count=0), pa.PA_ERR_INVALID_ARG),
    (dict(count=2), pa.PA_ERR_INVALID_ARG),
    (dict(count=3), pa.PA_OK),
    (dict(sinks=-1), pa.PA_ERR_INVALID_ARG),
    (dict(recent=-1), pa.PA_ERR_INVALID_ARG),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1, count=2 ** 31 - 1), pa.PA_ERR_INVALID_ARG),
    (dict(maxL=65), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=7), pa.PA_ERR_INVALID_ARG),
    (dict(q=FAKE + 2), pa.PA_ERR_INVALID_ARG),
    (dict(bounds=FAKE + 4), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=64), pa.PA_OK),
    (dict(Hq=66), pa.PA_ERR_UNSUPPORTED),
    (dict(q_len=9), pa.PA_ERR_UNSUPPORTED),
    (dict(q_len=2 ** 30, Hq=16), pa.PA_ERR_UNSUPPORTED),
    (dict(d=32), pa.PA_ERR_UNSUPPORTED),
    (dict(maxL=2 ** 30 + 1, M=2 ** 27), pa.PA_ERR_UNSUPPORTED),
])
def test_select_checks(over, status):
    assert _select(**over) == status


def _evict(**over):
    a = dict(k=FAKE, v=FAKE, w=FAKE, bt=FAKE, cl=FAKE, nt=FAKE, B=0, M=4, M2=2, NB=8, maxL=64, Hkv=2, d=128, bs=16, dt=0,
             ks=None, vs=None, keep=20, sinks=2, recent=3, out=FAKE)
    a.update(over)
    return pa.load_library().paged_attn_evict(*a.values(), None)


@pytest.mark.parametrize("over,status", [
    (dict(), pa.PA_OK),
    (dict(w=None), pa.PA_ERR_INVALID_ARG),
    (dict(nt=None), pa.PA_ERR_INVALID_ARG),
    (dict(w=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(out=None), pa.PA_ERR_INVALID_ARG),
    (dict(B=3), pa.PA_ERR_INVALID_ARG),  # new_lens is context_lens
    (dict(B=3, out=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(B=3, out=FAKE - 8), pa.PA_ERR_INVALID_ARG),
    (dict(keep=0), pa.PA_ERR_INVALID_ARG),
    (dict(keep=32), pa.PA_OK),
    (dict(keep=33), pa.PA_ERR_INVALID_ARG),
    (dict(sinks=18), pa.PA_ERR_INVALID_ARG),
    (dict(sinks=17), pa.PA_OK),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), pa.PA_ERR_INVALID_ARG),
    (dict(recent=-1), pa.PA_ERR_INVALID_ARG),
    (dict(M2=0), pa.PA_ERR_INVALID_ARG),
    (dict(maxL=65), pa.PA_ERR_INVALID_ARG),
    (dict(dt=1), pa.PA_ERR_INVALID_ARG),
    (dict(dt=1, ks=FAKE, vs=FAKE), pa.PA_OK),
    (dict(dt=2), pa.PA_OK),
    (dict(v=FAKE + 8), pa.PA_ERR_INVALID_ARG),
    (dict(d=32), pa.PA_ERR_UNSUPPORTED),
    (dict(B=65536), pa.PA_ERR_UNSUPPORTED),
])
def test_evict_checks(over, status):
    assert _evict(**over) == status


DEPENDENTS = {"block_pick_kernel", "fold_weights_kernel", "evict_move_kernel"}
BESIDE = {"decode_mma_kernel", "rows_mma_kernel", "prefill_tc_kernel"}  # over own tokens, beside the prefixes


def _without_lambdas(body):
    return re.sub(r"\[&\]\([^)]*\)\s*\{[^{}]*\}", "", body)


def test_every_dependent_waits_before_it_returns():
    """What launch_dependent launches behind a kernel whose outputs it reads: the wait stands in front of the first return,
    whatever the data."""
    found = set()
    for name, text in _all_sources().items():
        if "launch_dependent(" not in text or name in ("pa_api.cu", "pa_kernels.h"):
            continue
        for kernel in re.findall(r"__global__[^;{]*?\b(\w+_kernel)\(", text):
            body = _without_lambdas(_body(text, kernel))
            if WAIT in body:
                found.add(kernel)
                assert "return" not in body[: body.index(WAIT)], kernel
                head = re.search(r"__global__[^;{]*?\b%s\([^{;]*\{" % kernel, text).group(0)
                assert "__restrict__" not in head, kernel
    assert found == DEPENDENTS


@pytest.mark.parametrize("kernel", sorted(BESIDE))
def test_the_first_cta_over_own_tokens_ends_after_the_prefixes(kernel):
    """They read nothing of the prefixes' grid; the merge that waits for them reads both.  Every way out of their first CTA
    (partition 0, which none of the returns for a partition past the pages concerns) passes the wait, and it is last."""
    text = next(t for t in _all_sources().values() if re.search(r"__global__[^;{]*\b%s\(" % kernel, t))
    body = _body(text, kernel)
    assert body.rstrip().rstrip("}").rstrip().splitlines()[-1].strip() in (
        "if constexpr (OWN) after_prefixes();", "#endif"), kernel
    zeros = body.index("__float2bfloat16(0.f);")  # the rows of a sequence without tokens
    assert body[zeros: body.index("return;", zeros)].count("after_prefixes()") == 1
    device = _all_sources()["pa_device.cuh"]
    at = device.index("void after_prefixes()")
    assert "blockIdx.x | blockIdx.y | blockIdx.z) == 0" in device[at: at + 200] and WAIT in device[at: at + 200]


def test_the_oracle_on_closed_cases():
    assert [forms.code_exp(x) for x in (0, 127.0, 127.5, 1.0, 127 / 64, 2.0, 2.0 ** -140)] == [0, 0, 1, -6, -6, -5, -126]
    assert forms.pick([3, 1, 2, 2, 0], 3, 0, 1).tolist() == [0, 2, 4]
    assert forms.evict_positions([5.0, float("nan"), 1.0, 1.0, 0.0], 3, 0, 1).tolist() == [0, 2, 4]
    assert forms.evict_positions([float("-inf"), float("nan"), 1.0], 2, 0, 0).tolist() == [0, 2]
