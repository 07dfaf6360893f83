"""GB300 (sm_103a) paged-KV GQA attention: decode and speculative verify.

A thin Python binding over the C ABI in ``include/paged_attn.h``: it checks tensor devices
and dtypes, passes raw device pointers and sizes, and raises on a non-zero status.  All the
arithmetic runs in the library's CUDA kernels; there is no fallback.  PyTorch only provides
device memory and streams.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "PagedAttnError",
    "decode",
    "verify",
    "tree_verify",
    "prefill",
    "append_kv",
    "read_kv",
    "block_bounds",
    "select_blocks",
    "evict",
    "qk_norm_rope",
    "spec_accept",
    "check_device_errors",
    "set_max_partitions",
    "plan",
    "status_string",
    "version",
    "library_path",
    "load_library",
]

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_CUDA = 3
PA_ERR_NO_MEMORY = 4
PA_ERR_DEVICE_BOUNDS = 5
PA_ERR_DEVICE_TIMEOUT = 6
PA_ERR_SCRATCH_LIMIT = 7
PA_KV_BF16 = 0
PA_KV_FP8_E4M3 = 1
PA_KV_FP4_E2M1 = 2
PA_WAIT_LIMIT = 1 << 18   # suspending mbarrier polls before a kernel wait gives up
PA_SPIN_LIMIT = 1 << 22   # non-suspending probe iterations before an issuer loop gives up

_lib = None
_lock = threading.Lock()


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = True, timeline: Optional[bool] = None):
    """Load the in-tree shared library (building it first when it is missing or stale), or return
    the one already loaded.

    timeline=True loads the instrumented variant instead (per-CTA time stamps in the verify
    kernel, for ``paged_kv_gqa_attn_gb300.timeline``); it must be the first load of the process."""
    global _lib
    if _lib is not None and (timeline is None or timeline == _lib._pa_timeline):
        return _lib
    with _lock:
        if _lib is not None and timeline is not None and timeline != _lib._pa_timeline:
            raise RuntimeError("the other variant of the library is already loaded in this process")
        if _lib is None:
            timeline = bool(timeline)
            path = _build.TIMELINE_LIB_PATH if timeline else _build.LIB_PATH
            if build_if_missing and not _build.up_to_date(timeline):
                _build.build(timeline=timeline)
            if not os.path.exists(path):
                raise RuntimeError(f"paged attention library not built: {path}")
            lib = ctypes.CDLL(path)
            lib._pa_timeline = timeline
            P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            attn_args = [P, P, P, P, P, I, I, I, I, I, I, I, I, I, F, I, P, P, P, P]
            for name in ("paged_attn_decode", "paged_attn_verify"):
                fn = getattr(lib, name)
                fn.restype = I
                fn.argtypes = attn_args
            lib.paged_attn_tree_verify.restype = I
            lib.paged_attn_tree_verify.argtypes = attn_args[:5] + [P] + attn_args[5:]
            lib.paged_attn_prefill.restype = I
            lib.paged_attn_prefill.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F, I, P, P, P, P]
            for name in ("paged_attn_window_decode", "paged_attn_window_verify"):
                fn = getattr(lib, name)
                fn.restype = I
                fn.argtypes = attn_args[:14] + [I, I] + attn_args[14:]
            lib.paged_attn_window_prefill.restype = I
            lib.paged_attn_window_prefill.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, I, I, F, I, P,
                                                      P, P, P]
            lib.paged_attn_append_kv.restype = I
            lib.paged_attn_append_kv.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, P, P, P]
            lib.paged_attn_read_kv.restype = I
            lib.paged_attn_read_kv.argtypes = [P, P, P, P, I, I, I, I, I, I, I, I, P, P, P, P, P]
            for name in ("paged_attn_sparse_decode", "paged_attn_sparse_verify"):
                fn = getattr(lib, name)
                fn.restype = I
                fn.argtypes = attn_args[:5] + [P] + attn_args[5:10] + [I] + attn_args[10:]
            for name in ("paged_attn_prefix_decode", "paged_attn_prefix_verify"):
                fn = getattr(lib, name)
                fn.restype = I
                fn.argtypes = attn_args[:5] + [P, P] + attn_args[5:10] + [I, I, I] + attn_args[10:]
            lib.paged_attn_weighted_decode.restype = I
            lib.paged_attn_weighted_decode.argtypes = attn_args[:5] + [P] + attn_args[5:14] + [F] + attn_args[14:]
            lib.paged_attn_block_bounds.restype = I
            lib.paged_attn_block_bounds.argtypes = [P, P, P, I, I, I, I, I, I, I, I, P, P, P, P]
            lib.paged_attn_select_blocks.restype = I
            lib.paged_attn_select_blocks.argtypes = [P, P, P, P, P] + [I] * 12 + [P, P]
            lib.paged_attn_evict.restype = I
            lib.paged_attn_evict.argtypes = [P] * 6 + [I] * 9 + [P, P] + [I] * 3 + [P, P]
            L = ctypes.c_int64
            lib.paged_attn_qk_norm_rope.restype = I
            lib.paged_attn_qk_norm_rope.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, F, L, L, L, L, P, P, P]
            lib.paged_attn_spec_accept.restype = I
            lib.paged_attn_spec_accept.argtypes = [P, P, P, P, P, I, I, I, P, P, P]
            lib.paged_attn_check_device_errors.restype = I
            lib.paged_attn_check_device_errors.argtypes = [P]
            lib.paged_attn_selftest_wait.restype = I
            lib.paged_attn_selftest_wait.argtypes = [I, ctypes.c_uint, P, P]
            lib.paged_attn_status_string.restype = ctypes.c_char_p
            lib.paged_attn_status_string.argtypes = [I]
            lib.paged_attn_set_max_partitions.restype = I
            lib.paged_attn_set_max_partitions.argtypes = [I]
            lib.paged_attn_plan.restype = I
            lib.paged_attn_plan.argtypes = [I, I, I, I, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I)]
            lib.paged_attn_version.restype = I
            lib.paged_attn_version.argtypes = []
            _lib = lib
    return _lib


def _c_int(v) -> int:
    """An integer argument as the C int it is passed as: beyond the type, its largest (smallest) value, which the
    library takes or refuses like any other that large.  (ctypes would keep the low 32 bits.)"""
    return max(-(1 << 31), min((1 << 31) - 1, int(v)))


def status_string(status: int) -> str:
    return load_library().paged_attn_status_string(int(status)).decode()


def version() -> int:
    return int(load_library().paged_attn_version())


def set_max_partitions(p: int) -> None:
    """Force at most p split-KV partitions per sequence (0 = automatic, 1 = no split)."""
    st = load_library().paged_attn_set_max_partitions(_c_int(p))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_set_max_partitions")


def plan(num_sms: int, num_seqs: int, num_kv_heads: int, max_context_len: int, block_size: int = 16,
         q_len: int = 1, kv_dtype: int = PA_KV_BF16):
    """(pages_per_partition, max_partitions) the library chooses for decode of this shape (4-bit caches: groups
    of up to 8; q_len other than 1 is refused).  See paged_attn_plan."""
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    shape = map(_c_int, (num_sms, num_seqs, num_kv_heads, max_context_len, block_size, q_len, kv_dtype))
    st = load_library().paged_attn_plan(*shape, ctypes.byref(a), ctypes.byref(b))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_plan")
    return a.value, b.value


# The current stream's handle of a device, without building a Stream object (0.1 us against 3 us); and
# the index of the current device.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_handle(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is None:
        return _raw_stream(_current_device())
    return int(stream.cuda_stream)


def check_device_errors(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise the stream and return (and clear) the error status of its device."""
    with torch.cuda.device(stream.device if stream is not None else torch.cuda.current_device()):
        return int(load_library().paged_attn_check_device_errors(_stream_handle(stream)))


def selftest_wait(helper: int, polls: int, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Launch the failure-detection self-test: a bounded kernel wait on an mbarrier that never
    completes (helper 0: the decode kernels' wait, 1: the tcgen05 kernels', 2: the
    non-suspending probe loop of the tensor-core issuers), cut off after `polls` polls.  Returns
    a one-element int64 CUDA tensor with the wait's wall time in ns; the timeout shows up as
    PA_ERR_DEVICE_TIMEOUT in check_device_errors()."""
    s = stream if stream is not None else torch.cuda.current_stream()
    elapsed = torch.zeros(1, dtype=torch.int64, device=s.device)
    with torch.cuda.device(s.device):
        st = load_library().paged_attn_selftest_wait(int(helper), int(polls), elapsed.data_ptr(), _stream_handle(s))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_selftest_wait")
    return elapsed


class _Here:
    """The context of a call on the current device: nothing to change."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def _one_device(stream, *tensors, names="", **named):
    """Check that every tensor (and the stream, if one is given) is on one CUDA device and return
    a context that makes it the current device for the call: the library launches on the
    current device.  names: the tensors' names in order, for the error."""
    if named:
        tensors += tuple(named.values())
    index = None
    for t in tensors:
        if t is not None:
            at = t.get_device()
            if at != index:
                if index is not None or at < 0:
                    names = " ".join([names, *named])
                    where = {n: str(x.device) for n, x in zip(names.split(), tensors) if x is not None}
                    raise ValueError(f"tensors must be on one CUDA device, got {where}")
                index = at
    if index is None:
        raise ValueError("tensors must be on one CUDA device, got none")
    if stream is not None and stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, tensors on cuda:{index}")
    return _HERE if _current_device() == index else torch.cuda.device(index)


def _check_cuda(name, t, dtypes):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    raise ValueError(f"{name} must be contiguous")


# (names of the accepted types, made once: every call passes them)
_BF16, _I32, _F32, _BYTES = (torch.bfloat16,), (torch.int32,), (torch.float32,), (torch.uint8,)
_I8 = (torch.int8,)
_E4M3 = (torch.uint8, torch.float8_e4m3fn)


def _kv_dtype(k_cache, v_cache, head_dim, k_scale, v_scale):
    """The cache type by the caches' dtype and last dim (bf16 [.., d], E4M3 bytes [.., d], 4-bit bytes
    [.., 9 d / 16]), with the checks of the scales that it takes."""
    dtype = k_cache.dtype
    if dtype is torch.bfloat16:
        _check_cuda("k_cache", k_cache, _BF16)
        _check_cuda("v_cache", v_cache, _BF16)
        return PA_KV_BF16
    if dtype is torch.uint8 and k_cache.dim() == 4 and 16 * k_cache.shape[3] == 9 * head_dim:
        _check_cuda("k_cache", k_cache, _BYTES)
        _check_cuda("v_cache", v_cache, _BYTES)
        heads = k_cache.shape[1:2]
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None:
                _check_cuda(name, t, _F32)
                if t.shape != heads:
                    raise ValueError(f"{name} must be [num_kv_heads] for a 4-bit cache")
        return PA_KV_FP4_E2M1
    _check_cuda("k_cache", k_cache, _E4M3)
    _check_cuda("v_cache", v_cache, _E4M3)
    _check_cuda("k_scale", k_scale, _F32)
    _check_cuda("v_scale", v_scale, _F32)
    if k_cache.dim() == 4 and min(k_scale.numel(), v_scale.numel()) < k_cache.shape[0] * k_cache.shape[1]:
        raise ValueError("k_scale / v_scale must be [num_blocks, num_kv_heads]")  # (per-head ones are the 4-bit cache's)
    return PA_KV_FP8_E4M3


def _ptr(t):
    return None if t is None else t.data_ptr()


def _new(shape, like, stream, dtype=torch.bfloat16):
    """An output that a call makes itself.  It comes from the memory of the stream that writes it: a block of
    the current stream's could still be read there by work that was queued before it was freed, and the
    given stream does not wait for that.  The caller's stream, which the output is handed to, is recorded."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=like.device)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


_WINDOW_FORMS = {"paged_attn_decode": "paged_attn_window_decode", "paged_attn_verify": "paged_attn_window_verify",
                 "paged_attn_prefill": "paged_attn_window_prefill"}


def _window(fn_name, window, sinks):
    """The C entry of a call with or without a window, and the window's arguments."""
    if window is None:
        if sinks:
            raise ValueError("sinks need a window: without one every token is visible")
        return fn_name, ()
    return _WINDOW_FORMS[fn_name], (_c_int(window), _c_int(sinks))


_EXTRA_FORMS = {
    "blocks": {"paged_attn_decode": "paged_attn_sparse_decode", "paged_attn_verify": "paged_attn_sparse_verify"},
    "prefix": {"paged_attn_decode": "paged_attn_prefix_decode", "paged_attn_verify": "paged_attn_prefix_verify"},
    "weights": {"paged_attn_decode": "paged_attn_weighted_decode"},
}


def _extra(fn_name, shape, cache_shape, max_context_len, blocks, group_starts, prefix_lens, max_prefix_len, max_own_len,
           weights, decay, window):
    """The C entry of a call over listed blocks, with shared prefixes or with sums of the weights; its pointers behind
    the context lengths, its integers behind q_len, its floats before the scale, and the tensors to check the device of."""
    given = [n for n, t in (("blocks", blocks), ("prefix", group_starts), ("weights", weights)) if t is not None]
    if window is not None:
        given.append("window")
    if len(given) > 1:
        raise ValueError(f"a call takes one of blocks, group_starts, weights and window, got {given}")
    if group_starts is None and (prefix_lens is not None or max_prefix_len is not None or max_own_len is not None):
        raise ValueError("prefix_lens, max_prefix_len and max_own_len need group_starts")
    if weights is None and decay != 1.0:
        raise ValueError("decay needs weights")
    form = given[0]
    if fn_name not in _EXTRA_FORMS[form]:
        raise ValueError(f"{fn_name} takes no {form}")
    name = _EXTRA_FORMS[form][fn_name]
    B, NB, Hkv = shape[0], cache_shape[0], cache_shape[1]
    if form == "blocks":
        _check_cuda("blocks", blocks, _I32)
        if blocks.dim() != 3 or blocks.shape[:2] != (B, Hkv):
            raise ValueError("blocks must be [B, num_kv_heads, count]")
        return name, (blocks.data_ptr(),), (blocks.shape[2],), (), {"blocks": blocks}
    if form == "prefix":
        _check_cuda("group_starts", group_starts, _I32)
        _check_cuda("prefix_lens", prefix_lens, _I32)
        if group_starts.dim() != 1 or prefix_lens.shape != (group_starts.shape[0] - 1,):
            raise ValueError("group_starts must be [num_groups + 1] and prefix_lens [num_groups]")
        bounds = [max_context_len if v is None else v for v in (max_prefix_len, max_own_len)]
        return (name, (group_starts.data_ptr(), prefix_lens.data_ptr()), (prefix_lens.shape[0], *map(_c_int, bounds)), (),
                {"group_starts": group_starts, "prefix_lens": prefix_lens})
    _check_cuda("weights", weights, _F32)
    if weights.shape != (NB, Hkv, 16):
        raise ValueError("weights must be [num_blocks, num_kv_heads, 16]")
    return name, (weights.data_ptr(),), (), (float(decay),), {"weights": weights}


def _call(fn_name, q, k_cache, v_cache, block_table, context_lens, scale, *, k_scale=None,
          v_scale=None, max_context_len=None, out=None, stream=None, tree_mask=None, window=None, sinks=0, blocks=None,
          group_starts=None, prefix_lens=None, max_prefix_len=None, max_own_len=None, weights=None, decay=1.0):
    lib = load_library()
    _check_cuda("q", q, _BF16)
    cache_shape = k_cache.shape
    if q.dim() != 4 or len(cache_shape) != 4 or cache_shape != v_cache.shape or block_table.dim() != 2:
        raise ValueError("expected q [B, q_len, Hq, d], caches [NB, Hkv, bs, d], block_table [B, M]")
    B, q_len, Hq, d = q.shape
    kv = _kv_dtype(k_cache, v_cache, d, k_scale, v_scale)
    _check_cuda("block_table", block_table, _I32)
    _check_cuda("context_lens", context_lens, _I32)
    if kv == PA_KV_BF16:
        k_scale = v_scale = None
    NB, Hkv, bs, d2 = cache_shape
    rows, max_blocks = block_table.shape
    if (d2 != d and kv != PA_KV_FP4_E2M1) or rows != B or context_lens.shape != (B,):
        raise ValueError("shape mismatch between q, caches, block_table and context_lens")
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q.shape, q, stream)  # (a third of the time of empty)
    else:
        _check_cuda("out", out, _BF16)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if B == 0:  # (an empty tensor has no address)
        return out
    if max_context_len is None:
        max_context_len = max_blocks * bs  # an upper bound known without reading the device
    span = ()
    if window is not None or sinks:
        fn_name, span = _window(fn_name, window, sinks)
    counts, floats, more = (), (), {}
    mask = ()
    if not (blocks is group_starts is weights is prefix_lens is max_prefix_len is max_own_len is None) or decay != 1.0:
        fn_name, mask, counts, floats, more = _extra(fn_name, q.shape, cache_shape, max_context_len, blocks, group_starts,
                                                     prefix_lens, max_prefix_len, max_own_len, weights, decay, window)
        index = q.get_device()
        for t in more.values():
            if t.get_device() != index:
                _one_device(None, q=q, **more)  # (names them; the others are checked below)
    if fn_name == "paged_attn_tree_verify":
        _check_cuda("tree_mask", tree_mask, _I32)
        if tree_mask.shape != (B, q_len):
            raise ValueError("tree_mask must be [B, q_len]")
        mask = (tree_mask.data_ptr(),)
    with _one_device(stream, q, k_cache, v_cache, block_table, context_lens, tree_mask, out, k_scale, v_scale,
                     names="q k_cache v_cache block_table context_lens tree_mask out k_scale v_scale"):
        st = getattr(lib, fn_name)(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(), *mask,
            B, max_blocks, NB, _c_int(max_context_len), q_len, *counts, Hq, Hkv, d, bs, *span, *floats,
            float(scale), kv, _ptr(k_scale), _ptr(v_scale), out.data_ptr(), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, fn_name)
    return out


def decode(q, k_cache, v_cache, block_table, context_lens, scale, **kw):
    """Single-token paged GQA decode; q [B, 1, Hq, d] bf16.  With window=W (and sinks=S) the token sees
    the last W tokens, itself included, and the first S.  With blocks [B, Hkv, count] int32 each kv head
    reads the listed blocks only (select_blocks).  With group_starts [n + 1] and prefix_lens [n] int32 the
    sequences of a group share their first tokens' blocks, which are read once (max_prefix_len and max_own_len: host-side
    bounds of the shared and the own tokens).  With weights [NB, Hkv, 16] fp32 the step's softmax weights join the sums
    kept there, in place: decay * sum + weight.  One of the four a call.  See paged_attn_decode,
    paged_attn_window_decode, paged_attn_sparse_decode, paged_attn_prefix_decode, paged_attn_weighted_decode."""
    return _call("paged_attn_decode", q, k_cache, v_cache, block_table, context_lens, scale, **kw)


def verify(q, k_cache, v_cache, block_table, context_lens, scale, **kw):
    """(K+1)-row causal speculative-verify attention; q [B, K+1, Hq, d] bf16.  window and sinks as in
    decode, each row's window ending at its own token; blocks, group_starts and prefix_lens as in decode.  See
    paged_attn_verify, paged_attn_window_verify, paged_attn_sparse_verify, paged_attn_prefix_verify."""
    return _call("paged_attn_verify", q, k_cache, v_cache, block_table, context_lens, scale, **kw)


def tree_verify(q, k_cache, v_cache, block_table, context_lens, tree_mask, scale, **kw):
    """Verify over a tree of drafts: tree_mask int32 [B, q_len] ancestor bitmasks over the new
    tokens (bit t of row i: row i sees new token t).  It takes no window.  See
    paged_attn_tree_verify."""
    for name in ("window", "blocks", "group_starts", "weights"):
        if kw.get(name) is not None:
            raise ValueError(f"tree_verify takes no {name}")
    return _call("paged_attn_tree_verify", q, k_cache, v_cache, block_table, context_lens, scale,
                 tree_mask=tree_mask, **kw)


def prefill(q, k_cache, v_cache, block_table, context_lens, query_start_loc, scale, *,
            max_q_len=None, max_context_len=None, out=None, stream=None, k_scale=None, v_scale=None,
            window=None, sinks=0):
    """Paged attention over packed variable-length query rows (chunked prefill, with decode or
    verify rows alongside): q [total_q, Hq, d] bf16, query_start_loc [B+1] int32 (device); caches
    bf16, E4M3 bytes (uint8 / float8_e4m3fn) with k_scale / v_scale [NB, Hkv] fp32, or 4-bit.
    max_q_len must bound every sequence's rows; by default it is read from query_start_loc
    (one device-to-host copy).  window and sinks as in verify.  See paged_attn_prefill,
    paged_attn_window_prefill."""
    lib = load_library()
    _check_cuda("q", q, _BF16)
    if q.dim() != 3 or k_cache.dim() != 4 or k_cache.shape != v_cache.shape or block_table.dim() != 2:
        raise ValueError("expected q [total_q, Hq, d], caches [NB, Hkv, bs, d], block_table [B, M]")
    total_q, Hq, d = q.shape
    kv = _kv_dtype(k_cache, v_cache, d, k_scale, v_scale)
    _check_cuda("block_table", block_table, _I32)
    _check_cuda("context_lens", context_lens, _I32)
    _check_cuda("query_start_loc", query_start_loc, _I32)
    if kv == PA_KV_BF16:
        k_scale = v_scale = None
    NB, Hkv, bs, d2 = k_cache.shape
    B = int(block_table.shape[0])
    if (d2 != d and kv != PA_KV_FP4_E2M1) or context_lens.shape != (B,) or query_start_loc.shape != (B + 1,):
        raise ValueError("shape mismatch between q, caches, block_table, context_lens, query_start_loc")
    if out is None:
        out = torch.empty_like(q) if stream is None else _new(q.shape, q, stream)  # (a third of the time of empty)
    else:
        _check_cuda("out", out, _BF16)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if B == 0 or total_q == 0:
        return out
    if max_q_len is None:
        with torch.cuda.stream(stream):  # (None: the current one) the stream that the offsets are ready on
            qsl = query_start_loc.cpu()
        max_q_len = int((qsl[1:] - qsl[:-1]).max())
    max_blocks = int(block_table.shape[1])
    if max_context_len is None:
        max_context_len = max_blocks * bs
    fn_name, span = _window("paged_attn_prefill", window, sinks)
    with _one_device(stream, q, k_cache, v_cache, block_table, context_lens, query_start_loc, out, k_scale, v_scale,
                     names="q k_cache v_cache block_table context_lens query_start_loc out k_scale v_scale"):
        st = getattr(lib, fn_name)(
            q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
            context_lens.data_ptr(), query_start_loc.data_ptr(), B, total_q, max(1, _c_int(max_q_len)),
            max_blocks, NB, _c_int(max_context_len), Hq, Hkv, d, bs, *span, float(scale), kv, _ptr(k_scale),
            _ptr(v_scale), out.data_ptr(), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, fn_name)
    return out


def append_kv(k_new, v_new, k_cache, v_cache, block_table, context_lens, *, k_scale=None,
              v_scale=None, stream=None):
    """Store the new tokens' K/V [B, n_new, Hkv, d] bf16 in the paged cache, in place (and, for an
    fp8 cache, update the per-(block, head) scales; a 4-bit cache takes optional per-head scales
    [Hkv] that it only reads).  context_lens holds the lengths after the append.  See
    paged_attn_append_kv."""
    lib = load_library()
    _check_cuda("k_new", k_new, _BF16)
    _check_cuda("v_new", v_new, _BF16)
    if k_new.dim() != 4 or k_new.shape != v_new.shape or k_cache.dim() != 4 or k_cache.shape != v_cache.shape:
        raise ValueError("expected k_new/v_new [B, n_new, Hkv, d] and caches [NB, Hkv, bs, d]")
    B, n_new, Hkv, d = k_new.shape
    kv = _kv_dtype(k_cache, v_cache, d, k_scale, v_scale)
    _check_cuda("block_table", block_table, _I32)
    _check_cuda("context_lens", context_lens, _I32)
    NB, Hkv2, bs, d2 = k_cache.shape
    if Hkv2 != Hkv or (d2 != d and kv != PA_KV_FP4_E2M1) or block_table.dim() != 2 \
            or block_table.shape[0] != B or context_lens.shape != (B,):
        raise ValueError("shape mismatch between new rows, caches, block_table and context_lens")
    if kv == PA_KV_BF16:
        k_scale = v_scale = None
    if kv == PA_KV_FP8_E4M3 and (k_scale.shape != (NB, Hkv) or v_scale.shape != (NB, Hkv)):
        raise ValueError("k_scale / v_scale must be [num_blocks, num_kv_heads]")
    if B == 0 or n_new == 0:
        return
    with _one_device(stream, k_new, v_new, k_cache, v_cache, block_table, context_lens, k_scale, v_scale,
                     names="k_new v_new k_cache v_cache block_table context_lens k_scale v_scale"):
        st = lib.paged_attn_append_kv(
            k_new.data_ptr(), v_new.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
            block_table.data_ptr(), context_lens.data_ptr(), B, n_new, int(block_table.shape[1]), NB,
            Hkv, d, bs, kv, _ptr(k_scale), _ptr(v_scale), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_append_kv")


def read_kv(k_cache, v_cache, block_table, context_lens, n, *, k_scale=None, v_scale=None, k_out=None,
            v_out=None, head_dim=None, stream=None):
    """The last n stored tokens of every sequence as bf16 (k, v), each [B, n, Hkv, d]: the inverse of
    append_kv.  Caches and scales of any type; head_dim is needed only where a byte cache's last dim
    could be read two ways (E4M3 bytes of d against 4-bit bytes of 9 d / 16: 36 and 72 are 4-bit
    caches of 64 and 128).  See paged_attn_read_kv."""
    lib = load_library()
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or k_cache.shape != v_cache.shape \
            or block_table.dim() != 2:
        raise ValueError("expected caches [NB, Hkv, bs, d] and block_table [B, M]")
    NB, Hkv, bs, last = k_cache.shape
    if head_dim is None:
        head_dim = {36: 64, 72: 128}.get(last, last) if k_cache.dtype == torch.uint8 else last
    d = int(head_dim)
    kv = _kv_dtype(k_cache, v_cache, d, k_scale, v_scale)
    _check_cuda("block_table", block_table, _I32)
    _check_cuda("context_lens", context_lens, _I32)
    B, n = int(block_table.shape[0]), int(n)
    if context_lens.shape != (B,) or (last != d and kv != PA_KV_FP4_E2M1) or n < 0:
        raise ValueError("shape mismatch between caches, block_table, context_lens, n and head_dim")
    if kv == PA_KV_BF16:
        k_scale = v_scale = None
    if kv == PA_KV_FP8_E4M3 and (k_scale.shape != (NB, Hkv) or v_scale.shape != (NB, Hkv)):
        raise ValueError("k_scale / v_scale must be [num_blocks, num_kv_heads]")
    outs = []
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is None:
            t = _new((B, n, Hkv, d), k_cache, stream)
        else:
            _check_cuda(name, t, _BF16)
            if t.shape != (B, n, Hkv, d):
                raise ValueError(f"{name} must be [B, n, Hkv, d]")
        outs.append(t)
    if n == 0 or B == 0:
        return tuple(outs)
    with _one_device(stream, k_cache, v_cache, block_table, context_lens, k_scale, v_scale, *outs,
                     names="k_cache v_cache block_table context_lens k_scale v_scale k_out v_out"):
        st = lib.paged_attn_read_kv(
            k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(), B, n,
            int(block_table.shape[1]), NB, Hkv, d, bs, kv, _ptr(k_scale), _ptr(v_scale), outs[0].data_ptr(),
            outs[1].data_ptr(), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_read_kv")
    return tuple(outs)


def block_bounds(k_cache, block_table, context_lens, n, bounds, bound_scale, *, k_scale=None, stream=None):
    """Bounds of the keys of every block that holds one of a sequence's last n tokens, in place: bounds [NB, Hkv, 2, d]
    int8 and bound_scale [NB, Hkv] fp32, what select_blocks reads.  Called after append_kv with the same n, or
    once for a prompt with its length.  k_cache and k_scale of any cache type.  See paged_attn_block_bounds."""
    lib = load_library()
    _check_cuda("bounds", bounds, _I8)
    _check_cuda("bound_scale", bound_scale, _F32)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or bounds.dim() != 4 or block_table.dim() != 2:
        raise ValueError("expected k_cache [NB, Hkv, bs, d], bounds [NB, Hkv, 2, d] and block_table [B, M]")
    NB, Hkv, bs, last = k_cache.shape
    d = bounds.shape[3]
    if k_cache.dtype is torch.bfloat16:
        _check_cuda("k_cache", k_cache, _BF16)
        kv = PA_KV_BF16
    else:  # (the value cache's checks are the key cache's: there is none here)
        kv = _kv_dtype(k_cache, k_cache, d, k_scale, k_scale)
    _check_cuda("block_table", block_table, _I32)
    _check_cuda("context_lens", context_lens, _I32)
    B, M = block_table.shape
    n = int(n)
    if (last != d and kv != PA_KV_FP4_E2M1) or bounds.shape != (NB, Hkv, 2, d) or bound_scale.shape != (NB, Hkv) \
            or context_lens.shape != (B,) or n < 0:
        raise ValueError("shape mismatch between k_cache, bounds, bound_scale, block_table, context_lens and n")
    if kv == PA_KV_BF16:
        k_scale = None
    if B == 0 or n == 0:
        return
    with _one_device(stream, k_cache=k_cache, block_table=block_table, context_lens=context_lens, k_scale=k_scale,
                     bounds=bounds, bound_scale=bound_scale):
        st = lib.paged_attn_block_bounds(
            k_cache.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(), B, _c_int(n), M, NB, Hkv, d,
            bs, kv, _ptr(k_scale), bounds.data_ptr(), bound_scale.data_ptr(), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_block_bounds")


def select_blocks(q, bounds, bound_scale, block_table, context_lens, count, *, sink_blocks=1, recent_blocks=2,
                  max_context_len=None, out=None, stream=None):
    """The `count` blocks of each sequence and kv head that the rows q [B, q_len, Hq, d] bf16 score highest by the
    bounds of block_bounds, the first sink_blocks and last recent_blocks always among them: int32 [B, Hkv, count], columns
    of the block table, ascending, -1 where there are fewer.  For decode(blocks=) and verify(blocks=).  See
    paged_attn_select_blocks."""
    lib = load_library()
    _check_cuda("q", q, _BF16)
    _check_cuda("bounds", bounds, _I8)
    _check_cuda("bound_scale", bound_scale, _F32)
    _check_cuda("block_table", block_table, _I32)
    _check_cuda("context_lens", context_lens, _I32)
    if q.dim() != 4 or bounds.dim() != 4 or block_table.dim() != 2:
        raise ValueError("expected q [B, q_len, Hq, d], bounds [NB, Hkv, 2, d] and block_table [B, M]")
    B, q_len, Hq, d = q.shape
    NB, Hkv, ends, d2 = bounds.shape
    rows, M = block_table.shape
    count = int(count)
    if ends != 2 or d2 != d or bound_scale.shape != (NB, Hkv) or rows != B or context_lens.shape != (B,):
        raise ValueError("shape mismatch between q, bounds, bound_scale, block_table and context_lens")
    if count < 1:
        raise ValueError("count must be at least 1")
    if out is None:
        out = _new((B, Hkv, count), q, stream, torch.int32)
    else:
        _check_cuda("out", out, _I32)
        if out.shape != (B, Hkv, count):
            raise ValueError("out must be [B, num_kv_heads, count]")
    if B == 0:
        return out
    if max_context_len is None:
        max_context_len = M * 16
    with _one_device(stream, q=q, bounds=bounds, bound_scale=bound_scale, block_table=block_table,
                     context_lens=context_lens, out=out):
        st = lib.paged_attn_select_blocks(
            q.data_ptr(), bounds.data_ptr(), bound_scale.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(), B,
            M, NB, _c_int(max_context_len), q_len, Hq, Hkv, d, 16, _c_int(count), _c_int(sink_blocks),
            _c_int(recent_blocks), out.data_ptr(), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_select_blocks")
    return out


def evict(k_cache, v_cache, weights, block_table, context_lens, new_table, keep, *, sinks=0, recent=0, k_scale=None,
          v_scale=None, max_context_len=None, head_dim=None, new_lens=None, stream=None):
    """Keep of every sequence and kv head the first `sinks` tokens, the last `recent` and, up to `keep` in all, those of
    the largest sums in weights [NB, Hkv, 16] fp32 (decode(weights=)); they move in order, with their sums, to the
    blocks of new_table [B, M2] int32, which must hold no token of the batch.  Returns the new lengths [B] int32
    (new_lens, which may not be context_lens); the old blocks stay as they are for the caller to give back.  head_dim as in read_kv.  See paged_attn_evict."""
    lib = load_library()
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or k_cache.shape != v_cache.shape \
            or block_table.dim() != 2 or new_table.dim() != 2:
        raise ValueError("expected caches [NB, Hkv, bs, d], block_table [B, M] and new_table [B, M2]")
    NB, Hkv, bs, last = k_cache.shape
    if head_dim is None:
        head_dim = {36: 64, 72: 128}.get(last, last) if k_cache.dtype == torch.uint8 else last
    d = int(head_dim)
    kv = _kv_dtype(k_cache, v_cache, d, k_scale, v_scale)
    _check_cuda("weights", weights, _F32)
    _check_cuda("block_table", block_table, _I32)
    _check_cuda("context_lens", context_lens, _I32)
    _check_cuda("new_table", new_table, _I32)
    B = block_table.shape[0]
    if context_lens.shape != (B,) or new_table.shape[0] != B or weights.shape != (NB, Hkv, 16) \
            or (last != d and kv != PA_KV_FP4_E2M1):
        raise ValueError("shape mismatch between caches, weights, block_table, context_lens, new_table and head_dim")
    if kv == PA_KV_FP8_E4M3 and (k_scale.shape != (NB, Hkv) or v_scale.shape != (NB, Hkv)):
        raise ValueError("k_scale / v_scale must be [num_blocks, num_kv_heads]")
    if kv == PA_KV_BF16:
        k_scale = v_scale = None
    if new_lens is None:
        new_lens = _new((B,), k_cache, stream, torch.int32)
    else:
        _check_cuda("new_lens", new_lens, _I32)
        if new_lens.shape != (B,):
            raise ValueError("new_lens must be [B]")
    if B == 0:
        return new_lens
    if max_context_len is None:
        max_context_len = block_table.shape[1] * bs
    with _one_device(stream, k_cache=k_cache, v_cache=v_cache, weights=weights, block_table=block_table,
                     context_lens=context_lens, new_table=new_table, new_lens=new_lens, k_scale=k_scale, v_scale=v_scale):
        st = lib.paged_attn_evict(
            k_cache.data_ptr(), v_cache.data_ptr(), weights.data_ptr(), block_table.data_ptr(), context_lens.data_ptr(),
            new_table.data_ptr(), B, block_table.shape[1], new_table.shape[1], NB, _c_int(max_context_len), Hkv, d, bs, kv,
            _ptr(k_scale), _ptr(v_scale), _c_int(keep), _c_int(sinks), _c_int(recent), new_lens.data_ptr(),
            _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_evict")
    return new_lens


def _token_stride(name, t, heads_dims):
    """Elements from one token of a bf16 [T, heads, d] tensor to the next (a slice of a packed
    projection is strided), after its checks."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    shape = tuple(t.shape)
    if shape != heads_dims:
        raise ValueError(f"{name} must be {list(heads_dims)}, got {list(shape)}")
    step, head, one = t.stride()
    if shape[0] < 2:  # a single token's stride says nothing
        step = shape[1] * shape[2]
    if shape[0] and (one != 1 or (head != shape[2] and shape[1] > 1)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return step


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, *, eps=1e-6, interleaved=False, q_out=None,
                 k_out=None, stream=None):
    """RMS norm of every head row of q [T, Hq, d] and k [T, Hkv, d] bf16 and the rotation of its first
    cos_sin.shape[1] dims by the token's position, in one pass; returns (q_out, k_out).  q and k may be
    slices of one packed projection (tokens strided); q_out / k_out may be q / k themselves.  Weights
    [d] bf16, cos_sin [max_position, rotary_dim] fp32 (cosines, then sines), positions [T] int32.  See
    paged_attn_qk_norm_rope."""
    lib = load_library()
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("expected q [T, Hq, d] and k [T, Hkv, d]")
    T, Hq, d = q_shape = tuple(q.shape)
    Hkv = k.shape[1]
    k_shape = (T, Hkv, d)
    strides = [_token_stride("q", q, q_shape), _token_stride("k", k, k_shape)]
    _check_cuda("q_weight", q_weight, _BF16)
    _check_cuda("k_weight", k_weight, _BF16)
    _check_cuda("cos_sin", cos_sin, _F32)
    _check_cuda("positions", positions, _I32)
    if q_weight.shape != (d,) or k_weight.shape != (d,) or cos_sin.dim() != 2 or positions.shape != (T,):
        raise ValueError("expected weights [d], cos_sin [max_position, rotary_dim], positions [T]")
    if q_out is None:
        q_out = _new(q_shape, q, stream)
        strides.append(Hq * d)
    else:
        strides.append(_token_stride("q_out", q_out, q_shape))
    if k_out is None:
        k_out = _new(k_shape, k, stream)
        strides.append(Hkv * d)
    else:
        strides.append(_token_stride("k_out", k_out, k_shape))
    if T == 0:
        return q_out, k_out
    max_position, rotary = cos_sin.shape
    with _one_device(stream, q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out,
                     names="q k q_weight k_weight cos_sin positions q_out k_out"):
        st = lib.paged_attn_qk_norm_rope(
            q.data_ptr(), k.data_ptr(), q_weight.data_ptr(), k_weight.data_ptr(), cos_sin.data_ptr(),
            positions.data_ptr(), T, Hq, Hkv, d, rotary, 1 if interleaved else 0, max_position, eps, *strides,
            q_out.data_ptr(), k_out.data_ptr(), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_qk_norm_rope")
    return q_out, k_out


def spec_accept(p, q, draft_tokens, u_accept, u_sample, *, out_tokens=None, num_accepted=None,
                stream=None):
    """Speculative acceptance for a batch of rounds: p [B, K+1, V] and q [B, K, V] fp32
    probabilities, draft_tokens [B, K] int32, u_accept [B, K] fp32 uniforms, u_sample [B] int32
    (uint32 bit patterns).  Returns (num_accepted [B] int32, out_tokens [B, K+1] int32).  See
    paged_attn_spec_accept."""
    lib = load_library()
    _check_cuda("p", p, _F32)
    _check_cuda("u_sample", u_sample, _I32)
    if p.dim() != 3:
        raise ValueError("p must be [B, K+1, V]")
    B, K1, V = p.shape
    K = K1 - 1
    if K > 0:
        _check_cuda("q", q, _F32)
        _check_cuda("draft_tokens", draft_tokens, _I32)
        _check_cuda("u_accept", u_accept, _F32)
        if q.shape != (B, K, V) or draft_tokens.shape != (B, K) or u_accept.shape != (B, K):
            raise ValueError("q [B, K, V], draft_tokens [B, K] and u_accept [B, K] must match p")
    if u_sample.shape != (B,):
        raise ValueError("u_sample must be [B]")
    if out_tokens is None:
        out_tokens = _new((B, K + 1), p, stream, torch.int32)
    if num_accepted is None:
        num_accepted = _new((B,), p, stream, torch.int32)
    _check_cuda("out_tokens", out_tokens, _I32)
    _check_cuda("num_accepted", num_accepted, _I32)
    if out_tokens.shape != (B, K + 1) or num_accepted.shape != (B,):
        raise ValueError("out_tokens must be [B, K+1] and num_accepted [B]")
    if B == 0:
        return num_accepted, out_tokens
    ptr = (lambda t: t.data_ptr() if K > 0 else None)
    with _one_device(stream, p=p, u_sample=u_sample, out_tokens=out_tokens, num_accepted=num_accepted,
                     q=q if K > 0 else None, draft_tokens=draft_tokens if K > 0 else None,
                     u_accept=u_accept if K > 0 else None):
        st = lib.paged_attn_spec_accept(p.data_ptr(), ptr(q), ptr(draft_tokens), ptr(u_accept),
                                        u_sample.data_ptr(), B, K, V, out_tokens.data_ptr(),
                                        num_accepted.data_ptr(), _stream_handle(stream))
    if st != PA_OK:
        raise PagedAttnError(st, "paged_attn_spec_accept")
    return num_accepted, out_tokens


def run_problem(p, out=None, stream=None, max_context_len=None):
    """Run decode (q_len 1) or verify on a workloads.PagedAttnProblem whose tensors are on the GPU."""
    fn = decode if p.q_len == 1 else verify
    return fn(p.q, p.k_cache, p.v_cache, p.block_table, p.context_lens, p.scale,
              k_scale=p.k_scale, v_scale=p.v_scale, out=out, stream=stream,
              max_context_len=max_context_len)
