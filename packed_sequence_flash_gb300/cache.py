"""8-bit paged key/value cache: append, attention, eviction, gather.

Python binding of the ``psf_kv_cache_*`` and ``psf_attn_cache_*`` calls of
libpsf.so: argument marshalling only, as in ``attention.py`` (outputs and
workspaces from torch, the current stream, ``PSFError`` on a nonzero code).

A serving loop::

    cache = kv_cache(num_pages, Hkv, D, D, weights=True)
    kv_cache_append(cache, k, v, page_table, seq_lens, cu_new)        # prompts: seq_lens counts the new tokens
    while ...:
        seq_lens += 1
        kv_cache_append(cache, k1, v1, page_table, seq_lens)          # one new token per sequence
        out, lse = attn_cache_fwd(q1, cache, page_table, seq_lens, scale, accumulate=True)
    seq_lens = kv_cache_evict(cache, page_table, seq_lens, budget, recent)

Nothing here synchronises; every call can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import PSF_CACHE_ACCUMULATE, check
from .attention import _cap, _DTYPES, _dtype_code, _i32, _need, _need_view, _ptr, _window, _workspace


class KVCache:
    """The tensors of a cache.

    k [num_pages, Hkv, page_size, Dqk], v [num_pages, Hkv, page_size, Dv]
    (float8_e4m3fn, any strides with a contiguous last dim), k_scale and v_scale
    [num_pages, Hkv] fp32: a code c stands for c * scale. weight [num_pages, Hkv,
    page_size] fp32 or None: the attention weight each token has received, kept
    by ``attn_cache_fwd(accumulate=True)`` and used by ``kv_cache_evict``.
    """

    __slots__ = ("k", "v", "k_scale", "v_scale", "weight", "num_pages", "Hkv", "page_size", "Dqk", "Dv", "device",
                 "_struct", "_ref")

    def __init__(self, k, v, k_scale, v_scale, weight=None):
        _need_view(k, "cache k", torch.float8_e4m3fn)
        _need_view(v, "cache v", torch.float8_e4m3fn)
        if k.dim() != 4 or v.dim() != 4 or k.shape[:3] != v.shape[:3]:
            raise ValueError("cache k and v must be [num_pages, Hkv, page_size, D] with equal leading dims")
        num_pages, Hkv, page_size, Dqk = k.shape
        Dv = v.shape[3]
        device = k.device
        _cache_f32(k_scale, "k_scale", (num_pages, Hkv), device)
        _cache_f32(v_scale, "v_scale", (num_pages, Hkv), device)
        if weight is not None:
            _cache_f32(weight, "weight", (num_pages, Hkv, page_size), device)
        if v.device != device:
            raise ValueError("the cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale, self.weight = k, v, k_scale, v_scale, weight
        self.num_pages, self.Hkv, self.page_size, self.Dqk, self.Dv = num_pages, Hkv, page_size, Dqk, Dv
        self.device = device
        c = _lib.KVCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _ptr(weight),
                               num_pages, page_size, Hkv, Dqk, Dv)
        if not (k.is_contiguous() and v.is_contiguous()):
            c.k_strides[:] = k.stride()[:3]
            c.v_strides[:] = v.stride()[:3]
        self._struct = c
        self._ref = ctypes.byref(c)


def _cache_f32(t, name, shape, device):
    _need(t, name, torch.float32)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != device:
        raise ValueError("the cache's tensors must be on one device")


def kv_cache(num_pages, Hkv, Dqk, Dv, page_size=64, weights=False, device="cuda") -> KVCache:
    """A cache of num_pages pages (zeroed): page_size 16, 32, 64 or 128 tokens."""
    k = torch.zeros(num_pages, Hkv, page_size, Dqk, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    v = torch.zeros(num_pages, Hkv, page_size, Dv, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    ks = torch.zeros(num_pages, Hkv, dtype=torch.float32, device=device)
    w = torch.zeros(num_pages, Hkv, page_size, dtype=torch.float32, device=device) if weights else None
    return KVCache(k, v, ks, torch.zeros_like(ks), w)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _launch(device, call, *args) -> None:
    """call(*args, stream) with `device` current (a call's tensors may be on another than the current one)."""
    index = device.index
    before = torch.cuda.current_device()
    if before == index:
        rc = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = call(*args, _raw_stream(index))
    if rc:
        check(rc)


def _sequences(cache, page_table, seq_lens, *others):
    """(B, max_pages) of a call's sequences; `others`: further tensors that must be on the cache's device."""
    _i32(page_table, "page_table")
    _i32(seq_lens, "seq_lens")
    shape = page_table.shape
    if len(shape) != 2 or seq_lens.shape != shape[:1]:
        raise ValueError("page_table must be [B, max_pages] and seq_lens [B]")
    device = cache.device
    if page_table.device != device or seq_lens.device != device:
        raise ValueError("every tensor of a call must be on the cache's device")
    for t in others:
        if t is not None and t.device != device:
            raise ValueError("every tensor of a call must be on the cache's device")
    return shape


def _cu(cu, name, B):
    if cu is not None:
        _i32(cu, name)
        if cu.dim() != 1 or cu.shape[0] != B + 1:
            raise ValueError(f"{name} must be [B + 1]")
    return cu


def _thd_strides(a, b):
    """Element strides (batch, head, row) of two [T, H, D] tensors, or NULL when both are contiguous."""
    if a.is_contiguous() and b.is_contiguous():
        return None
    return (ctypes.c_int64 * 6)(0, a.stride(1), a.stride(0), 0, b.stride(1), b.stride(0))


def _rows3(t, name, H, D):
    if t.dim() != 3 or t.shape[1] != H or t.shape[2] != D:
        raise ValueError(f"{name} must be [T, {H}, {D}], got {list(t.shape)}")


def kv_cache_append(cache, k, v, page_table, seq_lens, cu_new=None) -> None:
    """Quantise new rows k [T, Hkv, Dqk], v [T, Hkv, Dv] (bf16 or fp16) into the cache, in place.

    Sequence b's new tokens are rows [cu_new[b], cu_new[b + 1]) (T / B each without cu_new) and go to its last
    positions: seq_lens (int32 [B], on the device) counts them already. See psf_kv_cache_append for the scales.
    """
    dt = _dtype_code([(k, "k"), (v, "v")], strided=True)
    _rows3(k, "k", cache.Hkv, cache.Dqk)
    _rows3(v, "v", cache.Hkv, cache.Dv)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have the same number of rows")
    B, max_pages = _sequences(cache, page_table, seq_lens, k, v, cu_new)
    _cu(cu_new, "cu_new", B)
    _launch(cache.device, _lib.load().psf_kv_cache_append, cache._ref, k.data_ptr(), v.data_ptr(), _thd_strides(k, v),
            dt, _ptr(cu_new), page_table.data_ptr(), seq_lens.data_ptr(), B, max_pages, k.shape[0])


@functools.lru_cache(maxsize=256)
def _attn_workspace(*sizes) -> int:
    return int(_lib.load().psf_attn_cache_workspace_size(*sizes))


def attn_cache_workspace_size(cache, B, max_pages, Hq, max_q=1, accumulate=False) -> int:
    return _attn_workspace(int(B), int(max_pages), cache.page_size, int(Hq), cache.Hkv, cache.Dqk, cache.Dv, int(max_q),
                           PSF_CACHE_ACCUMULATE if accumulate else 0)


def attn_cache_fwd(q, cache, page_table, seq_lens, scale, cu_q=None, max_q=None, causal=True, window=None,
                   softcap=None, accumulate=False, out=None, lse=None, workspace=None):
    """Attention of packed query rows over the cache -> (out [T, Hq, Dv] in q's type, lse [Hq, T] fp32).

    q [T, Hq, Dqk] bf16 or fp16: sequence b's rows are [cu_q[b], cu_q[b + 1]) with at most max_q of them, or T / B each
    without cu_q. They are the last tokens of the sequence (their keys are in the cache already), so one row per
    sequence is a decode step. window, softcap, GQA, lse as for ``attn_varlen_fwd``; causal is the default.
    accumulate: add every token's attention weight, over the rows and the heads of its KV head, to cache.weight.
    Long prompt chunks run faster through ``kv_cache_gather`` and ``attn_varlen_fwd``.
    """
    if q.dtype not in _DTYPES:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    _need_view(q, "q")
    if q.dim() != 3 or q.shape[2] != cache.Dqk:
        raise ValueError(f"q must be [T, Hq, {cache.Dqk}], got {list(q.shape)}")
    T, Hq, _ = q.shape
    B, max_pages = _sequences(cache, page_table, seq_lens, q, cu_q, out, lse, workspace)
    _cu(cu_q, "cu_q", B)
    if max_q is None:
        if cu_q is not None:
            raise ValueError("cu_q needs max_q, the most query rows of a sequence")
        max_q = T // B if B else 0
    if out is None:
        out = torch.empty((T, Hq, cache.Dv), dtype=q.dtype, device=q.device)
    else:
        _need_view(out, "out", q.dtype)
        _rows3(out, "out", Hq, cache.Dv)
        if out.shape[0] != T:
            raise ValueError("out must have q's rows")
    if lse is None:
        lse = torch.empty(Hq, T, dtype=torch.float32, device=q.device)
    else:
        _need(lse, "lse", torch.float32)
        if tuple(lse.shape) != (Hq, T):
            raise ValueError(f"lse must be [{Hq}, {T}], got {list(lse.shape)}")
    if workspace is None:
        workspace = _workspace(attn_cache_workspace_size(cache, B, max_pages, Hq, max_q, accumulate), q.device)
    _launch(cache.device, _lib.load().psf_attn_cache_fwd, q.data_ptr(), cache._ref, out.data_ptr(), lse.data_ptr(),
            _ptr(cu_q), page_table.data_ptr(), seq_lens.data_ptr(), B, max_pages, T, int(max_q), Hq,
            _thd_strides(q, out), _DTYPES[q.dtype], float(scale), int(bool(causal)), _window(window), _cap(softcap),
            PSF_CACHE_ACCUMULATE if accumulate else 0, workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return out, lse


@functools.lru_cache(maxsize=256)
def _evict_workspace(*sizes) -> int:
    return int(_lib.load().psf_kv_cache_evict_workspace_size(*sizes))


def kv_cache_evict_workspace_size(cache, B, max_pages, budget) -> int:
    return _evict_workspace(int(B), int(max_pages), cache.page_size, cache.Hkv, int(budget))


def kv_cache_evict(cache, page_table, seq_lens, budget, recent, new_lens=None, workspace=None):
    """Cut every sequence longer than budget down to it, in place -> new lengths (int32 [B]).

    For each KV head on its own: the last `recent` tokens stay, and of the others the budget - recent with the largest
    accumulated weight (of equal ones the earliest), in their order. Pages past ceil(budget / page_size) are free
    afterwards. See psf_kv_cache_evict for the scales.
    """
    B, max_pages = _sequences(cache, page_table, seq_lens, new_lens, workspace)
    if new_lens is None:
        new_lens = torch.empty(B, dtype=torch.int32, device=seq_lens.device)
    else:
        _i32(new_lens, "new_lens")
        if tuple(new_lens.shape) != (B,):
            raise ValueError("new_lens must be [B]")
    if workspace is None:
        workspace = _workspace(kv_cache_evict_workspace_size(cache, B, max_pages, budget), seq_lens.device)
    _launch(cache.device, _lib.load().psf_kv_cache_evict, cache._ref, page_table.data_ptr(), seq_lens.data_ptr(),
            new_lens.data_ptr(), B, max_pages, int(budget), int(recent), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return new_lens


def kv_cache_gather(cache, page_table, seq_lens, total_k, dtype=torch.bfloat16):
    """The cached rows of all sequences, packed -> (k [total_k, Hkv, Dqk], v [total_k, Hkv, Dv], cu_k int32 [B + 1]).

    total_k: at least the sum of the lengths (rows past it are not written). With cu_q these are the arguments of
    ``attn_varlen_fwd`` for a prompt chunk over its cached prefix (max_k=-1: no bound to check).
    """
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bfloat16 or float16, got {dtype}")
    B, max_pages = _sequences(cache, page_table, seq_lens)
    dev = seq_lens.device
    k = torch.empty(int(total_k), cache.Hkv, cache.Dqk, dtype=dtype, device=dev)
    v = torch.empty(int(total_k), cache.Hkv, cache.Dv, dtype=dtype, device=dev)
    cu_k = torch.empty(B + 1, dtype=torch.int32, device=dev)
    _launch(cache.device, _lib.load().psf_kv_cache_gather, cache._ref, page_table.data_ptr(), seq_lens.data_ptr(), B,
            max_pages, k.data_ptr(), v.data_ptr(), cu_k.data_ptr(), int(total_k), _DTYPES[dtype])
    return k, v, cu_k
