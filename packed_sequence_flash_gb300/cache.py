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
import operator

import torch

from . import _lib
from ._lib import PSF_CACHE_ACCUMULATE, check
from .attention import _cap, _DTYPES, _ptr, _window

_E4M3 = torch.float8_e4m3fn
# The call behind torch.cuda.current_stream(index).cuda_stream, without the Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


@functools.lru_cache(maxsize=None)
def _call(name):
    return getattr(_lib.load(), name)


def _tensor(t, name, dtype, device):
    """A contiguous tensor of a call, on the cache's device (an index)."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        _wrong_device(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _view(t, name, dtype, device):
    """A strided tensor whose last dim is contiguous and whose data starts on a 16-byte boundary; its address."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        _wrong_device(t, name)
    if not t.is_contiguous() and t.size(-1) > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last (head) dim must be contiguous")
    ptr = t.data_ptr()
    if ptr % 16:
        raise ValueError(f"{name}: data must start on a 16-byte boundary")
    return ptr


def _wrong_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must be on the cache's device, like every tensor of a call")


def _dtype16(t, name):
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return t.dtype


def _c_int(x, name) -> int:
    """A number of a call; the library's are 32 bits, and ctypes would cut it to them."""
    x = int(x)
    if not -0x80000000 <= x <= 0x7fffffff:
        raise ValueError(f"{name} must fit in 32 bits, got {x}")
    return x


def _launch(device, call, *args) -> None:
    """call(*args, stream) with `device` current (a call's tensors may be on another than the current one)."""
    if _current_device() == device:
        rc = call(*args, _raw_stream(device))
    else:
        with torch.cuda.device(device):
            rc = call(*args, _raw_stream(device))
    if rc:
        check(rc)


class KVCache:
    """The tensors of a cache.

    k [num_pages, Hkv, page_size, Dqk], v [num_pages, Hkv, page_size, Dv]
    (float8_e4m3fn, any strides with a contiguous last dim), k_scale and v_scale
    [num_pages, Hkv] fp32: a code c stands for c * scale. weight [num_pages, Hkv,
    page_size] fp32 or None: the attention weight each token has received, kept
    by ``attn_cache_fwd(accumulate=True)`` and used by ``kv_cache_evict``.

    Each of the five may be replaced (``cache.weight = w``) by a tensor that the
    constructor would have taken beside the others; the sizes are read-only. A
    captured graph keeps the memory that it was captured with.
    """

    __slots__ = ("_k", "_v", "_k_scale", "_v_scale", "_weight", "_num_pages", "_Hkv", "_page_size", "_Dqk", "_Dv",
                 "_device", "_struct", "_ref", "_addresses", "_held")

    def __init__(self, k, v, k_scale, v_scale, weight=None):
        self._take(k, v, k_scale, v_scale, weight)

    def _take(self, k, v, k_scale, v_scale, weight):
        """Checks the five tensors and makes them, and the struct that the calls get, the cache's."""
        device = k.get_device()
        if device < 0:
            _wrong_device(k, "cache k")
        kp, vp = _view(k, "cache k", _E4M3, device), _view(v, "cache v", _E4M3, device)
        _tensor(k_scale, "k_scale", torch.float32, device)
        _tensor(v_scale, "v_scale", torch.float32, device)
        if k.dim() != 4 or v.dim() != 4:
            raise ValueError("cache k and v must be [num_pages, Hkv, page_size, D]")
        num_pages, Hkv, page_size, Dqk = k.shape
        Dv = v.size(3)
        if v.shape != (num_pages, Hkv, page_size, Dv):
            raise ValueError("cache k and v must have equal leading dims [num_pages, Hkv, page_size]")
        if k_scale.shape != (num_pages, Hkv) or v_scale.shape != (num_pages, Hkv):
            raise ValueError(f"k_scale and v_scale must be {[num_pages, Hkv]}")
        wp = None
        if weight is not None:
            _tensor(weight, "weight", torch.float32, device)
            if weight.shape != (num_pages, Hkv, page_size):
                raise ValueError(f"weight must be {[num_pages, Hkv, page_size]}, got {list(weight.shape)}")
            wp = weight.data_ptr()
        ksp, vsp = k_scale.data_ptr(), v_scale.data_ptr()
        c = _lib.KVCacheStruct(kp, vp, ksp, vsp, wp, num_pages, page_size, Hkv, Dqk, Dv)
        if not (k.is_contiguous() and v.is_contiguous()):
            # (All strides 0 mean contiguous ones to the library.)
            for t, name in ((k, "cache k"), (v, "cache v")):
                if any(n > 1 and step == 0 for n, step in zip(t.shape[:3], t.stride())):
                    raise ValueError(f"{name}: an expanded tensor overlaps itself")
            c.k_strides[:] = k.stride()[:3]
            c.v_strides[:] = v.stride()[:3]
        self._k, self._v, self._k_scale, self._v_scale, self._weight = k, v, k_scale, v_scale, weight
        self._num_pages, self._Hkv, self._page_size, self._Dqk, self._Dv = num_pages, Hkv, page_size, Dqk, Dv
        self._device = device
        self._struct, self._ref = c, ctypes.byref(c)
        self._addresses = (kp, vp, ksp, vsp, wp)
        # While these storages live, other memory cannot come to have their addresses.
        self._held = (k.untyped_storage(), v.untyped_storage(), k_scale.untyped_storage(), v_scale.untyped_storage(),
                      None if weight is None else weight.untyped_storage())

    def _call_ref(self):
        """The struct for a call. Tensors whose memory was exchanged (t.data = u, t.set_(u)) are checked and taken anew."""
        w = self._weight
        if self._addresses != (self._k.data_ptr(), self._v.data_ptr(), self._k_scale.data_ptr(),
                               self._v_scale.data_ptr(), None if w is None else w.data_ptr()):
            self._take(self._k, self._v, self._k_scale, self._v_scale, w)
        return self._ref


def _replaceable(name):
    slot = "_" + name
    tensors = ("k", "v", "k_scale", "v_scale", "weight")

    def replace(cache, t):
        cache._take(*(t if n == name else getattr(cache, "_" + n) for n in tensors))

    return property(operator.attrgetter(slot), replace)


for _name in ("k", "v", "k_scale", "v_scale", "weight"):
    setattr(KVCache, _name, _replaceable(_name))
for _name in ("num_pages", "Hkv", "page_size", "Dqk", "Dv", "device"):
    setattr(KVCache, _name, property(operator.attrgetter("_" + _name)))


def kv_cache(num_pages, Hkv, Dqk, Dv, page_size=64, weights=False, device="cuda") -> KVCache:
    """A cache of num_pages pages (zeroed): page_size 16, 32, 64 or 128 tokens."""
    k = torch.zeros(num_pages, Hkv, page_size, Dqk, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    v = torch.zeros(num_pages, Hkv, page_size, Dv, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
    ks = torch.zeros(num_pages, Hkv, dtype=torch.float32, device=device)
    w = torch.zeros(num_pages, Hkv, page_size, dtype=torch.float32, device=device) if weights else None
    return KVCache(k, v, ks, torch.zeros_like(ks), w)


def _sequences(cache, page_table, seq_lens, cu=None, name=""):
    """(B, max_pages) of a call's sequences."""
    device = cache._device
    _tensor(page_table, "page_table", torch.int32, device)
    _tensor(seq_lens, "seq_lens", torch.int32, device)
    shape = page_table.shape
    if len(shape) != 2 or seq_lens.shape != shape[:1]:
        raise ValueError("page_table must be [B, max_pages] and seq_lens [B]")
    if shape[0] > 0x7fffffff or shape[1] > 0x7fffffff:
        raise ValueError(f"page_table must be below 2^31 both ways, got {list(shape)}")
    if cu is not None:
        _tensor(cu, name, torch.int32, device)
        if cu.shape != (shape[0] + 1,):
            raise ValueError(f"{name} must be [B + 1]")
    return shape


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
    ref, dtype = cache._call_ref(), _dtype16(k, "k")
    kp, vp = _view(k, "k", dtype, cache._device), _view(v, "v", dtype, cache._device)
    _rows3(k, "k", cache._Hkv, cache._Dqk)
    _rows3(v, "v", cache._Hkv, cache._Dv)
    T = _c_int(k.size(0), "the number of rows")
    if v.size(0) != T:
        raise ValueError("k and v must have the same number of rows")
    B, max_pages = _sequences(cache, page_table, seq_lens, cu_new, "cu_new")
    _launch(cache._device, _call("psf_kv_cache_append"), ref, kp, vp, _thd_strides(k, v), _DTYPES[dtype],
            _ptr(cu_new), page_table.data_ptr(), seq_lens.data_ptr(), B, max_pages, T)


@functools.lru_cache(maxsize=256)
def _attn_workspace(*sizes) -> int:
    for x in sizes:
        _c_int(x, "a size")
    return int(_call("psf_attn_cache_workspace_size")(*sizes))


def attn_cache_workspace_size(cache, B, max_pages, Hq, max_q=1, accumulate=False) -> int:
    return _attn_workspace(B, max_pages, cache._page_size, Hq, cache._Hkv, cache._Dqk, cache._Dv, max_q,
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
    ref, dtype, device = cache._call_ref(), _dtype16(q, "q"), cache._device
    qp = _view(q, "q", dtype, device)
    if q.dim() != 3 or q.size(2) != cache._Dqk:
        raise ValueError(f"q must be [T, Hq, {cache._Dqk}], got {list(q.shape)}")
    T, Hq, _ = q.shape
    if T * Hq > 0x7fffffff:
        raise ValueError(f"q must have fewer than 2^31 rows and heads, got {list(q.shape)}")
    B, max_pages = _sequences(cache, page_table, seq_lens, cu_q, "cu_q")
    if max_q is None:
        if cu_q is not None:
            raise ValueError("cu_q needs max_q, the most query rows of a sequence")
        max_q = T // B if B else 0
    max_q = _c_int(max_q, "max_q")
    if out is None:
        out = torch.empty((T, Hq, cache._Dv), dtype=dtype, device=q.device)
        op = out.data_ptr()
    else:
        op = _view(out, "out", dtype, device)
        _rows3(out, "out", Hq, cache._Dv)
        if out.size(0) != T:
            raise ValueError("out must have q's rows")
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    else:
        _tensor(lse, "lse", torch.float32, device)
        if lse.shape != (Hq, T):
            raise ValueError(f"lse must be [{Hq}, {T}], got {list(lse.shape)}")
    if workspace is None:
        size = attn_cache_workspace_size(cache, B, max_pages, Hq, max_q, accumulate)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    else:
        _tensor(workspace, "workspace", workspace.dtype, device)
        size = workspace.numel() * workspace.element_size()
    _launch(device, _call("psf_attn_cache_fwd"), qp, ref, op, lse.data_ptr(), _ptr(cu_q),
            page_table.data_ptr(), seq_lens.data_ptr(), B, max_pages, T, max_q, Hq, _thd_strides(q, out),
            _DTYPES[dtype], float(scale), 1 if causal else 0, _c_int(_window(window), "window"), _cap(softcap),
            PSF_CACHE_ACCUMULATE if accumulate else 0, workspace.data_ptr(), size)
    return out, lse


@functools.lru_cache(maxsize=256)
def _evict_workspace(*sizes) -> int:
    for x in sizes:
        _c_int(x, "a size")
    return int(_call("psf_kv_cache_evict_workspace_size")(*sizes))


def kv_cache_evict_workspace_size(cache, B, max_pages, budget) -> int:
    return _evict_workspace(B, max_pages, cache._page_size, cache._Hkv, budget)


def kv_cache_evict(cache, page_table, seq_lens, budget, recent, new_lens=None, workspace=None):
    """Cut every sequence longer than budget down to it, in place -> new lengths (int32 [B]).

    For each KV head on its own: the last `recent` tokens stay, and of the others the budget - recent with the largest
    accumulated weight (of equal ones the earliest), in their order. Pages past ceil(budget / page_size) are free
    afterwards. See psf_kv_cache_evict for the scales.
    """
    ref = cache._call_ref()
    B, max_pages = _sequences(cache, page_table, seq_lens)
    budget, recent = _c_int(budget, "budget"), _c_int(recent, "recent")
    if new_lens is None:
        new_lens = torch.empty_like(seq_lens)
    else:
        _tensor(new_lens, "new_lens", torch.int32, cache._device)
        if new_lens.shape != (B,):
            raise ValueError("new_lens must be [B]")
    if workspace is None:
        size = kv_cache_evict_workspace_size(cache, B, max_pages, budget)
        workspace = torch.empty(size, dtype=torch.uint8, device=seq_lens.device)
    else:
        _tensor(workspace, "workspace", workspace.dtype, cache._device)
        size = workspace.numel() * workspace.element_size()
    _launch(cache._device, _call("psf_kv_cache_evict"), ref, page_table.data_ptr(), seq_lens.data_ptr(),
            new_lens.data_ptr(), B, max_pages, budget, recent, workspace.data_ptr(), size)
    return new_lens


def kv_cache_gather(cache, page_table, seq_lens, total_k, dtype=torch.bfloat16):
    """The cached rows of all sequences, packed -> (k [total_k, Hkv, Dqk], v [total_k, Hkv, Dv], cu_k int32 [B + 1]).

    total_k: at least the sum of the lengths (rows past it are not written). With cu_q these are the arguments of
    ``attn_varlen_fwd`` for a prompt chunk over its cached prefix (max_k=-1: no bound to check).
    """
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bfloat16 or float16, got {dtype}")
    total_k = _c_int(total_k, "total_k")
    if total_k < 0:
        raise ValueError("total_k must not be negative")
    ref = cache._call_ref()
    B, max_pages = _sequences(cache, page_table, seq_lens)
    dev = seq_lens.device
    k = torch.empty((total_k, cache._Hkv, cache._Dqk), dtype=dtype, device=dev)
    v = torch.empty((total_k, cache._Hkv, cache._Dv), dtype=dtype, device=dev)
    cu_k = torch.empty(B + 1, dtype=torch.int32, device=dev)
    _launch(cache._device, _call("psf_kv_cache_gather"), ref, page_table.data_ptr(), seq_lens.data_ptr(), B,
            max_pages, k.data_ptr(), v.data_ptr(), cu_k.data_ptr(), total_k, _DTYPES[dtype])
    return k, v, cu_k
