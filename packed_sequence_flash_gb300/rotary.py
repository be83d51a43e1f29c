"""Position rotation of queries and keys, and the cache's append with it.

Python binding of ``psf_rotary_fwd`` / ``_bwd``, ``psf_rotary_varlen_fwd`` / ``_bwd`` and
``psf_kv_cache_append_rotary``: argument marshalling only, as in ``cache.py``.

Training::

    rotary = Rotary(rotary_frequencies(128))
    q, k = rotary_fwd(q, k, rotary, cu_seqlens=cu)             # positions start anew in every document
    out, lse = attn_varlen_fwd(q, k, v, cu, cu, ...)
    dq, dk, dv = attn_varlen_bwd(dout, q, k, v, out, lse, ...)
    dq, dk = rotary_bwd(dq, dk, rotary, cu_seqlens=cu)

A query shard of documents, with the segments of ``build_doc_segments``::

    q, _ = rotary_fwd(q, None, rotary, cu_seqlens=cu_q, dev_meta=meta, cu_seqlens_k=cu_k)   # also where it begins inside one
    _, k = rotary_fwd(None, k, rotary, cu_seqlens=cu_k, dev_meta=meta)

Serving::

    q = kv_cache_append_rotary(cache, k, v, rotary, page_table, seq_lens, cu_new, q=q)
    out, lse = attn_cache_fwd(q, cache, page_table, seq_lens, scale, cu_q=cu_new, max_q=m)

Nothing here synchronises; every call can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import PSF_LAYOUT_BHSD, PSF_LAYOUT_THD
from .attention import _DTYPES, _ptr
from .cache import _c_int, _call, _dtype16, _launch, _rows3, _sequences, _tensor, _view, _wrong_device


def rotary_frequencies(dim, base=10000.0, device="cuda") -> torch.Tensor:
    """base^(-2 i / dim) for the dim / 2 pairs, fp32."""
    if dim < 2 or dim % 2:
        raise ValueError(f"dim must be even and positive, got {dim}")
    i = torch.arange(0, dim, 2, dtype=torch.float64)
    return (float(base) ** (-i / dim)).float().to(device)


class Rotary:
    """A rotation: what turns, how fast, and after which axis.

    inv_freq (fp32 [dim / 2], on the device): radians per position of each pair. The pairs are components (i, i + dim / 2)
    of [start, start + dim) of a head, or (2 i, 2 i + 1) with interleaved. axes: the axis (0 to 7) that each pair takes
    its position from, as dim / 2 numbers; or sections: how many pairs, one run after the other, follow each axis. scale: a
    factor of the rotated components.
    """

    __slots__ = ("_inv_freq", "_axes", "_struct", "_ref", "_address", "_held", "_device")

    def __init__(self, inv_freq, axes=None, sections=None, start=0, interleaved=False, scale=1.0):
        device = inv_freq.get_device()
        if device < 0:
            _wrong_device(inv_freq, "inv_freq")
        _tensor(inv_freq, "inv_freq", torch.float32, device)
        if inv_freq.dim() != 1 or not 1 <= inv_freq.numel() <= 256:
            raise ValueError(f"inv_freq must be [dim / 2] with 1 to 256 pairs, got {list(inv_freq.shape)}")
        half = inv_freq.numel()
        if sections is not None:
            if axes is not None:
                raise ValueError("axes and sections exclude each other")
            axes = [axis for axis, pairs in enumerate(sections) for _ in range(pairs)]
        if axes is not None:
            axes = [int(a) for a in axes]
            if len(axes) != half or any(not 0 <= a < 8 for a in axes):
                raise ValueError(f"axes must name an axis, 0 to 7, for each of the {half} pairs")
            axes = (ctypes.c_uint8 * half)(*axes)
        self._inv_freq, self._axes, self._device = inv_freq, axes, device
        self._struct = _lib.RotaryStruct(inv_freq.data_ptr(), None if axes is None else ctypes.addressof(axes), 2 * half,
                                         _c_int(start, "start"), 1 if interleaved else 0, float(scale))
        self._ref = ctypes.byref(self._struct)
        self._address, self._held = inv_freq.data_ptr(), inv_freq.untyped_storage()

    @property
    def inv_freq(self):
        return self._inv_freq

    def _call_ref(self, device):
        if device != self._device:
            raise ValueError("the rotation's inv_freq must be on the tensors' device")
        if self._inv_freq.data_ptr() != self._address:  # its memory was exchanged (t.data = u, t.set_(u))
            t = self._inv_freq
            if t.shape != (self._struct.dim // 2,):
                raise ValueError("inv_freq no longer has its size")
            _tensor(t, "inv_freq", torch.float32, self._device)
            self._struct.inv_freq = self._address = t.data_ptr()
            self._held = t.untyped_storage()
        return self._ref


def _positions(positions, shape, device):
    """(address, axes) of positions [rows] or [axes, rows], rows as in shape ([T], or [B, S])."""
    _tensor(positions, "positions", torch.int32, device)
    if positions.shape == shape:
        return positions.data_ptr(), 1
    if positions.dim() != len(shape) + 1 or positions.shape[1:] != shape or not 1 <= positions.size(0) <= 8:
        raise ValueError(f"positions must be {list(shape)} or [axes, ...] of it, got {list(positions.shape)}")
    return positions.data_ptr(), positions.size(0)


def _steps(t):
    """Element strides (batch, head, row) of a [T, H, D] or [B, H, S, D] tensor."""
    return [0, t.stride(1), t.stride(0)] if t.dim() == 3 else [t.stride(0), t.stride(1), t.stride(2)]


def _strides(tensors):
    for t in tensors:
        if t is not None and not t.is_contiguous():
            break
    else:
        return None
    vals = [x for t in tensors for x in ([0, 0, 0] if t is None else _steps(t))]
    return (ctypes.c_int64 * len(vals))(*vals)


def _result(t, out, name, dtype, device):
    """The result of t and its address (made here, or the caller's)."""
    if out is None:
        out = torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=dtype, device=t.device)
        return out, out.data_ptr()
    if out is not t:
        if out.shape != t.shape:
            raise ValueError(f"{name} must be {list(t.shape)}, got {list(out.shape)}")
    return out, _view(out, name, dtype, device)


def _rotate(way, q, k, rotary, positions, cu_seqlens, dev_meta, q_out, k_out, cu_seqlens_k, names):
    first, first_name = (q, names[0]) if q is not None else (k, names[1])
    if first is None:
        raise ValueError(f"{names[0]} or {names[1]} must be given")
    dtype, device, shape = _dtype16(first, first_name), first.get_device(), first.shape
    if device < 0:
        _wrong_device(first, first_name)
    if len(shape) == 3:
        layout, B, S = PSF_LAYOUT_THD, 1, shape[0]
        rows = shape[:1]
    elif len(shape) == 4:
        layout, B, S = PSF_LAYOUT_BHSD, shape[0], shape[2]
        rows = torch.Size((B, S))
    else:
        raise ValueError(f"{first_name} must be [T, H, D] or [B, H, S, D], got {list(shape)}")
    if B * S > 0x7fffffff:
        raise ValueError("the number of rows must fit in 32 bits")
    Hq = Hkv = 0
    qp = kp = qo = ko = None
    if q is not None:
        qp, Hq = _view(q, names[0], dtype, device), shape[1]
        q_out, qo = _result(q, q_out, names[0] + "_out", dtype, device)
    elif q_out is not None:
        raise ValueError(f"{names[0]}_out without its input")
    if k is not None:
        kp, other = _view(k, names[1], dtype, device), k.shape
        if len(other) != len(shape) or other[0] != shape[0] or other[2:] != shape[2:]:
            raise ValueError(f"{names[0]} and {names[1]} must have the same rows and head dim")
        Hkv = other[1]
        k_out, ko = _result(k, k_out, names[1] + "_out", dtype, device)
    elif k_out is not None:
        raise ValueError(f"{names[1]}_out without its input")
    pos, axes = (None, 0) if positions is None else _positions(positions, rows, device)
    cu, nseg = None, 0
    if cu_seqlens is not None:
        _tensor(cu_seqlens, "cu_seqlens", torch.int32, device)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [segments + 1]")
        if positions is not None:
            raise ValueError("positions and cu_seqlens exclude each other")
        cu, nseg = cu_seqlens.data_ptr(), cu_seqlens.numel() - 1
    if cu_seqlens_k is not None:
        _tensor(cu_seqlens_k, "cu_seqlens_k", torch.int32, device)
        if cu_seqlens is None or cu_seqlens_k.shape != cu_seqlens.shape:
            raise ValueError("cu_seqlens_k must be [segments + 1] like cu_seqlens, which it comes with")
    if dev_meta is not None:
        _tensor(dev_meta, "dev_meta", torch.int32, device)
        dev_meta = dev_meta.data_ptr()
    if B:
        if cu_seqlens_k is None:
            call, places = "psf_rotary_" + way, (pos, axes, cu)
        else:
            call, places = "psf_rotary_varlen_" + way, (cu, cu_seqlens_k.data_ptr())
        _launch(device, _call(call), qp, kp, qo, ko, rotary._call_ref(device), *places, dev_meta, nseg, layout, B, S,
                Hq, Hkv, shape[-1], _strides((q, k, q_out, k_out)), _DTYPES[dtype])
    return q_out, k_out


def rotary_fwd(q, k, rotary, positions=None, cu_seqlens=None, dev_meta=None, q_out=None, k_out=None, cu_seqlens_k=None):
    """Turns q [T, Hq, D] and k [T, Hkv, D] (or [B, H, S, D]; bf16 or fp16; one may be None) -> (q_out, k_out).

    positions int32 [T] or [axes, T] (or [B, S], [axes, B, S]); or cu_seqlens int32 [segments + 1]: a row's place in its
    segment (dev_meta: the segment builder's, with the count on the device); neither: its place in its batch row. q_out
    may be q itself (in place), k_out k. See psf_rotary.
    cu_seqlens_k: with the keys' prefix sums beside the rows' own, a row's place is that among its segment's keys, to whose
    end the rows are aligned as in ``attn_varlen_fwd``. A shard that begins inside a document (q_global_start > 0) needs it:
    by cu_seqlens alone its rows would count from the shard's edge. See psf_rotary_varlen_fwd.
    """
    return _rotate("fwd", q, k, rotary, positions, cu_seqlens, dev_meta, q_out, k_out, cu_seqlens_k, ("q", "k"))


def rotary_bwd(dq, dk, rotary, positions=None, cu_seqlens=None, dev_meta=None, dq_out=None, dk_out=None, cu_seqlens_k=None):
    """The gradients of rotary_fwd's inputs from those of its results, with the same rotation and positions."""
    return _rotate("bwd", dq, dk, rotary, positions, cu_seqlens, dev_meta, dq_out, dk_out, cu_seqlens_k, ("dq", "dk"))


def kv_cache_append_rotary(cache, k, v, rotary, page_table, seq_lens, cu_new=None, positions=None, q=None, q_out=None):
    """``kv_cache_append`` with k turned on the way -> q_out, the same tokens' queries turned (None without q).

    positions int32 [T] or [axes, T]: default the tokens' places in their sequences (an evicted sequence counts its kept
    tokens only, so it wants positions). q [T, Hq, Dqk]; q_out may be q itself. See psf_kv_cache_append_rotary.
    """
    ref, dtype, device = cache._call_ref(), _dtype16(k, "k"), cache._device
    kp, vp = _view(k, "k", dtype, device), _view(v, "v", dtype, device)
    _rows3(k, "k", cache._Hkv, cache._Dqk)
    _rows3(v, "v", cache._Hkv, cache._Dv)
    T = _c_int(k.size(0), "the number of rows")
    if v.size(0) != T:
        raise ValueError("k and v must have the same number of rows")
    Hq, qp, qo = 0, None, None
    if q is not None:
        qp = _view(q, "q", dtype, device)
        if q.dim() != 3 or q.size(0) != T or q.size(2) != cache._Dqk:
            raise ValueError(f"q must be [{T}, Hq, {cache._Dqk}], got {list(q.shape)}")
        Hq = q.size(1)
        q_out, qo = _result(q, q_out, "q_out", dtype, device)
    elif q_out is not None:
        raise ValueError("q_out without its input")
    pos, axes = (None, 0) if positions is None else _positions(positions, k.shape[:1], device)
    B, max_pages = _sequences(cache, page_table, seq_lens, cu_new, "cu_new")
    _launch(device, _call("psf_kv_cache_append_rotary"), ref, kp, vp, qp, qo, rotary._call_ref(device), pos, axes,
            _strides((k, v, q, q_out)), _DTYPES[dtype], _ptr(cu_new), page_table.data_ptr(), seq_lens.data_ptr(), B, max_pages,
            T, Hq)
    return q_out
