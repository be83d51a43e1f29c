"""Host-side checks of the 8-bit cache's calls, on the CPU: every refusal of the C ABI (stand-in addresses, never
dereferenced; a missing workspace or a device check stops a call that slipped through) and of the binding."""
import ctypes

import pytest
import torch

import cache_reference as ref
from packed_sequence_flash_gb300 import _lib
import packed_sequence_flash_gb300 as psf

EINVAL, EUNSUPPORTED, EWORKSPACE = -1, -2, -6
A = 0x10000
NO_WINDOW = -(2 ** 31)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def struct(**kw):
    a = dict(k=A, v=A, k_scale=A, v_scale=A, weight=A, num_pages=10, page_size=64, Hkv=2, Dqk=128, Dv=128,
             k_strides=(0, 0, 0), v_strides=(0, 0, 0))
    a.update(kw)
    c = _lib.KVCacheStruct(*[a[n] for n in ("k", "v", "k_scale", "v_scale", "weight", "num_pages", "page_size", "Hkv",
                                            "Dqk", "Dv")])
    c.k_strides[:] = a["k_strides"]
    c.v_strides[:] = a["v_strides"]
    return c


CACHE_KEYS = {"k_", "num_pages", "page_size", "Hkv", "Dqk", "Dv", "k_strides", "v_strides", "k_scale", "weight", "ck"}


def split(kw):
    c = {("k" if n == "ck" else n): x for n, x in kw.items() if n in CACHE_KEYS}
    return struct(**c), {n: x for n, x in kw.items() if n not in CACHE_KEYS}


def attend(lib, **kw):
    c, kw = split(kw)
    a = dict(q=A, out=A, lse=A, cu=A, table=A, lens=A, B=4, max_pages=5, T=8, max_q=2, Hq=4, strides=None, dtype=0,
             scale=0.1, causal=1, window=NO_WINDOW, softcap=0.0, flags=0)
    a.update(kw)
    return lib.psf_attn_cache_fwd(a["q"], ctypes.byref(c), a["out"], a["lse"], a["cu"], a["table"], a["lens"], a["B"],
                                  a["max_pages"], a["T"], a["max_q"], a["Hq"], a["strides"], a["dtype"], a["scale"],
                                  a["causal"], a["window"], a["softcap"], a["flags"], None, 0, None)


def append(lib, **kw):
    c, kw = split(kw)
    a = dict(x=A, strides=None, dtype=0, cu=A, table=A, lens=A, B=4, max_pages=5, T=8)
    a.update(kw)
    return lib.psf_kv_cache_append(ctypes.byref(c), a["x"], a["x"], a["strides"], a["dtype"], a["cu"], a["table"],
                                   a["lens"], a["B"], a["max_pages"], a["T"], None)


def evict(lib, **kw):
    c, kw = split(kw)
    a = dict(table=A, lens=A, new=2 * A, B=4, max_pages=5, budget=100, recent=10)
    a.update(kw)
    return lib.psf_kv_cache_evict(ctypes.byref(c), a["table"], a["lens"], a["new"], a["B"], a["max_pages"], a["budget"],
                                  a["recent"], None, 0, None)


def gather(lib, **kw):
    c, kw = split(kw)
    a = dict(table=A, lens=A, B=4, max_pages=5, k=A, v=A, cu=A, total=100, dtype=0)
    a.update(kw)
    return lib.psf_kv_cache_gather(ctypes.byref(c), a["table"], a["lens"], a["B"], a["max_pages"], a["k"], a["v"],
                                   a["cu"], a["total"], a["dtype"], None)


def test_valid_calls_stop_at_the_workspace(lib):
    assert attend(lib) == EWORKSPACE
    assert attend(lib, cu=None) == EWORKSPACE
    assert evict(lib) == EWORKSPACE
    assert append(lib, T=0) == 0 and attend(lib, T=0) == 0


@pytest.mark.parametrize("call", [attend, append, evict, gather])
@pytest.mark.parametrize("kw,code,word", [
    (dict(page_size=48), EINVAL, b"page_size"), (dict(page_size=256), EINVAL, b"page_size"),
    (dict(num_pages=0), EINVAL, b"num_pages"), (dict(Hkv=0), EINVAL, b"Hkv"),
    (dict(Dqk=96, Dv=96), EUNSUPPORTED, b"head dims"), (dict(ck=None), EINVAL, b"null"),
    (dict(ck=A + 8), EINVAL, b"aligned"), (dict(k_scale=None), EINVAL, b"null"),
    (dict(k_strides=(64 * 256, 8, 128)), EINVAL, b"stride"), (dict(k_strides=(64 * 256, 64, 128)), EINVAL, b"overlaps"),
    (dict(v_strides=(-64 * 256, 8192, 128)), EINVAL, b"stride"),
    (dict(B=0), EINVAL, b"B"), (dict(B=70000), EINVAL, b"B"), (dict(max_pages=0), EINVAL, b"max_pages"),
    (dict(max_pages=2 ** 26), EINVAL, b"2^31"), (dict(table=None), EINVAL, b"null"), (dict(lens=None), EINVAL, b"null"),
])
def test_cache_and_sequences_are_checked(lib, call, kw, code, word):
    assert call(lib, **kw) == code
    assert word in lib.psf_last_error(), lib.psf_last_error()


@pytest.mark.parametrize("kw,code,word", [
    (dict(Hq=5), EINVAL, b"Hq"), (dict(window=0), EINVAL, b"window"), (dict(scale=0.0), EINVAL, b"scale"),
    (dict(scale=float("inf")), EINVAL, b"scale"), (dict(softcap=-1.0), EINVAL, b"softcap"),
    (dict(dtype=2), EINVAL, b"dtype"), (dict(flags=2), EINVAL, b"flags"), (dict(flags=1, weight=None), EINVAL, b"weights"),
    (dict(cu=None, T=7), EINVAL, b"divide"), (dict(cu=None, max_q=1), EINVAL, b"max_q"), (dict(max_q=-1), EINVAL, b"max_q"),
    (dict(max_q=2 ** 30, T=2 ** 30, cu=A), EINVAL, b"2^31"), (dict(max_q=2 ** 31 - 1, Hq=2), EINVAL, b"2^31"),
    (dict(T=2 ** 30, Hq=4), EINVAL, b"2^31"),
    (dict(q=None), EINVAL, b"null"), (dict(out=A + 4), EINVAL, b"aligned"), (dict(T=-1), EINVAL, b"T"),
    (dict(strides=(ctypes.c_int64 * 6)(0, 4, 512, 0, 128, 512)), EINVAL, b"stride"),
    (dict(strides=(ctypes.c_int64 * 6)(0, 128, 512, 0, 64, 512)), EINVAL, b"overlaps"),
])
def test_attention_arguments(lib, kw, code, word):
    assert attend(lib, **kw) == code
    assert word in lib.psf_last_error(), lib.psf_last_error()


@pytest.mark.parametrize("call,kw,word", [
    (append, dict(dtype=3), b"dtype"), (append, dict(x=None), b"null"), (append, dict(x=A + 2), b"aligned"),
    (append, dict(cu=None, T=7), b"divide"), (append, dict(T=-4), b"T"),
    (append, dict(strides=(ctypes.c_int64 * 6)(0, 100, 512, 0, 128, 512)), b"stride"),
    (evict, dict(weight=None), b"weights"), (evict, dict(budget=0), b"budget"), (evict, dict(recent=-1), b"recent"),
    (evict, dict(recent=101), b"recent"), (evict, dict(new=A), b"new_lens"), (evict, dict(new=None), b"new_lens"),
    (gather, dict(dtype=-1), b"dtype"), (gather, dict(total=-1), b"total_k"), (gather, dict(cu=None), b"null"),
    (gather, dict(k=A + 8), b"aligned"),
])
def test_other_arguments(lib, call, kw, word):
    assert call(lib, **kw) == EINVAL
    assert word in lib.psf_last_error(), lib.psf_last_error()


def test_workspace_sizes(lib):
    size = lib.psf_attn_cache_workspace_size
    assert size(4, 100, 64, 32, 8, 128, 128, 1, 0) > 0
    assert size(4, 100, 64, 32, 8, 128, 128, 1, 1) >= size(4, 100, 64, 32, 8, 128, 128, 1, 0)
    assert size(0, 100, 64, 32, 8, 128, 128, 1, 0) == 0 and size(4, 100, 64, 33, 8, 128, 128, 1, 0) == 0
    ev = lib.psf_kv_cache_evict_workspace_size
    assert ev(4, 100, 64, 8, 1000) >= 4 * 8 * 1000 * 12
    assert ev(4, 100, 64, 8, 0) == 0
    # a budget past what the table holds takes no more than one that fills it
    assert ev(4, 100, 64, 8, 10 ** 9) == ev(4, 100, 64, 8, 6400)


def test_binding_refuses_tensors_of_the_cpu():
    k = torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        psf.KVCache(k, k, s, s)


def test_reference_rounding_and_scale():
    """The tests' own e4m3 rounding against torch's, and the scale rule at its borders."""
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.logspace(-4, 2.6, 5000), torch.tensor([0.0])]).double()
    assert torch.equal(ref.e4m3(x.float().double()), x.float().to(torch.float8_e4m3fn).double())
    assert ref.scale_of(448.0) == 1.0 and ref.scale_of(448.5) == 2.0 and ref.scale_of(224.0) == 0.5
    assert ref.scale_of(0.0) == 2.0 ** -126 and ref.scale_of(1e-45) == 2.0 ** -126


def test_workspace_sizes_that_no_memory_holds(lib):
    """Products past 2^64 do not come out as small sizes: a call with such a workspace is refused."""
    big = 2 ** 64 - 1
    assert lib.psf_attn_cache_workspace_size(65534, 2 ** 24 - 1, 128, 4096, 2, 128, 128, 2 ** 19 - 1, 1) == big
    assert lib.psf_attn_cache_workspace_size(65534, 2 ** 24 - 1, 128, 4096, 2, 128, 128, 2 ** 19 - 1, 0) < 2 ** 30
    assert lib.psf_kv_cache_evict_workspace_size(65534, 2 ** 24 - 1, 128, 65535, 2 ** 31 - 1) == big
    assert attend(lib, B=65534, max_pages=2 ** 23, page_size=128, Hq=4096, max_q=2 ** 18, flags=1) == EWORKSPACE
