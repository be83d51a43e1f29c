"""The binding of the 8-bit cache on the CPU: what a KVCache hands to the library, with stand-ins for CUDA tensors."""
import ctypes

import pytest
import torch

import packed_sequence_flash_gb300 as psf
from packed_sequence_flash_gb300 import cache as binding


class OnDevice:
    """A CPU tensor that says it is on CUDA device 0. Nothing reads its memory here."""

    is_cuda = True

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


def e4m3(*shape):
    return torch.zeros(*shape, dtype=torch.uint8).view(torch.float8_e4m3fn)


def parts(pages=6, H=2, page=16, Dqk=64, Dv=64):
    return dict(k=OnDevice(e4m3(pages, H, page, Dqk)), v=OnDevice(e4m3(pages, H, page, Dv)),
                k_scale=OnDevice(torch.zeros(pages, H)), v_scale=OnDevice(torch.zeros(pages, H)),
                weight=OnDevice(torch.zeros(pages, H, page)))


class Calls:
    """Stands in for the library: keeps what each call was given as its cache, and the other arguments."""

    def __init__(self, monkeypatch):
        self.seen = []
        monkeypatch.setattr(binding, "_call", self.entry)
        monkeypatch.setattr(binding, "_current_device", lambda: 0)
        monkeypatch.setattr(binding, "_raw_stream", lambda device: 0)
        binding._attn_workspace.cache_clear()
        binding._evict_workspace.cache_clear()

    def entry(self, name):
        if name.endswith("workspace_size"):
            return lambda *args: 256

        def call(*args):
            struct = next(ctypes.cast(a, ctypes.POINTER(psf._lib.KVCacheStruct)).contents for a in args
                          if type(a).__name__ == "CArgObject")
            self.seen.append((struct, args))
            return 0

        return call

    def addresses(self):
        c = self.seen[-1][0]
        return dict(k=c.k, v=c.v, k_scale=c.k_scale, v_scale=c.v_scale, weight=c.weight)


@pytest.fixture
def calls(monkeypatch):
    yield Calls(monkeypatch)
    binding._attn_workspace.cache_clear()
    binding._evict_workspace.cache_clear()


def i32(x):
    return OnDevice(torch.tensor(x, dtype=torch.int32))


def every_call(cache):
    """Each of the four operators once, on two sequences."""
    table, lens = i32([[0, 1], [2, 3]]), i32([20, 30])
    x = lambda H, D: OnDevice(torch.zeros(2, H, D, dtype=torch.bfloat16))  # noqa: E731
    out, lse = x(4, cache.Dv), OnDevice(torch.zeros(4, 2))
    ws = OnDevice(torch.zeros(256, dtype=torch.uint8))
    yield lambda: psf.kv_cache_append(cache, x(cache.Hkv, cache.Dqk), x(cache.Hkv, cache.Dv), table, lens)
    yield lambda: psf.attn_cache_fwd(x(4, cache.Dqk), cache, table, lens, 0.1, out=out, lse=lse, workspace=ws)
    yield lambda: psf.kv_cache_evict(cache, table, lens, 16, 4, new_lens=i32([0, 0]), workspace=ws)
    yield lambda: psf.kv_cache_gather(cache, table, lens, 50)


NAMES = ("k", "v", "k_scale", "v_scale", "weight")


@pytest.mark.parametrize("name", NAMES)
def test_a_replaced_tensor_is_the_one_that_calls_get(calls, name):
    p = parts()
    cache = psf.KVCache(**p)
    fresh = parts()[name]
    setattr(cache, name, fresh)
    assert getattr(cache, name) is fresh
    for call in every_call(cache):
        call()
        want = {n: (fresh if n == name else p[n]).data_ptr() for n in NAMES}
        assert calls.addresses() == want


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("how", ["data", "set_"])
def test_a_tensor_with_other_memory_is_taken_anew(calls, name, how):
    p = parts()
    for i in range(4):  # each call is the first one after such a change
        cache = psf.KVCache(**p)
        call = list(every_call(cache))[i]
        fresh = parts()[name].t.clone()
        if how == "data":
            p[name].t.data = fresh
        else:
            p[name].t.set_(fresh)
        call()
        assert calls.addresses() == {n: p[n].data_ptr() for n in NAMES}
        assert calls.addresses()[name] == fresh.data_ptr()


def test_replacements_are_checked(calls):
    p = parts()
    cache = psf.KVCache(**p)
    for name, t in [("k", parts(pages=7)["k"]), ("v", parts(page=32)["v"]), ("k_scale", parts(H=3)["k_scale"]),
                    ("v_scale", OnDevice(torch.zeros(6, 2, dtype=torch.float64))), ("weight", parts(page=32)["weight"]),
                    ("weight", torch.zeros(6, 2, 16)), ("k", OnDevice(torch.zeros(6, 2, 16, 64)))]:
        with pytest.raises(ValueError):
            setattr(cache, name, t)
        assert all(getattr(cache, n) is p[n] for n in NAMES)
    for name in ("num_pages", "Hkv", "page_size", "Dqk", "Dv", "device"):
        with pytest.raises(AttributeError):
            setattr(cache, name, 1)
    cache.weight = None
    assert cache.weight is None
    p["k"].t.data = e4m3(7, 2, 16, 64)  # another number of pages than the scales have
    for call in every_call(cache):
        with pytest.raises(ValueError):
            call()
    assert not calls.seen


def test_memory_of_an_exchanged_tensor_is_not_given_away_before_the_next_call(calls):
    """An address can then be compared: no other memory comes to have it."""
    p = parts()
    cache = psf.KVCache(**p)
    old = p["weight"].t.untyped_storage()
    assert any(s.data_ptr() == old.data_ptr() for s in cache._held)
    p["weight"].t.data = torch.zeros(6, 2, 16)
    del old
    assert any(s.data_ptr() == cache._addresses[4] for s in cache._held)


def test_a_copy_of_a_cache_does_not_follow_its_replacements(calls):
    import copy

    p = parts()
    cache = psf.KVCache(**p)
    other = copy.copy(cache)
    other.weight = parts()["weight"]
    next(every_call(cache))()
    assert calls.addresses()["weight"] == p["weight"].data_ptr()
    next(every_call(other))()
    assert calls.addresses()["weight"] == other.weight.data_ptr()


@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 2, 16), (6, 1, 16), (6, 2, 1)])
def test_expanded_codes_are_refused(name, shape):
    """All strides 0 would be taken for contiguous ones: a cache of 6 pages over the memory of one row."""
    p = parts()
    p[name] = OnDevice(e4m3(*shape, 64).expand(6, 2, 16, 64))
    with pytest.raises(ValueError, match="overlaps"):
        psf.KVCache(**p)
    whole = parts()
    cache = psf.KVCache(**whole)
    with pytest.raises(ValueError, match="overlaps"):
        setattr(cache, name, p[name])
    assert getattr(cache, name) is whole[name]


def test_strides_of_dims_of_one_do_not_matter():
    one = OnDevice(e4m3(1, 1, 16, 64).as_strided((1, 1, 16, 64), (0, 0, 64, 1)))
    s = OnDevice(torch.zeros(1, 1))
    psf.KVCache(one, one, s, s)
    wide = OnDevice(e4m3(1, 1, 16, 128)[..., :64].as_strided((1, 1, 16, 64), (0, 0, 128, 1)))
    assert list(psf.KVCache(wide, one, s, s)._struct.k_strides) == [0, 0, 128]


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1])
def test_numbers_past_32_bits_are_refused(calls, big):
    """ctypes would cut them: a budget of 2^32 + 5 came out as 5."""
    cache = psf.KVCache(**parts())
    table, lens = i32([[0, 1], [2, 3]]), i32([20, 30])
    q = OnDevice(torch.zeros(2, 4, 64, dtype=torch.bfloat16))
    ws, new = OnDevice(torch.zeros(256, dtype=torch.uint8)), i32([0, 0])
    attend = lambda **kw: psf.attn_cache_fwd(q, cache, table, lens, 0.1, workspace=ws, **kw)  # noqa: E731
    for call in (lambda: psf.kv_cache_evict(cache, table, lens, big, 4, new, workspace=ws),
                 lambda: psf.kv_cache_evict(cache, table, lens, 20, big, new, workspace=ws),
                 lambda: attend(max_q=big), lambda: attend(window=big),
                 lambda: psf.kv_cache_gather(cache, table, lens, big),
                 lambda: psf.attn_cache_workspace_size(cache, 2, 2, 4, big),
                 lambda: psf.kv_cache_evict_workspace_size(cache, 2, 2, big)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    assert not calls.seen
    attend(max_q=2 ** 31 - 1, window=2 ** 31 - 1)
    psf.kv_cache_evict(cache, table, lens, 2 ** 31 - 1, 0, new, workspace=ws)
    assert len(calls.seen) == 2
