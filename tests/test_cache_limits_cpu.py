"""Sizes at the ends of the 8-bit cache's ranges, on the CPU (stand-in addresses, never dereferenced)."""
import ctypes

import pytest

from test_cache_cpu import A, EINVAL, EWORKSPACE, append, attend, evict, gather, lib, struct  # noqa: F401 (a fixture)


@pytest.mark.parametrize("call", [attend, append, evict, gather])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("tokens", [2 ** 31 - 128, 2 ** 31 - 4096, 2 ** 31 - 2 ** 16 + 128])
def test_tables_past_what_32_bit_counts_hold(lib, call, page, tokens):  # noqa: F811
    """Lengths that the kernels' rounding up and striding would carry past 2^31 - 1."""
    assert call(lib, page_size=page, max_pages=tokens // page) == EINVAL
    assert b"2^31" in lib.psf_last_error(), lib.psf_last_error()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_the_longest_table(lib, page):  # noqa: F811
    pages = (2 ** 31 - 2 ** 16) // page
    assert attend(lib, page_size=page, max_pages=pages) == EWORKSPACE
    assert evict(lib, page_size=page, max_pages=pages) == EWORKSPACE
    assert append(lib, page_size=page, max_pages=pages, T=0) == 0


@pytest.mark.parametrize("entries", [-3, -1, 0, 1, 3])
def test_new_lengths_that_overlap_the_old_ones(lib, entries):  # noqa: F811
    """Four sequences: new lengths written over others that a later selection still reads."""
    assert evict(lib, lens=A, new=A + 4 * entries) == EINVAL
    assert b"overlap" in lib.psf_last_error(), lib.psf_last_error()


@pytest.mark.parametrize("entries", [-4, 4])
def test_new_lengths_beside_the_old_ones(lib, entries):  # noqa: F811
    assert evict(lib, lens=A, new=A + 4 * entries) == EWORKSPACE


@pytest.mark.parametrize("kw", [dict(v=A), dict(v_scale=2 * A), dict(v_scale=2 * A + 4 * 19), dict(v_scale=2 * A - 4)])
def test_caches_whose_keys_and_values_share_memory_are_not_written(lib, kw):  # noqa: F811
    """Ten pages of two heads: the block that has K's scale rewrites it while another one has V's."""
    c = struct(**{**dict(k=A, v=4 * A, k_scale=2 * A, v_scale=3 * A), **kw})
    assert lib.psf_kv_cache_append(ctypes.byref(c), A, A, None, 0, A, A, A, 4, 5, 8, None) == EINVAL
    assert b"of their own" in lib.psf_last_error(), lib.psf_last_error()
    assert lib.psf_kv_cache_evict(ctypes.byref(c), A, A, 2 * A, 4, 5, 100, 10, A, 2 ** 40, None) == EINVAL
    assert b"of their own" in lib.psf_last_error(), lib.psf_last_error()
