"""Refusals of the rotation of a shard's rows, on the CPU (stand-in addresses, never dereferenced)."""
import ctypes

import pytest

from test_cache_cpu import A, EINVAL, lib  # noqa: F401 (a fixture)
from test_rotary_cpu import BAD_ROTATIONS, rot, strides


def rotate(lib, name, r=None, **kw):  # noqa: F811
    a = dict(q=A, k=A, qo=2 * A, ko=2 * A, cu=A, cu_k=A, meta=None, nseg=3, layout=0, B=1, S=8, Hq=4, Hkv=2, D=128,
             strides=None, dtype=0)
    a.update(kw)
    return getattr(lib, name)(a["q"], a["k"], a["qo"], a["ko"], ctypes.byref(r or rot()), a["cu"], a["cu_k"], a["meta"],
                              a["nseg"], a["layout"], a["B"], a["S"], a["Hq"], a["Hkv"], a["D"], a["strides"], a["dtype"],
                              None)


NAMES = pytest.mark.parametrize("name", ["psf_rotary_varlen_fwd", "psf_rotary_varlen_bwd"])


@NAMES
@pytest.mark.parametrize("kw", [
    dict(cu=None), dict(cu_k=None), dict(nseg=-1), dict(layout=2), dict(B=0), dict(B=2), dict(S=-1), dict(Hq=0, Hkv=0),
    dict(D=100), dict(dtype=2), dict(q=None), dict(ko=None), dict(k=A + 8),
    dict(strides=strides(0, 128, 512, 0, 128, 252, 0, 128, 512, 0, 128, 256))])
def test_arguments(lib, name, kw):  # noqa: F811
    assert rotate(lib, name, **kw) == EINVAL, lib.psf_last_error()


@NAMES
@pytest.mark.parametrize("bad", BAD_ROTATIONS)
def test_rotations(lib, name, bad):  # noqa: F811
    assert rotate(lib, name, r=rot(**bad)) == EINVAL


@NAMES
def test_calls_without_rows_are_done(lib, name):  # noqa: F811
    assert rotate(lib, name, S=0) == 0
