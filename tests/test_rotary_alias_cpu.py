"""Results of the rotation that would be written while others read or write them, on the CPU (stand-in addresses)."""
import pytest

from test_cache_cpu import A, EINVAL, lib, struct  # noqa: F401 (a fixture)
from test_rotary_cpu import append, rotate
from test_rotary_shard_cpu import rotate as rotate_shard

B, C = 2 * A, 3 * A


@pytest.mark.parametrize("kw", [dict(q=A, k=A, qo=A, ko=A), dict(q=A, k=B, qo=C, ko=C), dict(q=A, k=B, qo=B, ko=C),
                                dict(q=A, k=B, qo=C, ko=A)])
def test_one_place_for_both_tensors(lib, kw):  # noqa: F811
    for name in ("psf_rotary_fwd", "psf_rotary_bwd"):
        for call, n in ((rotate, name), (rotate_shard, name.replace("rotary", "rotary_varlen"))):
            assert call(lib, name=n, **kw) == EINVAL and b"of their own" in lib.psf_last_error()
            assert call(lib, name=n, S=0, **kw) == 0  # nothing is written


def test_append_of_queries_onto_keys(lib):  # noqa: F811
    c = struct(v=9 * A, v_scale=8 * A)
    for kw in (dict(k=A, v=B, q=C, qo=A), dict(k=A, v=B, q=C, qo=B), dict(k=A, v=B, q=A, qo=A)):
        assert append(lib, c=c, **kw) == EINVAL and b"q_out" in lib.psf_last_error()
