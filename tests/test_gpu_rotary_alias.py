"""GPU tests of one tensor given twice to the rotation: as inputs it may be, as results it is refused."""
import pytest
import torch

import packed_sequence_flash_gb300 as psf
from test_gpu_cache import i32, random_cache, tables
from test_gpu_rotary import normal

pytestmark = pytest.mark.gpu


def test_one_tensor_twice():
    x, r = normal(50, 4, 64), psf.Rotary(psf.rotary_frequencies(64))
    want = psf.rotary_fwd(x, None, r)[0]
    before = x.clone()
    q, k = psf.rotary_fwd(x, x, r)  # as inputs alone
    assert torch.equal(q, want) and torch.equal(k, want) and torch.equal(x, before)
    y = torch.empty_like(x)
    for kw in (dict(q_out=x, k_out=x), dict(q_out=y, k_out=y), dict(q_out=x), dict(k_out=x)):
        with pytest.raises(psf.PSFError, match="of their own"):
            psf.rotary_fwd(x, x, r, **kw)
    assert torch.equal(x, before)


def test_queries_of_an_append_onto_its_keys():
    rows, t, pages = tables([20], 16)
    cache, r = random_cache(pages, 2, 64, 64, 16), psf.Rotary(psf.rotary_frequencies(64))
    k, v = normal(20, 2, 64), normal(20, 2, 64, seed=1)
    codes, q = cache.k.view(torch.uint8).clone(), k.clone()
    for out in (k, v):
        with pytest.raises(psf.PSFError, match="q_out"):
            psf.kv_cache_append_rotary(cache, k, v, r, t, i32([20]), q=q, q_out=out)
    assert torch.equal(cache.k.view(torch.uint8), codes) and torch.equal(k, q)
    want = psf.rotary_fwd(q, None, r)[0]
    assert torch.equal(psf.kv_cache_append_rotary(cache, k, v, r, t, i32([20]), q=k), want)  # the keys as queries
