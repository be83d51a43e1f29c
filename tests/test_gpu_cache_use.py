"""GPU tests of the 8-bit cache: what a program may do with its tensors between calls, and less usual forms."""

import pytest
import torch

import cache_reference as ref
import packed_sequence_flash_gb300 as psf
from test_gpu_cache import close, i32, random_cache, same, tables

pytestmark = pytest.mark.gpu



@pytest.fixture(autouse=True)
def _clean_status():
    assert psf.device_status() == 0
    yield


@pytest.mark.parametrize("how", ["assigned", "data"])
def test_weights_cleared_by_new_tensors(how):
    """Weights replaced between requests are the ones that attention, append and eviction use; the old ones stay."""
    lens = [150, 90]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 2, 64, 64, 32, weights=True)
    old = cache.weight
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    if how == "assigned":
        cache.weight = torch.zeros_like(old)
    else:
        old = old.clone()
        cache.weight.data = torch.zeros_like(old)
    kept = old.clone()
    c = ref.from_cache(cache)
    psf.attn_cache_fwd(q, cache, t, i32(lens), 0.125, accumulate=True)
    want = ref.attend(c, q, rows, lens, [0, 1, 2], 0.125, accumulate=True)
    close(cache.weight, c["w"], want[4], "weight")
    c["w"] = cache.weight.cpu().double()
    x = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    psf.kv_cache_append(cache, x, x, t, i32(lens))
    ref.append(c, x, x, rows, lens, [0, 1, 2])
    assert psf.kv_cache_evict(cache, t, i32(lens), 60, 8).tolist() == ref.evict(c, rows, lens, 60, 8)
    same(cache, c)
    assert torch.equal(old, kept) and psf.device_status() == 0
