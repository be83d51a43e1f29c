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


def test_a_sequence_without_keys_and_very_many_rows():
    """2^27 rows of head dim 128, 2^31 vectors of 16 bytes, all zero; the row of a sequence behind them is right."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    rows, D = 2 ** 27, 128
    cache = random_cache(4, 1, D, D, 16)
    lens, table = [0, 20], [[-1, -1], [2, 1]]
    # query rows that overlap (8 elements apart): the rows without keys are not read
    q = torch.randn(rows * 8 + D, dtype=torch.bfloat16, device="cuda").as_strided((rows + 1, 1, D), (8, D, 1))
    out = torch.full((rows + 1, 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((1, rows + 1), 3.0, device="cuda")
    psf.attn_cache_fwd(q, cache, i32(table), i32(lens), 0.1, cu_q=i32([0, rows, rows + 1]), max_q=rows, out=out, lse=lse)
    assert psf.device_status() == 0
    for part in out[:rows].split(2 ** 24):
        assert not part.view(torch.int64).any()
    assert bool(lse[:, :rows].isneginf().all())
    want = ref.attend(ref.from_cache(cache), q[rows:], table[1:], lens[1:], [0, 1], 0.1)
    close(out[rows:], want[0], want[2], "out")
    close(lse[:, rows:], want[1], want[3], "lse")
    del q, out, lse, part
    torch.cuda.empty_cache()
