"""GPU test of the prompt attention's waits that run out: a status, and the next call is right."""
import pytest
import torch

import packed_sequence_flash_gb300 as psf
from test_gpu_cache import i32, prefix, random_cache
from test_gpu_prompt import DIMS, queries

pytestmark = pytest.mark.gpu

ETIMEOUT = -5


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("softcap,limit", [(None, 200_000), (30.0, 200_000), (None, 1)])
def test_waits_that_run_out(dims, softcap, limit):
    """Units of up to 128 rows leave half of the softmax warps waiting for the next unit, here for a millisecond and more: under
    a limit of 0.2 ms, or of none, they give up. The units behind them have rows for those warps, so that everything else stops there."""
    assert psf.device_status() == 0
    lens, m_rows, H, page = [1 << 19] * 4, [128, 400, 100, 256], 8, 128
    cache = random_cache(64, H, *dims, page)
    table = (torch.arange(4 * (lens[0] // page)).reshape(4, -1) % 64).int().cuda()  # (pages that are shared: small, and read alone)
    q, n, cu = queries(sum(m_rows), H, dims[0]), i32(lens), i32(prefix(m_rows))
    call = lambda: psf.attn_cache_prompt_fwd(q, cache, table, n, dims[0] ** -0.5, cu, max(m_rows), softcap=softcap)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    assert psf.device_status() == 0
    psf.set_wait_limit_ns(limit)
    try:
        for _ in range(3):
            call()
        torch.cuda.synchronize()
    finally:
        psf.set_wait_limit_ns(2_000_000_000)
    assert psf.device_status() == ETIMEOUT
    got = call()
    torch.cuda.synchronize()
    assert psf.device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
