"""GPU tests of the prompt attention where the other file's cases do not lead: capped logits over one scale per 64 keys, values whose
pages differ under a cap, hundreds of sequences of several row tiles, chunks beside decode steps, graphs that share a workspace."""
import random

import pytest
import torch

import packed_sequence_flash_gb300 as psf
from test_gpu_cache import i32, prefix, random_cache, tables
from test_gpu_prompt import DIMS, check, queries, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    assert psf.device_status() == 0
    yield


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("softcap,size", [(2.0, 2.0), (30.0, 1.0), (100.0, 20.0)])
@pytest.mark.parametrize("window", [None, 100])
def test_capped(dims, page, softcap, size, window):
    lens, m_rows = [90, 700, 0, 257, 300], [100, 300, 20, 257, 1]
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 2, *dims, page, seed=2)
    check(cache, queries(sum(m_rows), 6, dims[0], size=size), rows, t, lens, m_rows, 0.1, window=window, softcap=softcap)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("softcap", [None, 20.0])
def test_scales_of_very_different_pages(dims, softcap):
    lens, m_rows, page = [1000], [200], 64
    rows, t, pages = tables(lens, page)
    t = wide(t, page)
    cache = random_cache(pages, 1, *dims, page)
    g = torch.Generator().manual_seed(5)
    cache.v_scale = torch.exp2(torch.randint(-30, 30, (pages, 1), generator=g).float()).cuda()
    cache.k_scale = (torch.exp2(torch.randint(-40, -4, (pages, 1), generator=g).float()) * 1.37).cuda()
    cache.v_scale[rows[0][3]] = 0
    cache.k_scale[rows[0][5]] = 0
    check(cache, queries(200, 4, dims[0]), rows, t, lens, m_rows, 0.3, softcap=softcap)


@pytest.mark.parametrize("dims", DIMS)
def test_hundreds_of_sequences_of_several_row_tiles(dims):
    r = random.Random(9)
    lens = [r.choice([0, 3, 70, 150, 280]) for _ in range(700)]
    m_rows = [min(n, r.choice([0, 1, n, n, 130])) for n in lens]
    rows, t, pages = tables(lens, 128)
    cache = random_cache(pages, 1, *dims, 128)
    check(cache, queries(sum(m_rows), 4, dims[0]), rows, t, lens, m_rows, dims[0] ** -0.5)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 128])
def test_a_chunk_beside_decode_steps(dims, page):
    """Units of one row, whose half of the softmax has nothing to do, before, between and behind full ones; rows as in calls of
    their own."""
    lens = [900, 1000, 2000, 333, 1, 1500]
    m_rows = [1, 300, 1, 200, 1, 1]
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 2, *dims, page)
    check(cache, queries(sum(m_rows), 8, dims[0], torch.float16), rows, t, lens, m_rows, dims[0] ** -0.5)


def test_two_graphs_share_a_workspace():
    """Replayed one behind the other in one stream, in any order."""
    lens, page = [5000, 700], 64
    rows, t, pages = tables(lens, page)
    t = wide(t, page)
    cache = random_cache(pages, 2, 128, 128, page)
    ws = torch.empty(psf.attn_cache_prompt_workspace_size(cache, 2, t.size(1), 8, 300), dtype=torch.uint8, device="cuda")
    calls = []
    for m_rows, seed in (([300, 200], 1), ([40, 300], 2)):
        q, cu, n = queries(sum(m_rows), 8, 128, seed=seed), i32(prefix(m_rows)), i32(lens)
        out, lse = torch.empty_like(q), torch.empty(8, sum(m_rows), device="cuda")
        call = lambda q=q, cu=cu, n=n, out=out, lse=lse: psf.attn_cache_prompt_fwd(  # noqa: E731
            q, cache, t, n, 0.1, cu, 300, out=out, lse=lse, workspace=ws)
        want = [x.clone() for x in psf.attn_cache_prompt_fwd(q, cache, t, n, 0.1, cu, 300)]
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        calls.append((g, out, lse, want, call))  # (the call holds what the graph reads)
    for order in ([0, 1], [1, 0], [0, 0, 1, 1, 0]):
        for _, out, lse, _, _ in calls:
            out.fill_(7)
            lse.fill_(7)
        for i in order:
            calls[i][0].replay()
        torch.cuda.synchronize()
        for _, out, lse, want, _ in calls:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_many_runs_give_the_same_bits():
    """Capped and not, cut over shares: no order of execution shows in the results."""
    lens, m_rows, page = [9000, 700, 2000], [200, 300, 1], 16
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 2, 192, 128, page)
    q, n, cu = queries(501, 8, 192), i32(lens), i32(prefix(m_rows))
    for softcap in (None, 5.0):
        want = psf.attn_cache_prompt_fwd(q, cache, t, n, 0.1, cu, 300, softcap=softcap)
        for _ in range(20):
            got = psf.attn_cache_prompt_fwd(q, cache, t, n, 0.1, cu, 300, softcap=softcap)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_long_chunks_at_512_by_both_routes():
    """The gather with the varlen forward, which the documents name for them, gives what the call gives."""
    lens, m_rows, page = [1500, 300], [400, 300], 32
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 1, 512, 512, page)
    q, n, cu = queries(700, 4, 512), i32(lens), i32(prefix(m_rows))
    out, lse = psf.attn_cache_prompt_fwd(q, cache, t, n, 0.02, cu, 400)
    k, v, cu_k = psf.kv_cache_gather(cache, t, n, sum(lens))
    want, want_lse = psf.attn_varlen_fwd(q, k, v, cu, cu_k, 400, 1500, 0.02, True)
    # P sums to 1 and is rounded in both (fp16: 2^-11 of it, bf16: 2^-8), the results to bf16 (2^-8 each, and they are no larger
    # than the largest value): 2^-6 of that covers it.
    assert float((out.double() - want.double()).abs().max()) <= 2.0 ** -6 * float(v.abs().max())
    assert float((lse - want_lse).abs().max()) <= 1e-3  # the varlen forward's own bound
