"""GPU tests of the 8-bit paged cache against its definitions in 64 bits (cache_reference.py).

Append and eviction have to give the definition's codes, scales and weights
exactly; the attention's outputs lie within the roundings counted in
cache_reference.attend.
"""
import math
import random

import pytest
import torch

import cache_reference as ref
import packed_sequence_flash_gb300 as psf

pytestmark = pytest.mark.gpu

EDEVICE_ARGS = -4
DIMS = [(64, 64), (128, 128), (192, 128), (512, 512)]


@pytest.fixture(autouse=True)
def _clean_status():
    assert psf.device_status() == 0
    yield


def tables(lens, page, extra=0, seed=0, spare=3):
    """Disjoint pages in random order for sequences that may grow by `extra` tokens -> (list of lists, tensor, pages)."""
    r = random.Random(seed)
    need = [max(1, -(-(n + extra) // page)) for n in lens]
    ids = list(range(sum(need) + spare))
    r.shuffle(ids)
    rows, at = [], 0
    for k in need:
        rows.append(ids[at:at + k])
        at += k
    width = max(need)
    t = torch.tensor([x + [-1] * (width - len(x)) for x in rows], dtype=torch.int32, device="cuda")
    return rows, t, len(ids)


def random_cache(pages, H, Dqk, Dv, page, weights=False, seed=0, layout="hp"):
    """A cache of random codes and scales; layout "ph": memory order [pages, page, H, D]."""
    g = torch.Generator().manual_seed(seed)

    def codes(D):
        x = (torch.randn(pages, H, page, D, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        if layout == "ph":
            return x.transpose(1, 2).contiguous().cuda().transpose(1, 2).view(torch.float8_e4m3fn)
        return x.cuda().view(torch.float8_e4m3fn)

    scale = lambda: torch.exp2(torch.randint(-8, -3, (pages, H), generator=g).float()).cuda()  # noqa: E731
    w = None
    if weights:
        w = (torch.rand(pages, H, page, generator=g) ** 4).cuda()
    return psf.KVCache(codes(Dqk), codes(Dv), scale(), scale(), w)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prefix(rows):
    cu = [0]
    for m in rows:
        cu.append(cu[-1] + m)
    return cu


def check_attend(cache, q, rows, table_t, lens, m_rows, scale, accumulate=False, uniform=False, **kw):
    cu = prefix(m_rows)
    c = ref.from_cache(cache)
    got = psf.attn_cache_fwd(q, cache, table_t, i32(lens), scale, cu_q=None if uniform else i32(cu),
                             max_q=None if uniform else max(m_rows + [1]), accumulate=accumulate, **kw)
    torch.cuda.synchronize()
    assert psf.device_status() == 0
    want = ref.attend(c, q, rows, lens, cu, scale, accumulate=accumulate, **kw)
    close(got[0], want[0], want[2], "out")
    close(got[1], want[1], want[3], "lse")
    if accumulate:
        close(cache.weight, c["w"], want[4], "weight")
    return got


def close(got, want, tol, name):
    got = got.detach().cpu().double()
    assert torch.equal(got.isnan(), want.isnan()), f"{name}: NaN in other places"
    assert torch.equal(got.isneginf(), want.isneginf()), f"{name}: -inf in other places"
    fin = want.isfinite()
    over = ((got - want).abs() - tol)[fin]
    assert not over.numel() or float(over.max()) <= 0, f"{name}: off by {float((got - want).abs()[fin].max()):.3e}, " \
        f"{float(over.max()):.3e} more than allowed"


# ---------------------------------------------------------------------------
# attention

@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_one_token_per_sequence(dims, page, dtype):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000]
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 2, *dims, page)
    q = torch.randn(len(lens), 8, dims[0], generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    check_attend(cache, q, rows, t, lens, [1] * len(lens), dims[0] ** -0.5, uniform=True)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("G,H", [(1, 3), (2, 2), (5, 1), (8, 2), (16, 1), (20, 1)])
@pytest.mark.parametrize("m", [1, 3, 9])
def test_groups_and_rows(dims, G, H, m):
    lens = [2, 40, 200, 451]  # fewer tokens than rows in the first: its first rows see nothing
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, H, *dims, 32, seed=1)
    q = torch.randn(len(lens) * m, H * G, dims[0], generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, [m] * len(lens), dims[0] ** -0.5, uniform=True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [None, 1, 16, 100, 5000])
@pytest.mark.parametrize("softcap", [None, 2.0, 30.0])
def test_masks_and_cap_on_ragged_rows(causal, window, softcap):
    lens, m_rows = [90, 3, 700, 0, 64, 257], [1, 5, 40, 2, 0, 7]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 2, 128, 128, 16, seed=2)
    q = (2 * torch.randn(sum(m_rows), 6, 128, generator=torch.Generator().manual_seed(5))).half().cuda()
    check_attend(cache, q, rows, t, lens, m_rows, 0.1, causal=causal, window=window, softcap=softcap)


@pytest.mark.parametrize("dims", [(64, 64), (192, 128), (512, 512)])
@pytest.mark.parametrize("window", [None, 33])
def test_masks_on_other_head_dims(dims, window):
    lens, m_rows = [90, 3, 400, 0, 64], [1, 5, 20, 2, 0]
    rows, t, pages = tables(lens, 64)
    cache = random_cache(pages, 1, *dims, 64, seed=2)
    q = torch.randn(sum(m_rows), 4, dims[0], generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, m_rows, dims[0] ** -0.5, window=window)


@pytest.mark.parametrize("B,hi", [(1, 20000), (3, 9000), (200, 120)])
def test_long_and_many_sequences(B, hi):
    r = random.Random(B)
    lens = [hi] + [r.randint(0, hi) for _ in range(B - 1)]
    rows, t, pages = tables(lens, 64, seed=B)
    cache = random_cache(pages, 2, 128, 128, 64, seed=B)
    q = (3 * torch.randn(B, 8, 128, generator=torch.Generator().manual_seed(B))).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, [1] * B, 128 ** -0.5, uniform=True)


def test_more_sequences_than_a_block_has_threads():
    B = 1500
    lens = [(i * 7) % 40 for i in range(B)]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 1, 64, 64, 16)
    m_rows = [(i % 3) for i in range(B)]
    q = torch.randn(sum(m_rows), 1, 64, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, m_rows, 0.125)


@pytest.mark.parametrize("B,G,hi", [(700, 4, 60), (513, 2, 300), (1100, 1, 40)])
@pytest.mark.parametrize("softcap", [None, 5.0])
def test_more_units_than_shares(B, G, hi, softcap):
    """Sequences without keys, with few and with many among them, and rows past the last one."""
    r = random.Random(B)
    lens = [r.choice([0, 1, 20, hi, r.randint(0, hi)]) for _ in range(B)]
    lens[B // 2] = 4000
    m_rows = [r.choice([0, 1, 1, 2]) for _ in range(B)]
    m_rows[B // 2] = 1
    rows, t, pages = tables(lens, 16, seed=B)
    cache = random_cache(pages, 2, 64, 64, 16, seed=B, weights=True)
    cu = prefix(m_rows)
    q = torch.randn(cu[-1] + 9, 2 * G, 64, generator=torch.Generator().manual_seed(B)).bfloat16().cuda()
    out = torch.full_like(q, 3.0)
    c = ref.from_cache(cache)
    got = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.2, cu_q=i32(cu), max_q=2, softcap=softcap, out=out,
                             accumulate=True)
    assert psf.device_status() == 0
    want = ref.attend(c, q, rows, lens, cu, 0.2, softcap=softcap, accumulate=True)
    close(got[0], want[0], want[2], "out")
    close(got[1], want[1], want[3], "lse")
    close(cache.weight, c["w"], want[4], "weight")


@pytest.mark.parametrize("G,m", [(4, 1), (1, 1), (8, 5), (3, 2)])
@pytest.mark.parametrize("window", [None, 50])
def test_accumulated_weights(G, m, window):
    lens = [1, 64, 0, 333, 2500, 130]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 2, 128, 128, 32, weights=True, seed=4)
    q = (2 * torch.randn(len(lens) * m, 2 * G, 128, generator=torch.Generator().manual_seed(7))).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, [m] * len(lens), 128 ** -0.5, accumulate=True, uniform=True, window=window)


@pytest.mark.parametrize("dims", [(64, 64), (192, 128), (512, 512)])
def test_accumulated_weights_other_head_dims(dims):
    lens, m_rows = [70, 5, 200], [2, 3, 1]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 2, *dims, 16, weights=True, seed=4)
    q = torch.randn(6, 6, dims[0], generator=torch.Generator().manual_seed(7)).half().cuda()
    check_attend(cache, q, rows, t, lens, m_rows, dims[0] ** -0.5, accumulate=True)


def test_scales_far_apart():
    """Blocks whose V scales differ by 2^40, the large ones with next to no probability and the other way round."""
    lens = [640]
    rows, t, pages = tables(lens, 64)
    cache = random_cache(pages, 1, 128, 128, 64)
    for i, pg in enumerate(rows[0]):
        cache.v_scale[pg, 0] = 2.0 ** (-20 if i % 2 else 20)
        cache.k_scale[pg, 0] = 2.0 ** (-4 if i % 2 else -9)
    q = (4 * torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(8))).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, [1], 0.3, uniform=True)


def test_large_and_tiny_queries():
    lens = [200, 200, 200, 200]
    rows, t, pages = tables(lens, 64)
    cache = random_cache(pages, 1, 128, 128, 64)
    q = torch.randn(4, 4, 128, generator=torch.Generator().manual_seed(8))
    q = (q * torch.tensor([1e30, 1e-30, 0.0, 1.0])[:, None, None]).bfloat16().cuda()
    cache.k_scale[rows[0]] = 2.0 ** -100
    cache.k_scale[rows[1]] = 2.0 ** 100
    check_attend(cache, q, rows, t, lens, [1] * 4, 128 ** -0.5, uniform=True)


def poison(cache, rows, lens):
    """NaN in every code and scale that no sequence has a token in."""
    for name in ("k", "v"):
        raw = getattr(cache, name).view(torch.uint8)
        used = torch.zeros(raw.shape[:3], dtype=torch.bool)
        for row, n in zip(rows, lens):
            for p, pg in enumerate(row):
                used[pg, :, :max(0, min(cache.page_size, n - p * cache.page_size))] = True
        raw.masked_fill_(~used.cuda()[..., None], 0x7F)
        getattr(cache, name + "_scale").masked_fill_(~used.any(2).cuda(), math.nan)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 128])
def test_stale_rows_and_pages_are_not_seen(dims, page):
    lens = [1, 50, 130, 0, 191]
    rows, t, pages = tables(lens, page, extra=page)
    cache = random_cache(pages, 2, *dims, page, seed=9)
    poison(cache, rows, lens)
    q = torch.randn(10, 4, dims[0], generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, [2] * 5, dims[0] ** -0.5, uniform=True)


@pytest.mark.parametrize("dims", DIMS)
def test_nan_codes_reach_only_the_rows_that_see_them(dims):
    lens = [150]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 1, *dims, 32, seed=10)
    raw = cache.v.view(torch.uint8)
    raw[rows[0][149 // 32], 0, 149 % 32, 3] = 0x7F  # the last token: seen by the last row only
    raw[rows[0][20 // 32], 0, 20 % 32, 5] = 0xFF    # out of every row's window
    cache.k.view(torch.uint8)[rows[0][148 // 32], 0, 148 % 32, 1] = 0x7F  # seen by the last two rows
    q = torch.randn(4, 2, dims[0], generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    out, lse = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, window=100)
    assert out[2:].isnan().all() and lse[:, 2:].isnan().all()
    assert out[:2].isfinite().all() and lse[:, :2].isfinite().all()
    cache.k.view(torch.uint8)[rows[0][148 // 32], 0, 148 % 32, 1] = 0
    out, lse = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, window=100)
    assert lse.isfinite().all() and out[:3].isfinite().all()
    nan = out[3].isnan()
    assert nan[:, 3].all() and int(nan.sum()) == 2


@pytest.mark.parametrize("dims", DIMS)
def test_nan_codes_in_a_tile_of_sixteen_rows(dims):
    lens, G = [150], 4
    rows, t, pages = tables(lens, 64)
    cache = random_cache(pages, 1, *dims, 64, seed=10)
    raw = cache.v.view(torch.uint8)
    raw[rows[0][2], 0, 149 % 64, 7] = 0x7F  # seen by the last token's rows only
    raw[rows[0][2], 0, 148 % 64, 9] = 0xFF  # by the last two tokens'
    q = torch.randn(4, G, dims[0], generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    out, lse = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1)
    assert lse.isfinite().all() and out[:2].isfinite().all()
    nan = out.isnan()
    assert nan[2, :, 9].all() and int(nan[2].sum()) == G
    assert nan[3, :, 7].all() and nan[3, :, 9].all() and int(nan[3].sum()) == 2 * G


def test_windows_as_long_as_numbers_go():
    lens, m_rows = [5, 300, 40], [9, 2, 40]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 1, 64, 64, 16)
    q = torch.randn(sum(m_rows), 2, 64, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    for window in (2 ** 31 - 1, t.shape[1] * 16, t.shape[1] * 16 - 1):
        check_attend(cache, q, rows, t, lens, m_rows, 0.1, window=window)


def test_strided_cache_and_rows_with_guard_bands():
    lens, m_rows = [33, 200, 7], [2, 1, 4]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 2, 192, 128, 32, layout="ph")
    assert not cache.k.is_contiguous()
    fused = torch.randn(7, 6 * 192 + 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q = fused[:, 32:32 + 6 * 192].unflatten(1, (6, 192))
    buf = torch.full((7 + 2, 8, 128 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:8, 1:7, 8:136]
    lse_buf = torch.full((6 * 7 + 64,), 7.0, device="cuda")
    lse = lse_buf[32:32 + 42].view(6, 7)
    c = ref.from_cache(cache)
    psf.attn_cache_fwd(q, cache, t, i32(lens), 192 ** -0.5, cu_q=i32(prefix(m_rows)), max_q=4, out=out, lse=lse)
    want = ref.attend(c, q, rows, lens, prefix(m_rows), 192 ** -0.5)
    close(out, want[0], want[2], "out")
    close(lse, want[1], want[3], "lse")
    out.fill_(7.0)
    lse.fill_(7.0)
    assert bool((buf == 7.0).all()) and bool((lse_buf == 7.0).all())


def test_rows_past_the_last_sequence_are_zero():
    lens = [40, 9]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 1, 64, 64, 16)
    q = torch.randn(7, 2, 64).bfloat16().cuda()
    out = torch.full((7, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out, lse = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.125, cu_q=i32([0, 1, 3]), max_q=2, out=out)
    assert not out[3:].any() and bool(lse[:, 3:].isneginf().all()) and bool(lse[:, :3].isfinite().all())
    # no rows at all
    out, lse = psf.attn_cache_fwd(q[:0], cache, t, i32(lens), 0.125)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)


def test_shared_pages_and_a_page_twice():
    cache = random_cache(6, 2, 128, 128, 16, weights=True)
    rows = [[2, 4, 1], [2, 4, 5], [3, 3, 3]]
    t = i32(rows)
    lens = [40, 48, 45]
    q = torch.randn(3, 4, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    check_attend(cache, q, rows, t, lens, [1] * 3, 0.09, accumulate=True, uniform=True)


def test_offsets_past_32_bits():
    """K and V of 4.8 GB each, tokens at their far end."""
    page, H, D = 64, 8, 128
    pages = 73000
    k = torch.zeros(pages, H, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros(pages, H, page, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    small = random_cache(4, H, D, D, page, weights=True, seed=3)
    ks = torch.ones(pages, H, device="cuda")
    cache = psf.KVCache(k, v, ks, ks.clone(), torch.zeros(pages, H, page, device="cuda"))
    far = [72999, 70001, 66000, 40000]
    for name in ("k", "v"):
        getattr(cache, name).view(torch.uint8)[far] = getattr(small, name).view(torch.uint8)
        getattr(cache, name + "_scale")[far] = getattr(small, name + "_scale")
    lens = [250]
    q = torch.randn(1, 16, D, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    a = psf.attn_cache_fwd(q, cache, i32([far]), i32(lens), 0.09, accumulate=True)
    b = psf.attn_cache_fwd(q, small, i32([[0, 1, 2, 3]]), i32(lens), 0.09)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    kk, vv, cu = psf.kv_cache_gather(cache, i32([far]), i32(lens), 250)
    k2, v2, _ = psf.kv_cache_gather(small, i32([[0, 1, 2, 3]]), i32(lens), 250)
    assert torch.equal(kk, k2) and torch.equal(vv, v2)
    new = psf.kv_cache_evict(cache, i32([far]), i32(lens), 100, 10)
    assert new.tolist() == [100]
    assert float(cache.weight[far[0]].sum()) > 0
    x = torch.randn(1, H, D).bfloat16().cuda()
    psf.kv_cache_append(cache, x, x, i32([far]), i32([101]))
    got = psf.kv_cache_gather(cache, i32([far]), i32([101]), 101)[0][100]
    assert float((got.double() - x[0].double()).abs().max()) <= float(x.abs().max()) * 2.0 ** -4 + 2.0 ** -8
    assert psf.device_status() == 0


def test_results_do_not_depend_on_the_run():
    lens = [5000, 77, 1200, 0, 64]
    rows, t, pages = tables(lens, 64)
    cache = random_cache(pages, 4, 128, 128, 64, weights=True)
    q = torch.randn(10, 16, 128).bfloat16().cuda()
    w0 = cache.weight.clone()
    a = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, accumulate=True)
    w1 = cache.weight.clone()
    for _ in range(3):
        cache.weight.copy_(w0)
        ws = torch.randint(0, 255, (psf.attn_cache_workspace_size(cache, 5, t.shape[1], 16, 2, True),),
                           dtype=torch.uint8, device="cuda")
        b = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, accumulate=True, workspace=ws)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(cache.weight, w1)


def test_graphs_share_a_workspace_and_follow_the_lengths():
    lens = [300, 40, 129]
    rows, t, pages = tables(lens, 32, extra=300)
    cache = random_cache(pages, 2, 128, 128, 32)
    q = torch.randn(3, 8, 128).bfloat16().cuda()
    n = i32(lens)
    ws = torch.empty(psf.attn_cache_workspace_size(cache, 3, t.shape[1], 8), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 3, device="cuda")) for _ in range(2)]
    scales = [0.1, 0.2]

    def call(i):
        psf.attn_cache_fwd(q, cache, t, n, scales[i], out=outs[i][0], lse=outs[i][1], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for i in range(2):
            call(i)
        side.synchronize()
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call(i)
            graphs.append(g)
    torch.cuda.synchronize()
    for step in range(3):
        now = [x + 150 * step - step * step for x in lens]
        n.copy_(i32(now))
        for i in (0, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            want = ref.attend(ref.from_cache(cache), q, rows, now, [0, 1, 2, 3], scales[i])
            close(outs[i][0], want[0], want[2], "out")
            close(outs[i][1], want[1], want[3], "lse")


def decode(cache, t, n, data, sync):
    """Steps of a decode loop on the current stream, nothing between the calls unless sync."""
    outs = []
    for i, (k, v, q) in enumerate(data):
        n += 1
        psf.kv_cache_append(cache, k, v, t, n)
        if sync:
            torch.cuda.synchronize()
        outs += psf.attn_cache_fwd(q, cache, t, n, 0.09, accumulate=i % 2 == 0)
        if sync:
            torch.cuda.synchronize()
        if i % 7 == 6:
            n.copy_(psf.kv_cache_evict(cache, t, n, 900, 100))
        if i % 5 == 4:
            outs += psf.kv_cache_gather(cache, t, n, 4 * 1100)[2:]
        if sync:
            torch.cuda.synchronize()
    torch.cuda.synchronize()
    return outs


def test_calls_one_after_another_without_waiting():
    """Kernels that begin before the one in front is over must not read what it has yet to write."""
    lens = [905, 60, 1, 890]
    rows, t, pages = tables(lens, 32, extra=60)
    data = [(torch.randn(4, 2, 128).bfloat16().cuda(), torch.randn(4, 2, 128).bfloat16().cuda(),
             torch.randn(4, 8, 128).bfloat16().cuda()) for _ in range(30)]
    runs = []
    for sync in (True, False, False):
        cache = random_cache(pages, 2, 128, 128, 32, weights=True, seed=5)
        n = i32(lens)
        runs.append(decode(cache, t, n, data, sync) + [cache.k.view(torch.uint8), cache.v.view(torch.uint8),
                                                       cache.k_scale, cache.v_scale, cache.weight, n])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_a_captured_decode_step():
    """Length, append and attention in one graph, between a fill and a copy, replayed while the sequences grow."""
    lens = [31, 300, 0]
    rows, t, pages = tables(lens, 32, extra=20)
    k, v = (torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    n = i32(lens)
    cache = random_cache(pages, 2, 64, 64, 32, weights=True, seed=6)
    copy = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty(1024, device="cuda")

    def step():
        scratch.fill_(1.0)
        n.add_(1)
        psf.kv_cache_append(cache, k, v, t, n)
        out, lse = psf.attn_cache_fwd(q, cache, t, n, 0.125, accumulate=True)
        copy.copy_(out)
        return out, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = random_cache(pages, 2, 64, 64, 32, weights=True, seed=6)
        psf.kv_cache_append(warm, k, v, t, i32([x + 1 for x in lens]))
        psf.attn_cache_fwd(q, warm, t, i32([x + 1 for x in lens]), 0.125, accumulate=True)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = step()
    torch.cuda.synchronize()
    n.copy_(i32(lens))
    c = ref.from_cache(cache)
    g = torch.Generator().manual_seed(3)
    for _ in range(12):
        lens = [x + 1 for x in lens]
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g).bfloat16())
        ref.append(c, k, v, rows, lens, [0, 1, 2, 3])
        want = ref.attend(c, q, rows, lens, [0, 1, 2, 3], 0.125, accumulate=True)
        graph.replay()
        torch.cuda.synchronize()
        assert n.tolist() == lens
        close(out, want[0], want[2], "out")
        close(lse, want[1], want[3], "lse")
        assert torch.equal(copy, out)
        close(cache.weight, c["w"], want[4], "weight")
        c["w"] = cache.weight.cpu().double()
        same(cache, c)


def test_two_streams_at_once():
    lens = [4000, 2500, 900]
    rows, t, pages = tables(lens, 64)
    cache = random_cache(pages, 4, 128, 128, 64)
    n = i32(lens)
    qs = [torch.randn(3, 16, 128).bfloat16().cuda() for _ in range(2)]
    alone = [psf.attn_cache_fwd(q, cache, t, n, 0.1) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(psf.attn_cache_fwd(qs[i], cache, t, n, 0.1))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(l, alone[i][1])


@pytest.mark.parametrize("fault", ["page too large", "page negative", "length past the table", "length negative",
                                   "too many rows", "rows past the tensor"])
def test_device_checks_leave_the_other_sequences_alone(fault):
    lens, m_rows = [100, 70, 33], [1, 2, 1]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 2, 128, 128, 32, weights=True)
    q = torch.randn(4, 4, 128).bfloat16().cuda()
    good = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, cu_q=i32([0, 1, 3, 4]), max_q=2)
    bad_t, bad_n, cu = t.clone(), i32(lens), i32([0, 1, 3, 4])
    if fault == "page too large":
        bad_t[1, 1] = pages
    elif fault == "page negative":
        bad_t[1, 0] = -1
    elif fault == "length past the table":
        bad_n[1] = t.shape[1] * 32 + 1
    elif fault == "length negative":
        bad_n[1] = -5
    elif fault == "too many rows":
        cu = i32([0, 1, 1, 4])
    else:
        cu = i32([0, 1, 3, 5])
    out, lse = psf.attn_cache_fwd(q, cache, bad_t, bad_n, 0.1, cu_q=cu, max_q=2)
    assert psf.device_status() == EDEVICE_ARGS
    same = [0] if fault in ("too many rows", "rows past the tensor") else [0, 3]
    assert torch.equal(out[same], good[0][same]) and torch.equal(lse[:, same], good[1][:, same])
    if fault in ("too many rows", "rows past the tensor"):
        return
    # the calls that write: sequence 1 is left as it is, the others are done
    before = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.weight)]
    x = torch.randn(3, 2, 128).bfloat16().cuda()
    psf.kv_cache_append(cache, x, x, bad_t, bad_n)
    status = psf.device_status()
    if fault != "page negative":  # that page holds older tokens, the new one goes elsewhere
        if fault == "page too large":
            assert status == 0  # token 69 is in page 2
        else:
            assert status == EDEVICE_ARGS
            assert torch.equal(cache.k.view(torch.uint8)[rows[1]], before[0][rows[1]])
    for b in (0, 2):
        assert not torch.equal(cache.k.view(torch.uint8)[rows[b]], before[0][rows[b]])
    state = [x.clone() for x in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.weight)]
    new = psf.kv_cache_evict(cache, bad_t, bad_n, 30, 4)
    assert psf.device_status() == EDEVICE_ARGS
    assert new.tolist() == [30, int(bad_n[1]), 30]
    for a, z in zip((cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.weight), state):
        assert torch.equal(a[rows[1]], z[rows[1]])
    psf.kv_cache_gather(cache, bad_t, bad_n, 203)
    assert psf.device_status() == EDEVICE_ARGS


@pytest.mark.parametrize("cu", [[3, 5, 9], [0, 5, 2], [0, 5, 400], [0, -1, 4], [-40, 2, 4], [1000, 1001, 1002]])
def test_prefix_sums_that_cannot_be(cu):
    lens = [40, 30]
    rows, t, pages = tables(lens, 16, extra=16)
    cache = random_cache(pages, 1, 64, 64, 16)
    q = torch.randn(9, 2, 64).bfloat16().cuda()
    psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, cu_q=i32(cu), max_q=9)
    assert psf.device_status() == EDEVICE_ARGS
    before = cache.k.view(torch.uint8).clone()
    owned = torch.zeros(pages, dtype=torch.bool, device="cuda")
    owned[[pg for r in rows for pg in r]] = True
    x = torch.randn(9, 1, 64).bfloat16().cuda()
    psf.kv_cache_append(cache, x, x, t, i32(lens), cu_new=i32(cu))
    assert psf.device_status() == EDEVICE_ARGS
    assert torch.equal(cache.k.view(torch.uint8)[~owned], before[~owned])


@pytest.mark.parametrize("cu,each", [(None, 1), (None, 3), ([0, 3, 4, 6], 0)])
def test_more_new_rows_than_tokens(cu, each):
    """Such a sequence takes none and says so; the others take theirs. An idle entry without rows is fine."""
    lens = [0, 30, 2] if each != 3 else [2, 30, 0]
    rows, t, pages = tables([16, 30, 16], 16)
    cache = random_cache(pages, 2, 64, 64, 16)
    c = ref.from_cache(cache)
    x = torch.randn(3 * each or 6, 2, 64, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    psf.kv_cache_append(cache, x, x, t, i32(lens), None if cu is None else i32(cu))
    assert psf.device_status() == EDEVICE_ARGS
    at = prefix([each] * 3) if cu is None else cu
    for b in (1, 2) if each != 3 else (1,):
        ref.append(c, x, x, [[], [], []][:b] + [rows[b]], [0] * b + [lens[b]], [at[b]] * (b + 1) + [at[b + 1]])
    same(cache, c)
    psf.kv_cache_append(cache, x[:3], x[:3], t, i32([14, 0, 5]), i32([0, 2, 2, 3]))
    assert psf.device_status() == 0
    ref.append(c, x[:3], x[:3], rows, [14, 0, 5], [0, 2, 2, 3])
    same(cache, c)


def test_numbers_of_other_kinds():
    import numpy as np

    lens = [20, 30]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 1, 64, 64, 16, weights=True)
    q = torch.randn(3, 2, 64).bfloat16().cuda()
    a = psf.attn_cache_fwd(q, cache, t, i32(lens), np.float64(0.1), cu_q=i32([0, 1, 3]), max_q=np.int64(2))
    b = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, cu_q=i32([0, 1, 3]), max_q=7)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert psf.kv_cache_gather(cache, t, i32(lens), np.int32(50))[0].shape == (50, 1, 64)
    assert psf.kv_cache_evict(cache, t, i32(lens), np.int64(25), np.int64(3)).tolist() == [20, 25]


# ---------------------------------------------------------------------------
# append

def check_append(cache, k, v, rows, t, lens, new, uniform=False):
    c = ref.from_cache(cache)
    psf.kv_cache_append(cache, k, v, t, i32(lens), None if uniform else i32(prefix(new)))
    torch.cuda.synchronize()
    assert psf.device_status() == 0
    ref.append(c, k, v, rows, lens, prefix(new))
    same(cache, c)


def same(cache, c):
    for name, want in (("k", c["k"]), ("v", c["v"]), ("k_scale", c["ks"]), ("v_scale", c["vs"]), ("weight", c["w"])):
        t = getattr(cache, name)
        if t is not None:
            got = t.cpu().double()
            ok = (got == want) | (got.isnan() & want.isnan())
            assert bool(ok.all()), f"{name}: {int((~ok).sum())} of {ok.numel()} differ, first {(~ok).nonzero()[0].tolist()}"


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_prompts(dims, page, dtype):
    before, new = [0, 5, 16, 130, 0, 64], [1, 300, 16, 0, 129, 63]
    lens = [a + b for a, b in zip(before, new)]
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 2, *dims, page, weights=True)
    g = torch.Generator().manual_seed(1)
    k = (torch.randn(sum(new), 2, dims[0], generator=g) * torch.exp2(torch.randint(-6, 7, (sum(new), 1, 1), generator=g))).to(dtype).cuda()
    v = torch.randn(sum(new), 2, dims[1], generator=g).to(dtype).cuda()
    check_append(cache, k, v, rows, t, lens, new)


@pytest.mark.parametrize("page", [16, 64])
def test_append_token_by_token(page):
    """Scales that grow, page ends that are crossed; a page taken over from another sequence starts afresh."""
    lens = [0, 10, page - 1, 3]
    rows, t, pages = tables(lens, page, extra=page + 8)
    cache = random_cache(pages, 2, 128, 128, page, weights=True)
    g = torch.Generator().manual_seed(2)
    for step in range(page + 4):
        lens = [n + 1 for n in lens]
        x = (torch.randn(4, 2, 128, generator=g) * 2.0 ** (step % 9 - 4)).bfloat16().cuda()
        y = (torch.randn(4, 2, 128, generator=g) * 2.0 ** (step / 4)).bfloat16().cuda()
        check_append(cache, x, y, rows, t, lens, [1] * 4, uniform=True)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_one_token_to_every_sequence(dims, dtype):
    """Growing and shrinking rows, values that are not finite, rows at page ends, scales that are no powers of two."""
    lens = [1, 17, 32, 33, 64, 5, 40, 2, 31]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 3, *dims, 32, weights=True)
    cache.k_scale.mul_(1.3)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 3, dims[0], generator=g) * torch.exp2(torch.randint(-9, 12, (9, 3, 1), generator=g))
    y = torch.randn(9, 3, dims[1], generator=g) * torch.exp2(torch.randint(-9, 12, (9, 3, 1), generator=g))
    x[1, 0, 3], x[2, 1, 0], x[4, 2] = math.inf, math.nan, 0.0
    y[3, 0], y[5, 1, 7] = math.nan, -math.inf
    k = x.to(dtype).cuda()
    fused = torch.zeros(9, 3, 2 * dims[1], dtype=dtype, device="cuda")
    v = fused[:, :, dims[1]:]
    v.copy_(y.to(dtype))
    check_append(cache, k, v, rows, t, lens, [1] * 9, uniform=True)
    # the same rows through prefix sums (a page at a time) give the same cache
    other = random_cache(pages, 3, *dims, 32, weights=True)
    other.k_scale.mul_(1.3)
    psf.kv_cache_append(other, k, v, t, i32(lens), i32(list(range(10))))
    for name in ("k", "v", "k_scale", "v_scale", "weight"):
        a, b = getattr(cache, name), getattr(other, name)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append_values_at_the_borders():
    lens = [16 * 8]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 1, 64, 64, 16)
    k = torch.zeros(128, 1, 64)
    k[0:16] = 448.0                     # exactly the largest code
    k[16:32] = 449.0                    # bf16 has no 449: 448
    k[32:48] = 450.0                    # just above: the next scale
    k[48:64] = 0.0
    k[64:80] = 1e-38                    # the smallest scale
    k[64, 0, 0] = 3e38
    k[80, 0, 3] = math.inf
    k[81, 0, 4] = -math.inf
    k[82, 0, 5] = math.nan
    k[83] = 17.0
    k[96:112] = torch.linspace(-448, 448, 64)  # ties of the rounding among them
    k[112:128] = 1e-40
    check_append(cache, k.bfloat16().cuda(), (k / 7).bfloat16().cuda(), rows, t, lens, [128])


def test_append_strided_rows_and_cache():
    before, new = [3, 0], [20, 40]
    lens = [23, 40]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 2, 128, 128, 16, layout="ph")
    fused = torch.randn(60, 2 * 3 * 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    kv = fused.unflatten(1, (2, 3, 128))
    check_append(cache, kv[:, :, 1], kv[:, :, 2], rows, t, lens, new)


# ---------------------------------------------------------------------------
# eviction

def check_evict(cache, rows, t, lens, budget, recent):
    c = ref.from_cache(cache)
    got = psf.kv_cache_evict(cache, t, i32(lens), budget, recent)
    torch.cuda.synchronize()
    assert psf.device_status() == 0
    assert got.tolist() == ref.evict(c, rows, lens, budget, recent)
    same(cache, c)


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("budget,recent", [(100, 20), (1, 0), (1, 1), (64, 64), (33, 0), (129, 128)])
def test_evict(dims, page, budget, recent):
    lens = [300, budget, budget + 1, 0, 1, 170]
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 2, *dims, page, weights=True, seed=budget)
    check_evict(cache, rows, t, lens, budget, recent)


def test_evict_ties_and_odd_weights():
    lens = [500, 400]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 2, 64, 64, 32, weights=True)
    cache.weight.copy_(torch.randint(0, 3, cache.weight.shape).float())
    cache.weight[rows[0][0], 0, :4] = torch.tensor([math.nan, math.inf, -0.0, -1.0])
    cache.weight[rows[1]] = 0.0
    check_evict(cache, rows, t, lens, 150, 10)


def test_evict_scales_that_are_no_powers_of_two():
    """Ratios that fp32 rounds (17/16 over 3/2), ones whose products are ties (1/2, 13/16), and a zero scale."""
    lens = [150, 90, 300]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 2, 128, 128, 16, weights=True)
    g = torch.Generator().manual_seed(9)
    scales = torch.tensor([17 / 16, 3 / 2, 1.3, 0.65, 1.0, 0.5, 13 / 16, 0.0, 1.7, 1e-3])
    for x in (cache.k_scale, cache.v_scale):
        x.copy_(scales[torch.randint(0, len(scales), x.shape, generator=g)])
    check_evict(cache, rows, t, lens, 80, 20)


def test_evict_sequence_longer_than_shared_memory_holds():
    n = 50000
    rows, t, pages = tables([n, 200], 128)
    cache = random_cache(pages, 1, 64, 64, 128, weights=True)
    w = cache.weight.cpu()
    table = torch.tensor(rows[0])
    j = torch.arange(n)
    flat = w[table[j // 128], 0, j % 128]
    budget, recent = 3001, 500
    best = torch.argsort(-flat[:n - recent].double(), stable=True)[:budget - recent]
    kept = torch.cat([best.sort().values, j[n - recent:]])
    value = lambda: (cache.k.cpu().float() * cache.k_scale.cpu()[:, :, None, None])[table[j // 128], 0, j % 128]  # noqa: E731
    before = value()[kept]
    assert psf.kv_cache_evict(cache, t, i32([n, 200]), budget, recent).tolist() == [budget, 200]
    assert torch.equal(cache.weight.cpu()[table[j // 128], 0, j % 128][:budget], flat[kept])
    # a code is off by half a step of its new block's scale at most: 2^-4 relative, or 2^-10 of the scale
    after = value()[:budget]
    s = cache.k_scale.cpu()[table[j // 128], 0][:budget, None]
    assert bool(((after - before).abs() <= before.abs() * 2.0 ** -4 + s * 2.0 ** -10).all())


# ---------------------------------------------------------------------------
# gather, and the operators together

@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_gather(dims, page, dtype):
    lens = [3, 0, 128, 300, 0, 17]
    rows, t, pages = tables(lens, page)
    cache = random_cache(pages, 2, *dims, page)
    total = sum(lens) + 5
    c = ref.from_cache(cache)
    k, v, cu = psf.kv_cache_gather(cache, t, i32(lens), total, dtype=dtype)
    assert cu.tolist() == prefix(lens) and psf.device_status() == 0
    for b, n in enumerate(lens):
        for h in range(2):
            for name, x in (("k", k), ("v", v)):
                want = ref.rows_of(c, name, rows[b], n, h)
                assert torch.equal(x[cu[b]:cu[b + 1], h].cpu().double(), want.to(dtype).double())


def test_gather_with_too_little_room():
    lens = [30, 40]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 1, 64, 64, 16)
    full, _, _ = psf.kv_cache_gather(cache, t, i32(lens), 70)
    part, _, cu = psf.kv_cache_gather(cache, t, i32(lens), 41)
    assert psf.device_status() == EDEVICE_ARGS
    assert torch.equal(part, full[:41]) and cu.tolist() == [0, 30, 70]


@pytest.mark.parametrize("dims", DIMS)
def test_prompt_chunk_by_gather_and_by_cache(dims):
    """A chunk of query rows over its cached prefix: the packed forward on gathered rows, and the cache attention."""
    lens, m_rows = [200, 77, 40], [50, 77, 9]
    rows, t, pages = tables(lens, 64)
    cache = random_cache(pages, 2, *dims, 64)
    cu = prefix(m_rows)
    q = torch.randn(cu[-1], 4, dims[0], generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    scale = dims[0] ** -0.5 / 4
    k, v, cu_k = psf.kv_cache_gather(cache, t, i32(lens), sum(lens))
    out, lse = psf.attn_varlen_fwd(q, k, v, i32(cu), cu_k, max(m_rows), -1, scale, True)
    got = check_attend(cache, q, rows, t, lens, m_rows, scale)
    assert float((out.float() - got[0].float()).abs().max()) <= 2e-2 * float(out.float().abs().max())
    assert float((lse - got[1]).abs().max()) <= 1e-3


def test_a_serving_run():
    """Prompts in, tokens decoded with weights accumulated, eviction, further tokens: as one user's program."""
    H, G, D, page = 2, 4, 128, 16
    before = [0, 0, 0]
    new = [70, 3, 41]
    rows, t, pages = tables([130] * 3, page)
    cache = psf.kv_cache(pages, H, D, D, page_size=page, weights=True)
    c = ref.from_cache(cache)
    g = torch.Generator().manual_seed(11)
    draw = lambda T, h: torch.randn(T, h, D, generator=g).bfloat16().cuda()  # noqa: E731
    k, v = draw(sum(new), H), draw(sum(new), H)
    lens = [a + b for a, b in zip(before, new)]
    n = i32(lens)
    psf.kv_cache_append(cache, k, v, t, n, i32(prefix(new)))
    ref.append(c, k, v, rows, lens, prefix(new))
    one = [0, 1, 2, 3]
    tol = torch.zeros_like(c["w"])
    for step in range(24):
        lens = [x + 1 for x in lens]
        n += 1
        k, v, q = draw(3, H), draw(3, H), draw(3, H * G) * 3
        psf.kv_cache_append(cache, k, v, t, n)
        ref.append(c, k, v, rows, lens, one)
        out, lse = psf.attn_cache_fwd(q, cache, t, n, D ** -0.5, accumulate=True)
        want = ref.attend(c, q, rows, lens, one, D ** -0.5, accumulate=True)
        close(out, want[0], want[2], "out")
        close(lse, want[1], want[3], "lse")
        tol += want[4]
        close(cache.weight, c["w"], tol, "weight")
        c["w"] = cache.weight.cpu().double()  # so that near ties are cut the same way
        tol.zero_()
        if step in (9, 19):
            n = psf.kv_cache_evict(cache, t, n, 32, 8)
            lens = ref.evict(c, rows, lens, 32, 8)
            assert n.tolist() == lens
        same(cache, c)
    assert psf.device_status() == 0
