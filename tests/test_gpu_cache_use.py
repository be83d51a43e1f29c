"""GPU tests of the 8-bit cache: what a program may do with its tensors between calls, and less usual forms."""
import random

import pytest
import torch

import cache_reference as ref
import packed_sequence_flash_gb300 as psf
from test_gpu_cache import check_append, check_attend, check_evict, close, i32, prefix, random_cache, same, tables

pytestmark = pytest.mark.gpu

EDEVICE_ARGS = -4


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


def capped(c, q, row, n, scale, cap):
    """lse, out and weights of one query row per sequence over its n keys, in 64 bits, and how far a kernel may be off:
    as in cache_reference.attend, but with the cap's own roundings counted relative to the logit: tanh from its series
    (below 1/4: six roundings and the next term) or, from there on, off by 2^-21.8 at most where it is 0.245 or more, so
    20 u32 of the value, and four further products."""
    G, D = q.shape
    K, V = ref.rows_of(c, "k", row, n, 0), ref.rows_of(c, "v", row, n, 0)
    x = q.cpu().double()
    z0 = scale * (x @ K.T)
    z = cap * torch.tanh(z0 / cap)
    dz = ((D + 8) * (scale * (x.abs() @ K.abs().T)) + 24 * z.abs()) * ref.U32
    l = torch.logsumexp(z, -1)
    p = torch.exp(z - l[:, None])
    rel = (2 * dz.amax(-1) + 2.0 ** -21 + 4 * ref.U32 * (z.abs().amax(-1) + l.abs()) + n * ref.U32)[:, None]
    o, mass = p @ V, p @ V.abs()
    out_tol = ((rel + 2.0 ** -11) * mass + 2.0 ** -32 * n * V.abs().max() + ref.U16[q.dtype] * o.abs()) * 1.01 + 2.0 ** -24
    return l, rel[:, 0] + 4 * ref.U32 * l.abs(), o, out_tol, p.sum(0), (p * rel).sum(0) + G * ref.U32 + 8 * ref.U32 * p.sum(0)


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (192, 128), (512, 512)])
@pytest.mark.parametrize("G", [4, 12])
@pytest.mark.parametrize("cap", [0.5, 4.0, 9.0, 30.0, 1e3, 1e4, 1e6, 1e8, 1e20, 3e38])
def test_caps_near_and_far_above_the_logits(dims, G, cap):
    """The cap's error is relative to the logit: a cap far above all of them is next to none."""
    n = 300
    rows, t, pages = tables([n], 32)
    cache = random_cache(pages, 1, *dims, 32, seed=2, weights=True)
    cache.weight.zero_()
    q = (2 * torch.randn(1, G, dims[0], generator=torch.Generator().manual_seed(5))).half().cuda()
    c = ref.from_cache(cache)
    out, lse = psf.attn_cache_fwd(q, cache, t, i32([n]), 0.1, softcap=cap, accumulate=True)
    assert psf.device_status() == 0
    l, l_tol, o, o_tol, w, w_tol = capped(c, q[0], rows[0], n, 0.1, cap)
    close(lse[:, 0], l, l_tol, "lse")
    close(out[0], o, o_tol, "out")
    j = torch.arange(n)
    close(cache.weight[:, 0][torch.tensor(rows[0])[j // 32], j % 32], w, w_tol, "weight")


@pytest.mark.parametrize("cap", [1e-45, 1e-38, 1e-30])
def test_caps_that_leave_no_difference(cap):
    lens = [64, 100]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 1, 64, 64, 16)
    q = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    q[0, 1] = 0.0
    out, lse = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, softcap=cap)
    for b, n in enumerate(lens):
        l, l_tol, o, o_tol, _, _ = capped(ref.from_cache(cache), q[b], rows[b], n, 0.1, cap)
        close(lse[:, b], l, l_tol, "lse")
        close(out[b], o, o_tol, "out")


# ---------------------------------------------------------------------------
# wrong descriptions

def state(cache):
    return dict(k=cache.k.view(torch.uint8).clone(), v=cache.v.view(torch.uint8).clone(), k_scale=cache.k_scale.clone(),
                v_scale=cache.v_scale.clone(), weight=cache.weight.clone())


def unchanged(cache, before, pages):
    for name, now in state(cache).items():
        assert torch.equal(now[pages], before[name][pages]), name


# prefix sums over 9 rows, the sequences whose rows they still describe, and whether an append finds all of those
WRONG_SUMS = [([3, 5, 9], [0, 1], True), ([0, 5, 2], [0], True), ([0, 5, 400], [0], True), ([0, -1, 4], [], True),
              ([-40, 2, 4], [1], True), ([1000, 1001, 1002], [], True), ([0, 2, 500, 4, 6], [0, 3], False),
              ([0, 7, 7, 0, 5], [0, 1, 3], False), ([-2 ** 31, 2 ** 31 - 1, 3, 5], [2], False)]


@pytest.mark.parametrize("cu,good,found", WRONG_SUMS)
def test_wrong_prefix_sums_touch_nothing_else(cu, good, found):
    lens = [40, 30, 25, 50][:len(cu) - 1]
    rows, t, pages = tables(lens, 16, extra=16)
    cache = random_cache(pages, 2, 64, 64, 16, weights=True)
    q = torch.randn(9, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out_buf = torch.full((9 + 80, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse_buf = torch.full((4 * 9 + 160,), 7.0, device="cuda")
    out, lse = out_buf[40:49], lse_buf[80:116].view(4, 9)
    psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, cu_q=i32(cu), max_q=9, out=out, lse=lse)
    assert psf.device_status() == EDEVICE_ARGS
    claims = [sum(cu[b] <= r < cu[b + 1] for b in good) for r in range(9)]
    for b in good:
        want = ref.attend(ref.from_cache(cache), q[cu[b]:cu[b + 1]], rows[b:b + 1], lens[b:b + 1],
                          [0, cu[b + 1] - cu[b]], 0.1)
        alone = [r for r in range(cu[b], cu[b + 1]) if claims[r] == 1]
        at = [r - cu[b] for r in alone]
        close(out[alone], want[0][at], want[2][at], "out")
        close(lse[:, alone], want[1][:, at], want[3][:, at], "lse")
    out.fill_(7.0)
    lse.fill_(7.0)
    assert bool((out_buf == 7.0).all()) and bool((lse_buf == 7.0).all())

    before, c = state(cache), ref.from_cache(cache)
    x = torch.randn(9, 2, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    psf.kv_cache_append(cache, x, x, t, i32(lens), cu_new=i32(cu))
    assert psf.device_status() == EDEVICE_ARGS
    mine = {pg for b in good for pg in rows[b]}
    unchanged(cache, before, [pg for pg in range(pages) if pg not in mine])
    if found:
        for b in good:
            ref.append(c, x, x, [rows[b]], lens[b:b + 1], cu[b:b + 2])
        same(cache, c)


@pytest.mark.parametrize("how", ["one token", "prefix sums"])
@pytest.mark.parametrize("fault", ["page too large", "page negative", "length past the table", "length negative"])
def test_a_wrong_sequence_of_an_append_is_left_alone(how, fault):
    lens = [100, 70, 33]
    rows, t, pages = tables(lens, 32)
    cache = random_cache(pages, 2, 128, 128, 32, weights=True)
    n = i32(lens)
    if fault.startswith("page"):
        t[1, 69 // 32] = pages if fault == "page too large" else -1
    else:
        n[1] = t.shape[1] * 32 + 1 if fault == "length past the table" else -5
    before, c = state(cache), ref.from_cache(cache)
    x = torch.randn(3, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    psf.kv_cache_append(cache, x, x, t, n, None if how == "one token" else i32([0, 1, 2, 3]))
    assert psf.device_status() == EDEVICE_ARGS
    unchanged(cache, before, rows[1])
    for b in (0, 2):
        ref.append(c, x[b:b + 1], x[b:b + 1], [rows[b]], [lens[b]], [0, 1])
    same(cache, c)


# ---------------------------------------------------------------------------
# less usual forms

@pytest.mark.parametrize("dims", [(64, 64), (192, 128), (512, 512)])
def test_a_strided_cache_through_every_call(dims):
    """Rows of a page interleaved over the heads: one-token append, attention with weights, gather, eviction."""
    lens = [50, 1, 17, 140]
    rows, t, pages = tables(lens, 16)
    cache = random_cache(pages, 3, *dims, 16, weights=True, layout="ph")
    assert not cache.k.is_contiguous() and not cache.v.is_contiguous()
    g = torch.Generator().manual_seed(3)
    draw = lambda H, D: torch.randn(4, H, D, generator=g).bfloat16().cuda()  # noqa: E731
    check_append(cache, draw(3, dims[0]) * 5, draw(3, dims[1]) * 5, rows, t, lens, [1] * 4, uniform=True)
    check_attend(cache, draw(6, dims[0]), rows, t, lens, [1] * 4, dims[0] ** -0.5, accumulate=True, uniform=True)
    k, v, cu = psf.kv_cache_gather(cache, t, i32(lens), sum(lens))
    c = ref.from_cache(cache)
    for b, n in enumerate(lens):
        for h in range(3):
            for name, x in (("k", k), ("v", v)):
                assert torch.equal(x[cu[b]:cu[b + 1], h].cpu().double(), ref.rows_of(c, name, rows[b], n, h))
    check_evict(cache, rows, t, lens, 37, 10)


@pytest.mark.parametrize("dims,G,B", [((128, 128), 2, 480), ((128, 128), 12, 330), ((192, 128), 3, 330),
                                      ((512, 512), 2, 170), ((64, 64), 11, 330)])
@pytest.mark.parametrize("softcap", [None, 5.0])
def test_more_units_than_shares_on_other_tiles(dims, G, B, softcap):
    """Results joined by share, in tiles of 8 and of 16 rows and all widths; units that several shares have among them."""
    r = random.Random(B)
    lens = [r.choice([0, 1, 20, 40, r.randint(0, 40)]) for _ in range(B)]
    lens[0], lens[B // 2], lens[-1] = 700, 2500, 900
    m_rows = [r.choice([0, 1, 1, 2]) for _ in range(B)]
    m_rows[0] = m_rows[B // 2] = m_rows[-1] = 2
    rows, t, pages = tables(lens, 16, seed=B)
    cache = random_cache(pages, 2, *dims, 16, seed=B)
    cu = prefix(m_rows)
    q = torch.randn(cu[-1] + 5, 2 * G, dims[0], generator=torch.Generator().manual_seed(B)).bfloat16().cuda()
    out = torch.full((cu[-1] + 5, 2 * G, dims[1]), 3.0, dtype=torch.bfloat16, device="cuda")
    got = psf.attn_cache_fwd(q, cache, t, i32(lens), 0.1, cu_q=i32(cu), max_q=2, softcap=softcap, out=out)
    assert psf.device_status() == 0
    want = ref.attend(ref.from_cache(cache), q, rows, lens, cu, 0.1, softcap=softcap)
    close(got[0], want[0], want[2], "out")
    close(got[1], want[1], want[3], "lse")


@pytest.mark.parametrize("captured", [False, True])
def test_branches_that_meet_at_a_call(captured):
    """Queries from one stream and new tokens from another, joined by events before the attention; what comes of it goes
    to the first stream again while eviction and gather follow on the second."""
    lens = [700, 40, 129]
    rows, t, pages = tables(lens, 32, extra=8)
    g = torch.Generator().manual_seed(4)
    raw = torch.randn(3, 8, 128, generator=g).cuda()
    x = torch.randn(3, 2, 128, generator=g).bfloat16().cuda()
    n = i32([m + 1 for m in lens])
    a, b = torch.cuda.Stream(), torch.cuda.Stream()

    def step(cache):
        start = torch.cuda.current_stream()
        a.wait_stream(start)
        b.wait_stream(start)
        with torch.cuda.stream(a):
            q = raw
            for _ in range(20):  # long enough for the append to be over first, or not
                q = q * 1.0
            q = q.bfloat16()
        with torch.cuda.stream(b):
            psf.kv_cache_append(cache, x, x, t, n)
            b.wait_stream(a)
            out, lse = psf.attn_cache_fwd(q, cache, t, n, 0.1, accumulate=True)
            a.wait_stream(b)
            new = psf.kv_cache_evict(cache, t, n, 100, 20)
            k = psf.kv_cache_gather(cache, t, new, 300)[0]
        with torch.cuda.stream(a):
            copy = out.clone()
            q.record_stream(b)
            out.record_stream(a)
        start.wait_stream(a)
        start.wait_stream(b)
        return out, lse, copy, new, k[:241]

    cache = random_cache(pages, 2, 128, 128, 32, weights=True)
    c = ref.from_cache(cache)
    now = [m + 1 for m in lens]
    ref.append(c, x, x, rows, now, [0, 1, 2, 3])
    want = ref.attend(c, raw.bfloat16(), rows, now, [0, 1, 2, 3], 0.1, accumulate=True)
    if captured:
        step(random_cache(pages, 2, 128, 128, 32, weights=True))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(cache)
        graph.replay()
    else:
        got = step(cache)
    torch.cuda.synchronize()
    close(got[0], want[0], want[2], "out")
    close(got[1], want[1], want[3], "lse")
    assert torch.equal(got[2], got[0]) and got[3].tolist() == [100, 41, 100]
    again = random_cache(pages, 2, 128, 128, 32, weights=True)
    psf.kv_cache_append(again, x, x, t, n)
    psf.attn_cache_fwd(raw.bfloat16(), again, t, n, 0.1, accumulate=True)
    new = psf.kv_cache_evict(again, t, n, 100, 20)
    k = psf.kv_cache_gather(again, t, new, 300)[0]
    assert torch.equal(k[:241], got[4])
    for name, value in state(again).items():
        assert torch.equal(state(cache)[name], value), name
    assert psf.device_status() == 0
