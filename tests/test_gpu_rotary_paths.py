"""GPU tests of the rotation's kernels where the other files' cases do not lead: heads past a group of a CTA's, several rows a CTA in
layouts that are not whole units, pages without an angle table, captured appends of two kernels that overlap, single rows of
many kinds at once."""
import random

import pytest
import torch

import packed_sequence_flash_gb300 as psf
from test_gpu_cache import i32, prefix, random_cache, tables
from test_gpu_rotary import append_case, check, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    assert psf.device_status() == 0
    yield


@pytest.mark.parametrize("H", [5, 8, 9, 17])
@pytest.mark.parametrize("layout", ["hp", "ph"])
@pytest.mark.parametrize("part", ["all", "odd"])
@pytest.mark.parametrize("uniform", [False, True])
def test_append_of_many_heads(H, layout, part, uniform):
    """Rounds of four heads, CTAs of eight and a rest; pages that hold older rows, whose scale grows in some of the heads."""
    dim, start, inter = dict(all=(64, 0, False), odd=(18, 7, True))[part]

    def touch(k, v, cache):
        cache.k_scale[:, ::2] *= 2.0 ** -9  # Gaussian rows are larger than what these hold
        cache.v_scale[:, 1::3] *= 2.0 ** -9

    append_case([3, 15, 40, 16], [1, 1, 1, 1] if uniform else [30, 1, 70, 16], 16, H, 64, 64, torch.bfloat16,
                (psf.rotary_frequencies(dim), dict(start=start, interleaved=inter)), uniform=uniform, Hq=2 * H, weights=True,
                layout=layout, seed=H, touch=touch)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,start", [(430, 7), (512, 0), (418, 93), (416, 96)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_without_a_table(interleaved, dim, start, dtype):
    """Pages of 128 with more than 208 pairs, in whole units and not (416: the last that has a table)."""
    append_case([100, 0, 127], [60, 130, 2], 128, 2, 512, 512, dtype,
                (psf.rotary_frequencies(dim), dict(start=start, interleaved=interleaved, scale=0.75)), Hq=2, weights=True)


@pytest.mark.parametrize("T", [607, 608, 609, 1216, 1823, 2600, 5003])
@pytest.mark.parametrize("D,dim,start", [(72, 72, 0), (128, 50, 3), (24, 24, 0), (8, 2, 5)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_any_layout_with_several_rows_a_cta(T, D, dim, start, interleaved):
    """Sizes around which a CTA takes 2, 3 and 4 rows: as the rows in calls of 300, and the first against 64 bits; in place too."""
    inv = psf.rotary_frequencies(dim)
    r = psf.Rotary(inv, start=start, interleaved=interleaved)
    q, k = normal(T, 3, D, seed=T), normal(T, 2, D, seed=T + 1)
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
    at = pos.cuda()
    parts = [psf.rotary_fwd(q[a:a + 300], k[a:a + 300], r, positions=at[a:a + 300]) for a in range(0, T, 300)]
    check(q[:300], k[:300], inv, pos[:300], parts[0], start=start, interleaved=interleaved)
    got = psf.rotary_fwd(q, k, r, positions=at)
    for x, want in zip(got, zip(*parts)):
        assert torch.equal(x, torch.cat(want))
    psf.rotary_fwd(q, k, r, at, None, None, q, k)
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])


@pytest.mark.parametrize("T", [2, 700, 3001])
def test_any_layout_in_documents_and_batches(T):
    inv = psf.rotary_frequencies(50)
    r = psf.Rotary(inv, start=3)
    q, k = normal(2 * T, 3, 128), normal(2 * T, 1, 128, seed=1)
    places = torch.arange(T, dtype=torch.int32, device="cuda").repeat(2)
    want = psf.rotary_fwd(q, k, r, positions=places)
    got = psf.rotary_fwd(q, k, r, cu_seqlens=i32([0, T, 2 * T]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    view = lambda x: x.view(2, T, x.size(1), 128).transpose(1, 2)  # noqa: E731
    got = psf.rotary_fwd(view(q), view(k), r)
    assert torch.equal(got[0], view(want[0])) and torch.equal(got[1], view(want[1]))


@pytest.mark.parametrize("part", ["all", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
def test_captured_append_of_prompts_with_queries(part, in_place):
    """The pages' and the queries' kernel overlap; what is captured before and behind them waits for both: the keys, values and
    queries are made anew in front of each append, and changed behind it."""
    dim, start = dict(all=(128, 0), odd=(50, 3))[part]
    r = psf.Rotary(psf.rotary_frequencies(dim), start=start)
    lens, new = [700, 40, 333], [500, 40, 200]
    rows, t, pages = tables([x + 300 for x in lens], 32)
    caches = [random_cache(pages, 8, 128, 128, 32) for _ in range(2)]
    T = sum(new)
    src = [normal(T, h, 128, seed=s) for s, h in enumerate((8, 8, 32))]
    mine = [torch.empty_like(x) for x in src]
    n, cu, step = i32(lens), i32(prefix(new)), torch.ones((), device="cuda")
    seen = torch.empty_like(src[2])

    def call(cache, k, v, q, out):
        got = psf.kv_cache_append_rotary(cache, k, v, r, t, n, cu, q=q, q_out=out)
        return psf.rotary_bwd(got, None, r, cu_seqlens=cu)[0]  # reads the queries at once

    def body():
        for a, b in zip(mine, src):
            torch.mul(b, step, out=a)
        seen.copy_(call(caches[0], *mine, mine[2] if in_place else None))
        for a in mine:
            a.fill_(float("nan"))
        n.add_(100)
        step.add_(1)

    body()
    n.copy_(i32(lens))
    step.fill_(1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        body()
    for name in ("k", "v"):
        getattr(caches[0], name).view(torch.uint8).copy_(getattr(caches[1], name).view(torch.uint8))
    for name in ("k_scale", "v_scale"):
        getattr(caches[0], name).copy_(getattr(caches[1], name))
    n.copy_(i32(lens))
    step.fill_(1)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    n.copy_(i32(lens))
    for i in range(3):
        want = call(caches[1], *[x * (i + 1) for x in src], None)
        torch.cuda.synchronize()
        n.add_(100)
    assert torch.equal(seen, want)
    for name in ("k", "v"):
        assert torch.equal(getattr(caches[0], name).view(torch.uint8), getattr(caches[1], name).view(torch.uint8))
    for name in ("k_scale", "v_scale"):
        assert torch.equal(getattr(caches[0], name), getattr(caches[1], name))


def test_appends_from_two_streams_at_once():
    """Two caches, one rotation, calls from two streams in turn."""
    r = psf.Rotary(psf.rotary_frequencies(128))
    lens, new = [600, 90], [600, 90]
    rows, t, pages = tables(lens, 64)
    k, v, q = normal(690, 4, 128), normal(690, 4, 128, seed=1), normal(690, 16, 128, seed=2)
    n, cu = i32(lens), i32(prefix(new))
    want_cache = random_cache(pages, 4, 128, 128, 64)
    want = psf.kv_cache_append_rotary(want_cache, k, v, r, t, n, cu, q=q)
    caches, streams = [random_cache(pages, 4, 128, 128, 64) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for c, s in zip(caches, streams):
            with torch.cuda.stream(s):
                got.append(psf.kv_cache_append_rotary(c, k, v, r, t, n, cu, q=q))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
    for c in caches:
        assert torch.equal(c.k.view(torch.uint8), want_cache.k.view(torch.uint8)) and torch.equal(c.k_scale, want_cache.k_scale)


def test_random_rotations():
    """Heads from 1 to 40, any head dim, part, kind of places and strides, forward and backward, against 64 bits."""
    r = random.Random(5)
    for trial in range(40):
        D = 8 * r.randint(1, 40)
        dim = 2 * r.randint(1, D // 2)
        kw = dict(start=r.randint(0, D - dim), interleaved=r.random() < 0.5, scale=r.choice([1.0, 1.25, 0.5]))
        inv = psf.rotary_frequencies(dim)
        T, Hq, Hkv = r.choice([1, 3, 64, 333, 900]), r.choice([1, 2, 5, 12, 40]), r.choice([0, 1, 3, 8])
        dt = r.choice([torch.bfloat16, torch.float16])
        fused = normal(T, Hq + 2 * Hkv + 1, D, dtype=dt, seed=trial)
        q, k = fused[:, :Hq], fused[:, Hq:Hq + Hkv] if Hkv else None
        pos = torch.randint(-1000, 1 << 20, (T,), generator=torch.Generator().manual_seed(trial), dtype=torch.int32)
        back = r.random() < 0.5
        rotary = psf.Rotary(inv, **kw)
        got = (psf.rotary_bwd if back else psf.rotary_fwd)(q, k, rotary, positions=pos.cuda())
        some = sorted(r.sample(range(T), min(T, 40)))  # (the reference is slow)
        check(q[some], None if k is None else k[some], inv, pos[some], [None if x is None else x[some] for x in got], back=back,
              **kw)
