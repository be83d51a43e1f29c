"""Cases of the 8-bit key/value cache: append, attention, eviction, gather.

Each case is one pass through one operator, in its plain form (elementary torch
operations in 32 bits) or, with ``own`` set, through the package's entry points.
``exact`` computes the same outputs in 64 bits from the definitions.

The cache holds e4m3 codes in pages of ``page`` tokens, [pages, Hkv, page, D],
with one fp32 scale per (page, head); ``table`` [B, max_pages] lists a
sequence's pages and ``lens`` [B] its tokens.
"""
import math
import random
import typing

import torch

own = False

NEG = float("-inf")


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one user, a short chat turn: a single query token, where latency is all there is
        dict(name="attend one at 777", op="attend", B=1, lo=777, hi=777, lens=1, m=1, ragged=False, Hq=16, Hkv=4,
             Dqk=128, Dv=128, page=64, dtype="bf16", window=0, softcap=0.0, weights=False),
        # one user, one long document behind the question: the key axis has to be split
        dict(name="attend one at 32768", op="attend", B=1, lo=32768, hi=32768, lens=1, m=1, ragged=False, Hq=32,
             Hkv=8, Dqk=128, Dv=128, page=64, dtype="bf16", window=0, softcap=0.0, weights=False),
        # an ordinary server batch: ragged lengths over the range of packed documents
        dict(name="attend 32 to 8192", op="attend", B=32, lo=64, hi=8192, lens=2, m=1, ragged=False, Hq=32, Hkv=8,
             Dqk=128, Dv=128, page=64, dtype="bf16", window=0, softcap=0.0, weights=False),
        # the largest: a full batch of long contexts
        dict(name="attend 64 to 32768", op="attend", B=64, lo=16384, hi=32768, lens=3, m=1, ragged=False, Hq=32,
             Hkv=8, Dqk=128, Dv=128, page=128, dtype="bf16", window=0, softcap=0.0, weights=False),
        # drafted tokens checked together, capped logits, small pages, fp16
        dict(name="attend 16 drafts capped", op="attend", B=16, lo=5, hi=4099, lens=4, m=5, ragged=True, Hq=32, Hkv=8,
             Dqk=128, Dv=128, page=16, dtype="fp16", window=0, softcap=30.0, weights=False),
        # a cache that will be evicted from: attention weights are accumulated
        dict(name="attend 24 weights", op="attend", B=24, lo=512, hi=12000, lens=5, m=1, ragged=False, Hq=16, Hkv=4,
             Dqk=128, Dv=128, page=64, dtype="bf16", window=0, softcap=0.0, weights=True),
        # the widest heads, with a left window
        dict(name="attend 8 wide windowed", op="attend", B=8, lo=300, hi=8192, lens=6, m=1, ragged=False, Hq=8, Hkv=2,
             Dqk=512, Dv=512, page=32, dtype="bf16", window=4096, softcap=0.0, weights=False),
        # prompts going into the cache
        dict(name="append 8 prompts", op="append", B=8, lo=0, hi=100, new_lo=300, new_hi=4000, lens=7, Hkv=8, Dqk=128,
             Dv=128, page=64, dtype="bf16", weights=False),
        # the new token of every sequence of a batch
        dict(name="append 64 tokens", op="append", B=64, lo=64, hi=8192, new_lo=1, new_hi=1, lens=8, Hkv=8, Dqk=128,
             Dv=128, page=64, dtype="bf16", weights=True),
        # a few sequences over their budget, others not
        dict(name="evict 4 to 1000", op="evict", B=4, lo=900, hi=1500, lens=9, budget=1000, recent=256, Hkv=4,
             Dqk=128, Dv=128, page=64),
        # a batch cut to a quarter of its memory
        dict(name="evict 48 to 4096", op="evict", B=48, lo=6000, hi=16384, lens=10, budget=4096, recent=512, Hkv=8,
             Dqk=128, Dv=128, page=64),
        # the cached keys and values of long prompts, for the packed attention over their next chunk
        dict(name="gather 16 to 8192", op="gather", B=16, lo=64, hi=8192, lens=11, Hkv=8, Dqk=128, Dv=128, page=64,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "evict", "gather"])
    Dqk, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128), (512, 512)])
    Hkv = rng.choice([1, 2, 4, 8]) if Dqk < 512 else rng.choice([1, 2])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    B = _log(rng, 1, 64)
    hi = _log(rng, 1, 32768)
    cap = 3e9 / (B * Hkv * (Dqk + Dv))  # tokens per sequence at the largest listed case's bytes
    hi = max(1, min(hi, int(cap)))
    lo = rng.randint(1, hi)
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    lens = rng.randint(100, 1 << 30)
    if op == "attend":
        m = rng.choice([1, 1, 1, 2, 3, 5, 8])
        return dict(op=op, B=B, lo=lo, hi=hi, lens=lens, m=m, ragged=m > 1 and rng.random() < 0.5, Hq=Hkv * G, Hkv=Hkv,
                    Dqk=Dqk, Dv=Dv, page=page, dtype=dtype, window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                    softcap=rng.choice([0.0, 0.0, 30.0]), weights=rng.random() < 0.3 and m * G <= 16)
    if op == "append":
        new_hi = _log(rng, 1, 4096) if rng.random() < 0.5 else 1
        new_hi = max(1, min(new_hi, 65536 // B))
        return dict(op=op, B=B, lo=0, hi=min(hi, 8192), new_lo=rng.randint(1, new_hi), new_hi=new_hi, lens=lens, Hkv=Hkv,
                    Dqk=Dqk, Dv=Dv, page=page, dtype=dtype, weights=rng.random() < 0.5)
    if op == "evict":
        hi = max(16, min(hi, 16384))
        budget = rng.randint(max(1, hi // 8), hi - 1)
        return dict(op=op, B=min(B, 48), lo=max(1, hi // 2), hi=hi, lens=lens, budget=budget, recent=rng.randint(0, budget),
                    Hkv=Hkv, Dqk=Dqk, Dv=Dv, page=page)
    hi = max(1, min(hi, 131072 // B))
    return dict(op=op, B=B, lo=min(lo, hi), hi=hi, lens=lens, Hkv=Hkv, Dqk=Dqk, Dv=Dv, page=page, dtype=dtype)


def _lengths(case):
    """The sequences' lengths (and new or query tokens), from the case alone; the first is the longest."""
    r = random.Random(case["lens"])
    lens = [case["hi"]] + [r.randint(case["lo"], case["hi"]) for _ in range(case["B"] - 1)]
    if case["op"] == "append":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
        return [n + k for n, k in zip(lens, new)], new  # seq_lens counts the new tokens
    if case["op"] == "attend" and case["ragged"]:
        return lens, [r.randint(1, case["m"]) for _ in range(case["B"])]
    return lens, [case.get("m", 1)] * case["B"]


def work(case):
    lens, rows = _lengths(case)
    Hkv, Dqk, Dv = case["Hkv"], case["Dqk"], case["Dv"]
    if case["op"] == "attend":
        W, Hq = case["window"], case["Hq"]
        seen = [min(n, W + m - 1) if W else n for n, m in zip(lens, rows)]
        pairs = sum(max(0, min(n, i + n - m + 1) - (max(0, i + n - m - W + 1) if W else 0))
                    for n, m in zip(lens, rows) for i in range(m))
        nbytes = sum(seen) * Hkv * (Dqk + Dv) + sum(rows) * Hq * (2 * (Dqk + Dv) + 4)
        if case["weights"]:
            nbytes += 8 * Hkv * sum(seen)
        return {"bytes": nbytes, "flops": 2 * (Dqk + Dv) * Hq * pairs}
    if case["op"] == "append":
        return {"bytes": 3 * (Dqk + Dv) * Hkv * sum(rows), "flops": 2 * (Dqk + Dv) * Hkv * sum(rows)}
    if case["op"] == "evict":
        over = [n for n in lens if n > case["budget"]]
        b = case["budget"]
        return {"bytes": sum(4 * n * Hkv + b * Hkv * (2 * (Dqk + Dv) + 4) for n in over) or 4 * case["B"],
                "flops": 2 * (Dqk + Dv) * Hkv * b * len(over)}
    return {"bytes": 3 * (Dqk + Dv) * Hkv * sum(lens), "flops": (Dqk + Dv) * Hkv * sum(lens)}


# ---------------------------------------------------------------------------
# inputs

class Cache(typing.NamedTuple):
    """The cache's tensors, as the package's KVCache holds them."""

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    weight: typing.Optional[torch.Tensor]


def _pow2_scale(a):
    """The smallest power of two s >= 2^-126 with a <= 448 s, of fp32 a."""
    bits = a.contiguous().view(torch.int32)
    e = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()
    return (e.clamp(1, 254) << 23).view(torch.float32)


def _filled(pages, H, page, D, gen, dev):
    """Codes and scales of Gaussian rows whose size differs from block to block."""
    codes = torch.empty(pages, H, page, D, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.empty(pages, H, dtype=torch.float32, device=dev)
    step = max(1, (1 << 28) // (H * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, H, page, D, generator=gen, device=dev, dtype=torch.float16).float()
        x = x * torch.exp2(torch.randint(-1, 2, (n, H, 1, 1), generator=gen, device=dev).float())
        s = _pow2_scale(x.abs().amax((2, 3)))
        scale[p:p + n] = s
        codes[p:p + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn)
    return codes, scale


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, Hkv, Dqk, Dv, page = case["B"], case["Hkv"], case["Dqk"], case["Dv"], case["page"]
    lens, rows = _lengths(case)
    need = [-(-n // page) for n in lens]
    total, width = sum(need), max(need)
    pages = total + 1  # one page that no sequence owns
    perm = torch.randperm(total, generator=gen, device=dev).int() + 1
    first = torch.tensor([sum(need[:b]) for b in range(B)], device=dev)
    count = torch.tensor(need, device=dev)
    at = torch.arange(width, device=dev)[None]
    idx = (first[:, None] + at).clamp(max=total - 1)
    table = torch.where(at < count[:, None], perm[idx], torch.tensor(-1, dtype=torch.int32, device=dev)).contiguous()
    k, ks = _filled(pages, Hkv, page, Dqk, gen, dev)
    v, vs = _filled(pages, Hkv, page, Dv, gen, dev)
    weight = None
    if case["op"] == "evict" or case.get("weights"):
        # accumulated weights: most tokens little, a few much, some never seen
        weight = torch.rand(pages, Hkv, page, generator=gen, device=dev) ** 8 * 4
        weight = torch.where(weight < 1e-6, 0.0, weight)
    cache = Cache(k, v, ks, vs, weight)
    lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    T = sum(rows)
    dt = torch.float16 if case.get("dtype") == "fp16" else torch.bfloat16
    s = dict(case=case, cache=cache, table=table, lens=lens, T=T, cu=None, total=int(lens.sum()))
    cu = [sum(rows[:b]) for b in range(B + 1)]
    s["cu_all"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["op"] == "attend":
        s["q"] = (1.5 * torch.randn(T, case["Hq"], Dqk, generator=gen, device=dev)).to(dt)
        s["cu"] = s["cu_all"] if case["ragged"] else None
        s["scale"] = Dqk ** -0.5
    elif case["op"] == "append":
        s["k"] = torch.randn(T, Hkv, Dqk, generator=gen, device=dev).to(dt)
        s["v"] = torch.randn(T, Hkv, Dv, generator=gen, device=dev).to(dt)
        s["cu"] = s["cu_all"] if case["new_hi"] > 1 else None
    s["dtype"] = dt
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    return {"attend": _attend, "append": _append, "evict": _evict, "gather": _gather}[s["case"]["op"]](s)


def _rows(s):
    """Sequence and place in it of each of the T packed rows, and each sequence's rows."""
    cu = s["cu_all"].long()
    t = torch.arange(s["T"], device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    return b, t - cu[b], cu[1:] - cu[:-1]


def _paged(x, table):
    """The pages of a [pages, Hkv, page, ...] tensor in the order of a table, as [B, Hkv, tokens, ...]."""
    b, p = table.shape
    y = x.view(torch.uint8)[table].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[table]
    y = y.transpose(1, 2)
    return y.reshape(b, y.shape[1], p * y.shape[3], *y.shape[4:])


def _values(codes, scale, table, page):
    per_token = scale[table].transpose(1, 2).repeat_interleave(page, 2)
    return _paged(codes, table).float() * per_token[..., None]


def _attend(s):
    c, cache = s["case"], s["cache"]
    window, softcap = c["window"] or None, c["softcap"] or None
    if own:
        import packed_sequence_flash_gb300 as psf
        out, lse = psf.attn_cache_fwd(s["q"], psf.KVCache(*cache), s["table"], s["lens"], s["scale"], cu_q=s["cu"],
                                      max_q=c["m"], window=window, softcap=softcap, accumulate=c["weights"])
        return (out, lse, cache.weight) if c["weights"] else (out, lse)
    table = s["table"].clamp(min=0).long()
    B, Hkv, Hq, m = c["B"], c["Hkv"], c["Hq"], c["m"]
    G = Hq // Hkv
    b, i, n_rows = _rows(s)
    n = s["lens"].long()
    k = _values(cache.k, cache.k_scale, table, c["page"])
    L = k.shape[2]
    at = (s["cu_all"][:-1, None].long() + torch.arange(m, device=n.device)).clamp(max=s["T"] - 1)
    q = s["q"][at].float().reshape(B, m, Hkv, G, c["Dqk"]).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, c["Dqk"])
    z = torch.matmul(q, k.transpose(2, 3)).reshape(B, Hkv, G, m, L) * s["scale"]
    del k
    if softcap:
        z = softcap * torch.tanh(z / softcap)
    j = torch.arange(L, device=n.device)
    last = torch.arange(m, device=n.device)[None] + (n - n_rows)[:, None]  # the last key a row sees
    seen = (j <= last[..., None]) & (j < n[:, None, None])
    if window:
        seen &= j > last[..., None] - window
    seen &= (torch.arange(m, device=n.device)[None] < n_rows[:, None])[..., None]
    z = z.masked_fill(~seen[:, None, None], NEG)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(top == NEG, 0.0, top))
    total = e.sum(-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    p = e / torch.where(total == 0, 1.0, total)
    v = _values(cache.v, cache.v_scale, table, c["page"]).masked_fill((j >= n[:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p.reshape(B, Hkv, G * m, L), v).reshape(B, Hkv, G, m, c["Dv"])
    out = o.permute(0, 3, 1, 2, 4)[b, i].reshape(s["T"], Hq, c["Dv"]).to(s["dtype"])
    lse = lse.permute(0, 3, 1, 2)[b, i].reshape(s["T"], Hq).t().contiguous()
    if not c["weights"]:
        return out, lse
    w = p.sum((2, 3)).reshape(B, Hkv, L // c["page"], c["page"]).transpose(1, 2)
    cache.weight.index_add_(0, table.reshape(-1), w.reshape(-1, Hkv, c["page"]))
    return out, lse, cache.weight


def _append(s):
    c, cache = s["case"], s["cache"]
    state = (cache.k, cache.v, cache.k_scale, cache.v_scale) + ((cache.weight,) if c["weights"] else ())
    if own:
        import packed_sequence_flash_gb300 as psf
        psf.kv_cache_append(psf.KVCache(*cache), s["k"], s["v"], s["table"], s["lens"], cu_new=s["cu"])
        return state
    page, table, n = c["page"], s["table"].long(), s["lens"].long()
    b, i, n_new = _rows(s)
    pos = (n - n_new)[b] + i
    pg, row = table[b, pos // page], pos % page
    begin = n - n_new
    older = begin % page  # older tokens in the page that the first new token enters
    pg0 = table.gather(1, (begin // page)[:, None])[:, 0]
    _quantised(cache.k, cache.k_scale, s["k"], pg, row, pg0, older, page)
    _quantised(cache.v, cache.v_scale, s["v"], pg, row, pg0, older, page)
    if c["weights"]:
        cache.weight[pg, :, row] = 0.0
    return state


def _quantised(codes, scale, x, pg, row, pg0, older, page):
    raw = codes.view(torch.uint8)
    x = x.float()
    H = x.shape[1]
    top = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)
    fresh = torch.full_like(scale, -1.0).scatter_reduce(0, pg[:, None].expand(-1, H), top, "amax")
    entered = fresh >= 0
    s = torch.where(entered, _pow2_scale(fresh.clamp(min=0)), scale)
    kept = torch.where((older > 0)[:, None], torch.maximum(s[pg0], scale[pg0]), s[pg0])
    s[pg0] = kept
    held = raw[pg0].view(torch.float8_e4m3fn).float() * (scale[pg0] / kept)[:, :, None, None]
    is_older = (torch.arange(page, device=x.device) < older[:, None])[:, None, :, None]
    raw[pg0] = torch.where(is_older, held.to(torch.float8_e4m3fn).view(torch.uint8), raw[pg0])
    new = (x / s[pg][..., None]).to(torch.float8_e4m3fn)
    raw[pg, :, row] = new.view(torch.uint8)
    scale.copy_(s)


def _evict(s):
    c, cache = s["case"], s["cache"]
    budget, recent, page, Hkv, B = c["budget"], c["recent"], c["page"], c["Hkv"], c["B"]
    state = (cache.k, cache.v, cache.k_scale, cache.v_scale, cache.weight)
    if own:
        import packed_sequence_flash_gb300 as psf
        return state + (psf.kv_cache_evict(psf.KVCache(*cache), s["table"], s["lens"], budget, recent),)
    n = s["lens"].long()
    dev = n.device
    table = s["table"].clamp(min=0).long()
    w = _paged(cache.weight, table)
    L = w.shape[2]
    if L < budget:  # no sequence is that long
        return state + (s["lens"].clone(),)
    j = torch.arange(L, device=dev)
    old = (j < (n - recent)[:, None])[:, None]
    order = torch.sort(torch.where(old, w, NEG), dim=2, descending=True, stable=True).indices
    tail = (n - recent).clamp(min=0)[:, None, None] + torch.arange(recent, device=dev)
    src = torch.cat([order[:, :, :budget - recent], tail.expand(-1, Hkv, -1)], 2).sort(2).values.clamp(max=L - 1)
    over = n > budget
    head = torch.arange(Hkv, device=dev)[None, :, None]
    row = torch.arange(budget, device=dev)
    spare = torch.arange(budget, device=dev) % page
    b = torch.arange(B, device=dev)[:, None, None]
    spg, srow = table[b, src // page], src % page
    dpg = torch.where(over[:, None], table[:, row // page], 0)[:, None].expand(-1, Hkv, -1)
    drow = torch.where(over[:, None], row % page, spare)[:, None].expand(-1, Hkv, -1)
    live = over[:, None, None]
    moved = torch.where(live, cache.weight[spg, head, srow], cache.weight[dpg, head, drow])
    _moved(cache.k, cache.k_scale, spg, srow, dpg, drow, head, live, page)
    _moved(cache.v, cache.v_scale, spg, srow, dpg, drow, head, live, page)
    cache.weight[dpg, head, drow] = moved
    return state + (s["lens"].clamp(max=budget),)


def _moved(codes, scale, spg, srow, dpg, drow, head, live, page):
    raw = codes.view(torch.uint8)
    B, H, n = spg.shape
    blocks = -(-n // page)
    s = scale[spg, head]
    pad = torch.nn.functional.pad(s, (0, blocks * page - n))
    new = pad.reshape(B, H, blocks, page).amax(3)
    per = new.repeat_interleave(page, 2)[:, :, :n]
    x = raw[spg, head, srow].view(torch.float8_e4m3fn).float() * (s / per)[..., None]
    x = x.to(torch.float8_e4m3fn).view(torch.uint8)
    raw[dpg, head, drow] = torch.where(live[..., None], x, raw[dpg, head, drow])
    block_pg = dpg[:, :, ::page]
    scale[block_pg, head] = torch.where(live, new, scale[block_pg, head])


def _gather(s):
    c, cache = s["case"], s["cache"]
    if own:
        import packed_sequence_flash_gb300 as psf
        return psf.kv_cache_gather(psf.KVCache(*cache), s["table"], s["lens"], s["total"], dtype=s["dtype"])
    n = s["lens"].long()
    cu = torch.nn.functional.pad(n.cumsum(0), (1, 0))
    t = torch.arange(s["total"], device=n.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = t - cu[b]
    pg, row = s["table"].long()[b, pos // c["page"]], pos % c["page"]
    k = cache.k.view(torch.uint8)[pg, :, row].view(torch.float8_e4m3fn).float() * cache.k_scale[pg][..., None]
    v = cache.v.view(torch.uint8)[pg, :, row].view(torch.float8_e4m3fn).float() * cache.v_scale[pg][..., None]
    return k.to(s["dtype"]), v.to(s["dtype"]), cu.int()


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time

def _e4m3(x):
    """Nearest e4m3 value (ties to even) of a float64 tensor with |x| <= 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "evict": _exact_evict,
            "gather": _exact_gather}[case["op"]](s)


def _sequence(codes, scale, pages, n):
    """[Hkv, n, D] values of one sequence."""
    x = codes.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double() * scale[pages].double()[:, :, None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_attend(s):
    c, cache = s["case"], s["cache"]
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    lens, cu = s["lens"].tolist(), s["cu_all"].tolist()
    out = torch.zeros(s["T"], c["Hq"], c["Dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["Hq"], s["T"]), NEG, dtype=torch.float64, device="cuda")
    weight = cache.weight.double() if c["weights"] else None
    for b, n in enumerate(lens):
        m = cu[b + 1] - cu[b]
        pages = s["table"][b, :-(-n // c["page"])].long()
        q = s["q"][cu[b]:cu[b + 1]].double().reshape(m, Hkv, G, c["Dqk"]).permute(1, 2, 0, 3)
        z = torch.einsum("hgid,hjd->hgij", q, _sequence(cache.k, cache.k_scale, pages, n)) * s["scale"]
        if c["softcap"]:
            z = c["softcap"] * torch.tanh(z / c["softcap"])
        last = torch.arange(m, device="cuda")[:, None] + n - m
        j = torch.arange(n, device="cuda")[None]
        hide = j > last
        if c["window"]:
            hide = hide | (j < last - c["window"] + 1)
        z = z.masked_fill(hide, NEG)
        l = torch.logsumexp(z, -1)
        p = torch.nan_to_num(torch.exp(z - l[..., None]), nan=0.0)
        o = torch.einsum("hgij,hjd->ihgd", p, _sequence(cache.v, cache.v_scale, pages, n))
        out[cu[b]:cu[b + 1]] = o.reshape(m, c["Hq"], c["Dv"])
        lse[:, cu[b]:cu[b + 1]] = l.reshape(c["Hq"], m)
        if c["weights"]:
            add = torch.zeros(Hkv, len(pages) * c["page"], dtype=torch.float64, device="cuda")
            add[:, :n] = p.sum((1, 2))
            weight[pages] += add.reshape(Hkv, len(pages), c["page"]).transpose(0, 1)
    return (out, lse, weight) if c["weights"] else (out, lse)


def _exact_append(s):
    c, cache = s["case"], s["cache"]
    lens, cu, page = s["lens"].tolist(), s["cu_all"].tolist(), c["page"]
    table = s["table"].tolist()
    answer = []
    for codes, scale, x in ((cache.k, cache.k_scale, s["k"]), (cache.v, cache.v_scale, s["v"])):
        codes, scale = codes.double(), scale.double()
        for b, n in enumerate(lens):
            begin = n - (cu[b + 1] - cu[b])
            for p in range(begin // page, (n - 1) // page + 1):
                r0, r1 = max(begin - p * page, 0), min(n - p * page, page)
                t0 = cu[b] + p * page + r0 - begin
                new, pg = x[t0:t0 + r1 - r0].double().transpose(0, 1), table[b][p]
                top = new.abs().amax((1, 2))
                fresh = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(min=-126)), 2.0 ** -126)
                use = torch.maximum(fresh, scale[pg]) if r0 else fresh
                codes[pg, :, :r0] = _e4m3(codes[pg, :, :r0] * (scale[pg] / use)[:, None, None])
                codes[pg, :, r0:r1] = _e4m3(new / use[:, None, None])
                scale[pg] = use
        answer += [codes, scale]
    answer = [answer[0], answer[2], answer[1], answer[3]]
    if c["weights"]:
        w = cache.weight.double()
        for b, n in enumerate(lens):
            for t in range(n - (cu[b + 1] - cu[b]), n):
                w[table[b][t // page], :, t % page] = 0
        answer.append(w)
    return answer


def _exact_evict(s):
    c, cache = s["case"], s["cache"]
    budget, recent, page, Hkv = c["budget"], c["recent"], c["page"], c["Hkv"]
    lens = s["lens"].tolist()
    pools = [(cache.k.double(), cache.k_scale.double()), (cache.v.double(), cache.v_scale.double())]
    weight = cache.weight.double()
    h = torch.arange(Hkv, device="cuda")[:, None]
    row = torch.arange(budget, device="cuda")
    for b, n in enumerate(lens):
        if n <= budget:
            continue
        table = s["table"][b].long()
        j = torch.arange(n, device="cuda")
        w = weight[table[j // page], :, j % page].t()[:, :n - recent]
        best = torch.argsort(-w, dim=1, stable=True)[:, :budget - recent]
        src = torch.cat([best, j[n - recent:].expand(Hkv, -1)], 1).sort(1).values
        spg, dpg = table[src // page], table[row // page].expand(Hkv, -1)
        moved = weight[spg, h, src % page]
        weight[dpg, h, row % page] = moved
        for codes, scale in pools:
            old = scale[spg, h]
            x = codes[spg, h, src % page] * old[..., None]
            for p in range(-(-budget // page)):
                r = slice(p * page, min((p + 1) * page, budget))
                top = old[:, r].amax(1)
                codes[table[p], :, :r.stop - r.start] = _e4m3(x[:, r] / top[:, None, None])
                scale[table[p]] = top
    return [pools[0][0], pools[1][0], pools[0][1], pools[1][1], weight, None]


def _exact_gather(s):
    c, cache = s["case"], s["cache"]
    parts = [[_sequence(codes, scale, s["table"][b, :-(-n // c["page"])].long(), n).transpose(0, 1)
              for b, n in enumerate(s["lens"].tolist())]
             for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    return [torch.cat(parts[0]), torch.cat(parts[1]), None]
