"""The 8-bit cache in 64 bits, from its definitions, one token at a time where that is plain.

Shares no code with the package. A cache here is a dict of CPU tensors: k, v
(float64 e4m3 values), ks, vs (float64 scales), w (float64 weights or None).
"""
import math

import torch

U16 = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
U32 = 2.0 ** -24


def e4m3(x):
    """Nearest e4m3 value, ties to even; what is not finite is NaN; |x| <= 448 up to a rounding."""
    x = torch.where(x.isfinite(), x, math.nan)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def scale_of(a):
    """Smallest power of two s >= 2^-126 with a <= 448 s."""
    if a == 0:
        return 2.0 ** -126
    e = math.ceil(math.log2(a / 448))
    if a <= 448 * 2.0 ** (e - 1):
        e -= 1
    if a > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -126)


def from_cache(c):
    up = lambda t: t.detach().cpu().double()  # noqa: E731
    return dict(k=up(c.k), v=up(c.v), ks=up(c.k_scale), vs=up(c.v_scale), w=None if c.weight is None else up(c.weight),
                page=c.page_size)


def append(c, k, v, table, lens, cu):
    page, H = c["page"], c["k"].shape[1]
    k, v = k.detach().cpu().double(), v.detach().cpu().double()
    for b, n in enumerate(lens):
        first = n - (cu[b + 1] - cu[b])
        for p in range(first // page, (n + page - 1) // page):
            r0, r1 = max(first - p * page, 0), min(n - p * page, page)
            if r1 <= r0:
                continue
            t0, pg = cu[b] + p * page + r0 - first, table[b][p]
            for codes, scale, x in ((c["k"], c["ks"], k), (c["v"], c["vs"], v)):
                for h in range(H):
                    new = x[t0:t0 + r1 - r0, h]
                    fin = new[new.isfinite()].abs()
                    s = scale_of(float(fin.max()) if fin.numel() else 0.0)
                    if r0:
                        old = float(scale[pg, h])
                        s = max(s, old)
                        codes[pg, h, :r0] = e4m3(codes[pg, h, :r0] * (old / s))
                    codes[pg, h, r0:r1] = e4m3(new / s)
                    scale[pg, h] = s
            if c["w"] is not None:
                c["w"][pg, :, r0:r1] = 0


def rows_of(c, name, table_row, n, h):
    page = c["page"]
    D = c[name].shape[3]
    x = torch.zeros(n, D, dtype=torch.float64)
    for p in range((n + page - 1) // page):
        r = min(page, n - p * page)
        pg = table_row[p]
        x[p * page:p * page + r] = c[name][pg, h, :r] * c[name + "s"][pg, h]
    return x


def attend(c, q, table, lens, cu, scale, causal=True, window=None, softcap=None, accumulate=False):
    """-> out, lse (float64), and how far a kernel may be from each, by counting its roundings:

    a score is a sum of D products in fp32 and a few factors, so it is off by at most (D + 8) u32 sum |q||k| scale (the
    cap has slope <= 1, and its own roundings are below 8 u32 cap); a probability relative to that, plus 2^-21 for
    exp2 and its argument's rounding (|z| log2(e) u32 each side), plus half a step of fp16 (2^-11) where it enters
    the product with V, or 2^-32 of the largest one's scale where fp16 has no normal number for it; the sums of n
    terms add n u32; the result is rounded once to its type.
    """
    q64 = q.detach().cpu().double()
    T, Hq, D = q64.shape
    H = c["k"].shape[1]
    G, Dv = Hq // H, c["v"].shape[3]
    out = torch.zeros(T, Hq, Dv, dtype=torch.float64)
    lse = torch.full((Hq, T), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    add = torch.zeros_like(c["w"]) if accumulate else None
    add_tol = torch.zeros_like(c["w"]) if accumulate else None
    for b, n in enumerate(lens):
        m = cu[b + 1] - cu[b]
        for h in range(H):
            K, V = rows_of(c, "k", table[b], n, h), rows_of(c, "v", table[b], n, h)
            for i in range(m):
                at = i + n - m
                hi = min(n, at + 1) if causal else n
                lo = max(0, at - window + 1) if window else 0
                if hi <= lo:
                    continue
                x = q64[cu[b] + i, h * G:(h + 1) * G]
                z = scale * (x @ K[lo:hi].T)
                big = scale * (x.abs() @ K[lo:hi].abs().T)
                dz = (D + 8) * U32 * big
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                    dz = dz + 8 * U32 * softcap
                l = torch.logsumexp(z, -1)
                p = torch.exp(z - l[:, None])
                top = dz.amax(-1, keepdim=True)
                rel = 2 * top + 2.0 ** -21 + 4 * U32 * (z.abs().amax(-1, keepdim=True) + l.abs()[:, None]) + (hi - lo) * U32
                t = cu[b] + i
                o = p @ V[lo:hi]
                out[t, h * G:(h + 1) * G] = o
                lse[h * G:(h + 1) * G, t] = l
                mass = p @ V[lo:hi].abs()
                out_tol[t, h * G:(h + 1) * G] = ((rel + 2.0 ** -11) * mass + 2.0 ** -32 * (hi - lo) * V[lo:hi].abs().max()
                                                 ) * 1.01 + U16[q.dtype] * 1.01 * o.abs() + 2.0 ** -24
                lse_tol[h * G:(h + 1) * G, t] = rel[:, 0] + 4 * U32 * l.abs()
                if accumulate:
                    w, tol = p.sum(0), (p * rel).sum(0) + G * U32
                    for j in range(lo, hi):
                        add[table[b][j // c["page"]], h, j % c["page"]] += w[j - lo]
                        add_tol[table[b][j // c["page"]], h, j % c["page"]] += tol[j - lo]
    if accumulate:
        c["w"] += add
        return out, lse, out_tol, lse_tol, add_tol + 8 * U32 * c["w"].abs()
    return out, lse, out_tol, lse_tol


def evict(c, table, lens, budget, recent):
    page, H = c["page"], c["k"].shape[1]
    new_lens = []
    for b, n in enumerate(lens):
        if n <= budget:
            new_lens.append(n)
            continue
        for h in range(H):
            at = lambda name, j: c[name][table[b][j // page], h, j % page]  # noqa: E731
            key = [(-math.inf if math.isnan(w) else -w, j) for j, w in
                   ((j, float(at("w", j))) for j in range(n - recent))]
            kept = sorted(j for _, j in sorted(key)[:budget - recent]) + list(range(n - recent, n))
            for name in ("k", "v"):
                old = [float(c[name + "s"][table[b][j // page], h]) for j in kept]
                x = [at(name, j).clone() for j in kept]
                for p in range((budget + page - 1) // page):
                    r0, r1 = p * page, min((p + 1) * page, budget)
                    s = max(old[r0:r1])
                    for r in range(r0, r1):
                        ratio = float(torch.tensor(old[r] / s, dtype=torch.float32)) if s > 0 else 1.0  # as declared
                        c[name][table[b][p], h, r - r0] = e4m3(x[r] * ratio)
                    c[name + "s"][table[b][p], h] = s
            w = [float(at("w", j)) for j in kept]
            for r, x in enumerate(w):
                c["w"][table[b][r // page], h, r % page] = x
        new_lens.append(budget)
    return new_lens
