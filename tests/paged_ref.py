"""Plain 64-bit implementations of the paged cache's operators, entry by entry,
and the seeded caches their tests use."""

import math

import torch


def entries(pool, table, b, n, page):
    """The n entries [n][kv][hd] of sequence b, in 64 bits, and which of them
    lie in a page that exists."""
    j = torch.arange(n, device=pool.device)
    pages = table[b].long()[j // page]
    there = (pages >= 0) & (pages < pool.shape[0])
    return pool[pages.clamp(0, pool.shape[0] - 1), j % page].double(), there


def attention(q, k, v, table, lens, page, scale=None):
    """(out, weights received [seqs][kv][slots], bound): ``bound`` is the largest
    sum over head dims of |q k| scale, which scales a score's rounding."""
    n_seqs, heads, hd = q.shape
    kv = k.shape[2]
    scale = 1 / math.sqrt(hd) if scale is None else scale
    slots = table.shape[1] * page
    out = torch.zeros(n_seqs, heads, hd, dtype=torch.float64, device=q.device)
    got = torch.zeros(n_seqs, kv, slots, dtype=torch.float64, device=q.device)
    bound = 0.0
    for b in range(n_seqs):
        n = max(0, min(int(lens[b]), slots))
        kk, there = entries(k, table, b, n, page)
        vv, _ = entries(v, table, b, n, page)
        if not bool(there.any()):
            continue
        kk, vv = kk[there], vv[there]
        for h in range(heads):
            g = h // (heads // kv)
            x = (kk[:, g] * q[b, h].double()).sum(1) * scale
            bound = max(bound, float((kk[:, g] * q[b, h].double()).abs().sum(1).max()) * abs(scale))
            p = torch.exp(x - x.max())
            p = p / p.sum()
            out[b, h] = (p[:, None] * vv[:, g]).sum(0)
            got[b, g, :n][there] += p
    return out, got, bound


def rotated(x, pos, theta):
    x = x.double()
    if theta == 0:
        return x
    half = x.shape[2] // 2
    i = torch.arange(half, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None] * theta ** (-2 * i / x.shape[2])
    c, s = ang.cos()[:, None], ang.sin()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * s, b * c + a * s], dim=2)


def evict(weight, pos, n, budget, first_young):
    """For one (sequence, KV head): (slots that stay in order of preference,
    moves [(from, to)]). ``first_young`` None: none is protected."""
    m = min(n, budget)
    w, p = weight.tolist(), pos.tolist()

    def order(j):
        young = first_young is not None and p[j] >= first_young
        x = -math.inf if math.isnan(w[j]) else w[j]
        return (not young, 0.0 if young else -x, j)

    best = sorted(range(n), key=order)[:m]
    held = set(best)
    return best, list(zip(sorted(j for j in best if j >= m), (j for j in range(m) if j not in held)))


def cache(seed, lens, kv, hd, page, width=None, layout="slots"):
    """Random pools with the pages of all sequences in a random order, NaN in
    every slot that holds no entry, and table entries behind the last page that
    name no page. layout: "slots" [pages][page][kv][hd], "heads"
    [pages][kv][page][hd] in memory, "both" keys and values of a page together."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    used = [-(-n // page) for n in lens]
    width = max(1, max(used)) if width is None else width
    total = sum(used) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[:, ::2] = 1 << 30
    shape = (total, page, kv, hd)
    if layout == "heads":
        pools = [torch.empty(total, kv, page, hd, device="cuda", dtype=torch.bfloat16).transpose(1, 2) for _ in "kv"]
    elif layout == "both":
        both = torch.empty(total, 2, page, kv, hd, device="cuda", dtype=torch.bfloat16)
        pools = [both[:, 0], both[:, 1]]
    else:
        pools = [torch.empty(shape, device="cuda", dtype=torch.bfloat16) for _ in "kv"]
    for t in pools:
        t.fill_(math.nan)
    at = 0
    for b, n in enumerate(lens):
        pages = perm[at:at + used[b]]
        at += used[b]
        table[b, :used[b]] = pages
        j = torch.arange(n, device="cuda")
        for t in pools:
            t[pages.long()[j // page], j % page] = torch.randn(n, kv, hd, generator=g, device="cuda").to(torch.bfloat16)
    slots = width * page
    weight = torch.rand(len(lens), kv, slots, generator=g, device="cuda")
    pos = torch.argsort(torch.rand(len(lens), kv, slots, generator=g, device="cuda"), dim=2).to(torch.int32)
    return {"k": pools[0], "v": pools[1], "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "weight": weight, "pos": pos}, g
