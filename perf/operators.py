"""Measured cases of the paged key-value cache's operators.

Three operators that a decoding program runs in turn over one paged cache:

* ``append``  rotates the new queries and keys by their positions and writes the
  keys and values into the pages of their sequences;
* ``attend``  attention of one new token for each sequence over its pages, and,
  where the cache is bounded, the sum of the attention weights that each cached
  entry received;
* ``evict``   brings every sequence back to its budget: the newest entries and
  the heaviest of the others stay.

The cache: ``k`` and ``v`` [pages][page][kv heads][head dim] bf16, ``table``
[sequences][pages of a sequence] int32 (-1: no page), ``lens`` [sequences] int32,
``weight`` fp32 and ``pos`` int32 [sequences][kv heads][slots].

With ``own`` false ``run`` computes in plain 32-bit torch operations, with ``own``
true through the package's entry points.
"""

from __future__ import annotations

import math

import torch

own = False

THETA = 1e7


# ------------------------------------------------------------------ the cases

def _attend(name, seqs, lo, hi, heads, kv, hd, page, dtype, accumulate):
    return {"name": name, "op": "attend", "seqs": seqs, "lo": lo, "hi": hi, "heads": heads, "kv": kv, "hd": hd,
            "page": page, "dtype": dtype, "accumulate": accumulate}


def _append(name, seqs, rows, heads, kv, hd, page, dtype, rotate):
    return {"name": name, "op": "append", "seqs": seqs, "rows": rows, "heads": heads, "kv": kv, "hd": hd,
            "page": page, "dtype": dtype, "rotate": rotate}


def _evict(name, seqs, lo, hi, budget, recent, kv, hd, page):
    return {"name": name, "op": "evict", "seqs": seqs, "lo": lo, "hi": hi, "budget": budget, "recent": recent,
            "kv": kv, "hd": hd, "page": page}


def listed():
    return [
        # the first tokens of one conversation: nothing but latency
        _attend("attend 1x97", 1, 97, 97, 16, 2, 128, 64, "float32", False),
        # one sequence at the context of the block's decode benchmark
        _attend("attend 1x4096", 1, 4096, 4096, 16, 2, 128, 64, "float32", False),
        # one sequence with a whole book in its context: all SMs on two KV heads
        _attend("attend 1x131075", 1, 131075, 131075, 16, 2, 128, 64, "bfloat16", False),
        # a serving batch of unequal sequences, empty slots of the batch among
        # them, with a bounded cache (weights accumulated)
        _attend("attend 64x0..8191 weights", 64, 0, 8191, 16, 2, 128, 32, "bfloat16", True),
        # the largest batch, fp32 rows as the block hands them over
        _attend("attend 256x4096", 256, 3500, 4608, 16, 2, 128, 64, "float32", False),
        # one KV head for each query head, small heads and pages
        _attend("attend 24x513 heads 8/8 hd 64", 24, 1, 1025, 8, 8, 64, 16, "bfloat16", False),
        # one token of one sequence: latency
        _append("append 1 row", 1, 1, 16, 2, 128, 64, "float32", True),
        # one token for each sequence of a batch
        _append("append 64 rows", 64, 1, 16, 2, 128, 32, "float32", True),
        # prompts that were computed in contiguous caches go into the pages
        _append("append 4x4093 rows", 4, 4093, 16, 2, 128, 64, "bfloat16", False),
        # the steady state of one bounded sequence: a few entries over the budget
        _evict("evict 1x4112->4096", 1, 4112, 4112, 4096, 512, 2, 128, 64),
        # a batch in which some sequences are under the budget
        _evict("evict 64x1500..8190->4096", 64, 1500, 8190, 4096, 256, 2, 128, 32),
        # long prompts are cut to a quarter
        _evict("evict 3x65537->16384", 3, 65537, 65537, 16384, 1024, 2, 128, 64),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "evict"])
    heads, kv, hd = rng.choice([(16, 2, 128), (16, 2, 128), (8, 8, 64), (8, 1, 128), (16, 4, 64), (12, 4, 96),
                                (16, 1, 128), (8, 2, 256), (20, 2, 128)])
    page = rng.choice([16, 32, 64, 128])
    if op == "attend":
        # at most as many cached entries as the largest listed case has
        seqs = _between(rng, 1, 256)
        hi = _between(rng, 1, max(1, min(131072, int(900_000 * 256 / (kv * hd) / seqs))))
        lo = rng.choice([0, max(0, hi // 3), hi])
        return _attend("", seqs, lo, hi, heads, kv, hd, page, rng.choice(["float32", "bfloat16"]), rng.random() < 0.5) | {"name": "drawn"}
    if op == "append":
        seqs = _between(rng, 1, 128)
        rows = _between(rng, 1, max(1, 16000 * 256 // (kv * hd) // seqs))
        return _append("", seqs, rows, heads, kv, hd, page, rng.choice(["float32", "bfloat16"]), rng.random() < 0.7) | {"name": "drawn"}
    seqs = _between(rng, 1, 64)
    hi = _between(rng, 2, max(2, min(65537, int(400_000 * 256 / (kv * hd) / seqs))))
    budget = max(1, int(hi * rng.uniform(0.15, 1.05)))
    return _evict("", seqs, rng.choice([hi, max(1, hi // 2)]), hi, budget, int(budget * rng.uniform(0, 0.5)), kv, hd,
                  page) | {"name": "drawn"}


# ------------------------------------------------------------------ inputs

def _lens(case):
    """The sequences' lengths, evenly from lo to hi (the same for every seed)."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _cache(g, lens, kv, hd, page, spare, filled=True):
    """Pages in a random order over the pool, a table with -1 behind each
    sequence's last page, and the pools' contents."""
    n = len(lens)
    used = [-(-(m + spare) // page) for m in lens]
    width = max(1, max(used))
    total = max(1, sum(used))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([sum(used[:i]) for i in range(n)], device="cuda")
    count = torch.tensor(used, device="cuda")
    at = torch.arange(width, device="cuda")
    index = (first[:, None] + at).clamp(max=total - 1)
    table = torch.where(at < count[:, None], perm[index], torch.full_like(perm[index], -1)).contiguous()
    k = torch.empty(total, page, kv, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    for t in (k, v):  # in parts, so that the fp32 draws stay small
        for i in range(0, total, 4096):
            part = t[i:i + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") if filled else torch.zeros(part.shape, device="cuda"))
    return {"k": k, "v": v, "table": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "weight": torch.zeros(n, kv, width * page, device="cuda"),
            "pos": torch.zeros(n, kv, width * page, dtype=torch.int32, device="cuda")}


def _kept(state):
    """What a user of the package keeps between calls: the cache's handle, the
    output tensors and a workspace."""
    from quantized_moe_transformer_gb300 import binding as qb
    c = state["cache"]
    state["handle"] = qb.PagedCache(c["k"], c["v"], c["table"], c["lens"], c["weight"], c["pos"])
    return qb


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, kv, hd, page = case["op"], case["kv"], case["hd"], case["page"]
    s = {"op": op}
    if op == "attend":
        order = torch.randperm(case["seqs"], generator=g, device="cuda").tolist()
        lens = _lens(case)
        lens = [lens[i] for i in order]
        s["cache"] = _cache(g, lens, kv, hd, page, 0)
        # trained queries and keys give scores of a few units
        s["q"] = _randn(g, case["seqs"], case["heads"], hd) * 1.5
        s["q"] = s["q"].to(getattr(torch, case["dtype"]))
        s["accumulate"] = case["accumulate"]
        if case["accumulate"]:
            s["cache"]["weight"].copy_(torch.rand(s["cache"]["weight"].shape, generator=g, device="cuda"))
        s["out"] = torch.empty_like(s["q"])
        if own:
            qb = _kept(s)
            s["ws"] = qb.paged_attention_workspace(s["handle"], case["heads"], case["accumulate"])
    elif op == "append":
        seqs, rows, dtype = case["seqs"], case["rows"], getattr(torch, case["dtype"])
        # a cached beginning of each sequence, then the new rows; one row in
        # sixteen of a long call is padding (slot -1)
        start = [0 if rows > 16 else 37 * (i % 9) for i in range(seqs)]
        s["cache"] = _cache(g, start, kv, hd, page, rows, filled=False)
        s["cache"]["weight"].fill_(1.0)
        n = seqs * rows
        at = torch.arange(n, device="cuda")
        s["seq"] = (at // rows).to(torch.int32)
        base = torch.tensor(start, device="cuda")[s["seq"].long()]
        slot = base + at % rows
        pad = (at % 16 == 15) & (rows > 16)
        s["slot"] = torch.where(pad, torch.full_like(slot, -1), slot).to(torch.int32)
        # a bounded cache's positions run ahead of its slots
        ahead = torch.randint(0, 100000, (seqs,), generator=g, device="cuda")
        s["at"] = (slot + ahead[s["seq"].long()]).to(torch.int32)
        s["rotate"] = case["rotate"]
        s["kn"], s["vn"] = _randn(g, n, kv, hd, dtype=dtype), _randn(g, n, kv, hd, dtype=dtype)
        # the queries are there where the rows come from a projection
        s["q"] = _randn(g, n, case["heads"], hd, dtype=dtype) if case["rotate"] else None
        s["q_out"] = torch.empty_like(s["q"]) if case["rotate"] else None
        if own:
            _kept(s)
    else:
        order = torch.randperm(case["seqs"], generator=g, device="cuda").tolist()
        lens = _lens(case)
        lens = [lens[i] for i in order]
        c = s["cache"] = _cache(g, lens, kv, hd, page, 0)
        n, slots = case["seqs"], c["pos"].shape[2]
        # slots below the budget hold an earlier eviction's entries in any
        # order, the slots behind them the newest entries in their order
        length = c["lens"].long()[:, None, None]
        below = length.clamp(max=case["budget"])
        at = torch.arange(slots, device="cuda").expand(n, kv, slots)
        shuffle = torch.rand(n, kv, slots, generator=g, device="cuda")
        old = torch.where(at < below, shuffle, 1.0 + at.float()).argsort(dim=2).argsort(dim=2)
        ahead = torch.randint(0, 100000, (n, 1, 1), generator=g, device="cuda")
        c["pos"].copy_((torch.where(at < below, old, at) + ahead).to(torch.int32))
        s["next"] = (length + ahead)[:, 0, 0].to(torch.int32)
        # accumulated weights: a few heavy entries, many light ones, equal ones
        w = torch.exp(2.5 * torch.randn(n, kv, slots, generator=g, device="cuda"))
        same = torch.rand(n, kv, slots, generator=g, device="cuda")
        c["weight"].copy_(torch.where(same < 0.1, torch.zeros_like(w), torch.where(same < 0.2, torch.round(w), w)))
        s["budget"], s["recent"] = case["budget"], case["recent"]
        s["new"] = {"lens": torch.zeros_like(c["lens"]), "weight": torch.zeros_like(c["weight"]),
                    "pos": torch.zeros_like(c["pos"])}
        if own:
            qb = _kept(s)
            s["ws"] = qb.cache_evict_workspace(s["handle"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"attend": _plain_attend, "append": _plain_append, "evict": _plain_evict}[state["op"]](state)


def _run_own(s):
    from quantized_moe_transformer_gb300 import binding as qb
    c = s["cache"]
    if s["op"] == "attend":
        qb.paged_attention(s["handle"], s["q"], out=s["out"], accumulate=s["accumulate"], ws=s["ws"])
        return {"out": s["out"], "weight": c["weight"]} if s["accumulate"] else {"out": s["out"]}
    if s["op"] == "append":
        qb.paged_append(s["handle"], s["kn"], s["vn"], s["at"], q=s["q"], q_out=s["q_out"], seq=s["seq"], slot=s["slot"],
                        rope_theta=THETA if s["rotate"] else 0.0)
        got = {"k": c["k"], "v": c["v"], "lens": c["lens"], "weight": c["weight"], "pos": c["pos"]}
        return got | {"q": s["q_out"]} if s["rotate"] else got
    new = s["new"]
    qb.cache_evict(s["handle"], s["next"], s["budget"], s["recent"], lens_out=new["lens"], weight_out=new["weight"],
                   pos_out=new["pos"], ws=s["ws"])
    return {"k": c["k"], "v": c["v"], **new}


def _plain_attend(s):
    c, q = s["cache"], s["q"]
    n, heads, hd = q.shape
    page, kv = c["k"].shape[1], c["k"].shape[2]
    slots = c["table"].shape[1] * page
    table = c["table"].long().clamp(min=0)
    k = c["k"][table].reshape(n, slots, kv, hd).permute(0, 2, 3, 1).float()
    v = c["v"][table].reshape(n, slots, kv, hd).permute(0, 2, 1, 3).float()
    there = (torch.arange(slots, device=q.device) < c["lens"][:, None])[:, None, None]
    x = q.float().reshape(n, kv, heads // kv, hd) @ k / math.sqrt(hd)
    x = torch.where(there, x, torch.full_like(x, -math.inf))
    top = x.amax(dim=3, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(dim=3, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_((p @ torch.where(there.transpose(2, 3), v, torch.zeros_like(v))).reshape(n, heads, hd))
    if not s["accumulate"]:
        return {"out": s["out"]}
    c["weight"].add_(p.sum(dim=2))
    return {"out": s["out"], "weight": c["weight"]}


def _rotated(x, at):
    """x [rows][heads][hd] with pairs (i, i + hd/2) turned by at * THETA^(-2i/hd)."""
    half = x.shape[2] // 2
    angle = at.double()[:, None] * THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)


def _plain_append(s):
    c = s["cache"]
    page = c["k"].shape[1]
    k = _rotated(s["kn"], s["at"]) if s["rotate"] else s["kn"].float()
    real = (s["slot"] >= 0).nonzero()[:, 0]
    seq, slot = s["seq"].long()[real], s["slot"].long()[real]
    where = c["table"].long()[seq, slot // page], slot % page
    c["k"][where] = k[real].to(torch.bfloat16)
    c["v"][where] = s["vn"][real].to(torch.bfloat16)
    c["pos"][seq, :, slot] = s["at"][real][:, None].expand(-1, c["pos"].shape[1])
    c["weight"][seq, :, slot] = 0.0
    c["lens"].copy_(torch.zeros_like(c["lens"]).scatter_reduce(0, seq, (slot + 1).to(torch.int32), "amax").maximum(c["lens"]))
    got = {"k": c["k"], "v": c["v"], "lens": c["lens"], "weight": c["weight"], "pos": c["pos"]}
    if not s["rotate"]:
        return got
    s["q_out"].copy_(_rotated(s["q"], s["at"]))
    return got | {"q": s["q_out"]}


def _plain_evict(s):
    c, new = s["cache"], s["new"]
    page, slots = c["k"].shape[1], c["pos"].shape[2]
    at = torch.arange(slots, device=c["pos"].device)
    length = c["lens"].long()[:, None, None]
    keep_n = length.clamp(max=s["budget"])
    there = at < length
    young = c["pos"] >= s["next"][:, None, None] - s["recent"]
    rank_of = torch.where(there, torch.where(young, 2, 1), 0)
    w = torch.where(young | torch.isnan(c["weight"]), torch.full_like(c["weight"], -math.inf), c["weight"])
    order = w.sort(dim=2, descending=True, stable=True).indices
    order = order.gather(2, rank_of.gather(2, order).sort(dim=2, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(2, order, at.expand_as(order))
    kept = rank < keep_n
    b, g, src = (kept & (at >= keep_n)).nonzero(as_tuple=True)
    dst = (~kept & (at < keep_n)).nonzero(as_tuple=True)[2]
    from_, to = c["table"].long()[b, src // page], c["table"].long()[b, dst // page]
    for pool in (c["k"], c["v"]):
        pool[to, dst % page, g] = pool[from_, src % page, g]
    for name in ("weight", "pos"):
        new[name].copy_(torch.where(at < keep_n, c[name], new[name]))
        new[name][b, g, dst] = c[name][b, g, src]
    new["lens"].copy_(keep_n[:, 0, 0])
    return {"k": c["k"], "v": c["v"], **new}


# ------------------------------------------------------------------ its work

def work(case):
    """Each cached entry, row and table read once and each result written once."""
    kv, hd, page = case["kv"], case["hd"], case["page"]
    row = kv * hd * 2 * 2  # one entry's key and value over all KV heads
    if case["op"] == "attend":
        lens, size = _lens(case), 4 if case["dtype"] == "float32" else 2
        total = sum(lens)
        moved = total * row + 2 * case["seqs"] * case["heads"] * hd * size
        moved += 4 * case["seqs"] + 4 * sum(-(-m // page) for m in lens)
        return {"bytes": moved + (8 * total * kv if case["accumulate"] else 0), "flops": 4 * total * case["heads"] * hd}
    if case["op"] == "append":
        n, size = case["seqs"] * case["rows"], 4 if case["dtype"] == "float32" else 2
        real = n - sum(i % 16 == 15 for i in range(n)) if case["rows"] > 16 else n
        moved = real * (2 * kv * hd * size + row + 8 * kv) + 12 * n + 4 * case["seqs"]
        q = 2 * n * case["heads"] * hd * size if case["rotate"] else 0
        return {"bytes": moved + q, "flops": 3 * hd * (n * case["heads"] + real * kv) if case["rotate"] else 0}
    moved, flops = 4 * case["seqs"] * 3, 0
    for m in _lens(case):
        keep = min(m, case["budget"])
        more = m - keep
        # the newest entries move to holes, and as many of the other new ones
        # as the same share of all others stays
        young = min(more, case["recent"])
        held = min(keep, case["recent"])
        share = (keep - held) / max(1, m - held)
        moves = young + (more - young) * share if more else 0
        moved += 8 * m * kv + 8 * keep * kv + 2 * moves * row
        flops += m * kv
    return {"bytes": moved, "flops": flops}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["cache"]
    page, kv = c["k"].shape[1], c["k"].shape[2]
    table, lens = c["table"].tolist(), c["lens"].tolist()
    if case["op"] == "attend":
        heads, hd = case["heads"], case["hd"]
        out = torch.zeros(case["seqs"], heads, hd, dtype=torch.float64, device="cuda")
        weight = c["weight"].double()
        for b, m in enumerate(lens):
            if m == 0:
                continue
            pages = torch.tensor(table[b][:-(-m // page)], device="cuda")
            k = c["k"][pages].flatten(0, 1)[:m].double()
            v = c["v"][pages].flatten(0, 1)[:m].double()
            for g in range(kv):
                mine = slice(g * (heads // kv), (g + 1) * (heads // kv))
                p = torch.softmax(s["q"][b, mine].double() @ k[:, g].T * hd ** -0.5, dim=1)
                out[b, mine] = p @ v[:, g]
                weight[b, g, :m] += p.sum(dim=0)
        return {"out": out, "weight": weight} if case["accumulate"] else {"out": out}
    if case["op"] == "append":
        def turned(x):
            x, half = x.double(), x.shape[2] // 2
            z = torch.complex(x[..., :half], x[..., half:])
            i = torch.arange(half, dtype=torch.float64, device="cuda")
            angle = s["at"].double()[:, None] * torch.exp(-i / half * math.log(THETA))
            z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
            return torch.cat([z.real, z.imag], dim=2)
        k, v = c["k"].double(), c["v"].double()
        kn = turned(s["kn"]) if case["rotate"] else s["kn"].double()
        real = s["slot"] >= 0
        seq, slot = s["seq"][real].long(), s["slot"][real].long()
        flat = c["table"].long()[seq].gather(1, (slot // page)[:, None])[:, 0] * page + slot % page
        k.view(-1, *k.shape[2:]).index_copy_(0, flat, kn[real])
        v.view(-1, *v.shape[2:]).index_copy_(0, flat, s["vn"][real].double())
        weight = c["weight"].double()
        weight.transpose(1, 2)[seq, slot] = 0
        got = {"k": k, "v": v, "lens": None, "weight": weight, "pos": None}
        return got | {"q": turned(s["q"])} if case["rotate"] else got
    k, v, weight = c["k"].double(), c["v"].double(), s["new"]["weight"].double()
    w, pos, after = c["weight"].double().cpu().numpy(), c["pos"].cpu().numpy(), s["next"].tolist()
    for b, m in enumerate(lens):
        keep = min(m, case["budget"])
        for g in range(kv):
            young = pos[b, g, :m] >= after[b] - case["recent"]
            best = sorted(range(m), key=lambda j: (not young[j], 0.0 if young[j] else -w[b, g, j], j))[:keep]
            held = set(best)
            to = [j for j in range(keep) if j not in held]
            come = sorted(j for j in best if j >= keep)
            weight[b, g, :keep] = c["weight"][b, g, :keep].double()
            if not to:
                continue
            to, come = torch.tensor(to, device="cuda"), torch.tensor(come, device="cuda")
            at = torch.tensor(table[b], device="cuda")
            weight[b, g, to] = c["weight"][b, g, come].double()
            for pool, old in ((k, c["k"]), (v, c["v"])):
                pool[at[to // page], to % page, g] = old[at[come // page], come % page, g].double()
    return {"k": k, "v": v, "lens": None, "weight": weight, "pos": None}
