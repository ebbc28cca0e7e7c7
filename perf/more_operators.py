"""Measured cases of the operators that bring prompts into the paged key-value cache.

Four calls that a serving program makes in turn for a step of packed rows (whole
prompts, parts of prompts and single new tokens of many sequences, one after the
other in one tensor):

* ``plan``    cuts sequences back, gives their pages to the pool, hands out pages
  for each sequence's new rows and writes the rows' sequences, slots and positions;
* ``rope``    turns queries and keys by their positions (both layouts of pairs, a
  part of the head, frequencies scaled for long contexts), and its transpose;
* ``append``  the same inside the call that writes the rows into the cache;
* ``attend``  causal attention of the packed rows over their sequences' pages.

The cache: ``k`` and ``v`` [pages][page][kv heads][head dim] bf16, ``table``
[sequences][pages of a sequence] int32 (-1: no page), ``lens`` [sequences] int32.
The pool: ``free`` [pages] int32, of which the first ``n_free`` [1] are free pages,
a stack whose top is the last of them.

With ``own`` false ``run`` computes in plain torch operations, with ``own`` true
through the package's entry points.
"""

from __future__ import annotations

import math

import torch

own = False

THETA = 1e7
ROTATIONS = {
    # the first half of the head, pairs half the turned part apart
    "half": dict(layout="half", share=0.5, scaling=None),
    # neighbours turn together; every position counts for a quarter
    "neighbours": dict(layout="interleaved", share=1.0, scaling="linear"),
    # frequencies that turned often within the first context stay, slow ones are stretched
    "long": dict(layout="half", share=1.0, scaling="parts"),
    "neighbours long": dict(layout="interleaved", share=0.25, scaling="parts"),
}
FACTOR, CONTEXT, LOW, HIGH = 4.0, 32768.0, 1.0, 32.0


# ------------------------------------------------------------------ the cases

def _attend(name, seqs, lo, hi, before, heads, kv, hd, page, dtype):
    """``seqs`` sequences with lo..hi new rows behind 0..before cached entries (the first
    sequence has all of ``before`` and hi rows)."""
    return {"name": name, "op": "attend", "seqs": seqs, "lo": lo, "hi": hi, "before": before, "heads": heads, "kv": kv,
            "hd": hd, "page": page, "dtype": dtype}


def _rope(name, rows, heads, kv, hd, dtype, rotation, transpose):
    return {"name": name, "op": "rope", "rows": rows, "heads": heads, "kv": kv, "hd": hd, "dtype": dtype,
            "rotation": rotation, "transpose": transpose}


def _append(name, seqs, rows, heads, kv, hd, page, dtype, rotation):
    return {"name": name, "op": "append", "seqs": seqs, "rows": rows, "heads": heads, "kv": kv, "hd": hd, "page": page,
            "dtype": dtype, "rotation": rotation}


def _plan(name, seqs, lo, hi, before, page, slots, ended, spare):
    """lo..hi new rows behind 0..before entries; every ``ended``-th sequence is given up first; the pool
    has ``spare`` hundredths of the pages that are asked for."""
    return {"name": name, "op": "plan", "seqs": seqs, "lo": lo, "hi": hi, "before": before, "page": page, "slots": slots,
            "ended": ended, "spare": spare}


def listed():
    return [
        # a short question as the first prompt of a conversation: latency
        _attend("attend 1x37", 1, 37, 37, 0, 16, 2, 128, 64, "float32"),
        # the prompt length of the block's prefill benchmark, fp32 rows as the block has them
        _attend("attend 1x4096", 1, 4096, 4096, 0, 16, 2, 128, 64, "float32"),
        # a step that mixes single tokens, parts of prompts and prompts behind what is cached
        _attend("attend 32x1..1000 behind 0..3000", 32, 1, 1000, 3000, 16, 2, 128, 32, "bfloat16"),
        # prompts of a batch, one KV head for each query head, small heads and pages
        _attend("attend 8x300..2048 heads 8/8 hd 64", 8, 300, 2048, 0, 8, 8, 64, 16, "bfloat16"),
        # a part of a prompt behind a whole book: few rows on a long axis
        _attend("attend 1x256 behind 65000", 1, 256, 256, 65000, 16, 4, 64, 64, "bfloat16"),
        # the longest prompt, the most work
        _attend("attend 1x16384", 1, 16384, 16384, 0, 16, 2, 128, 128, "bfloat16"),
        # one token of one sequence: latency
        _rope("rope 1 row", 1, 16, 2, 128, "float32", "half", False),
        # the packed rows of a long prompt out of a joint projection, positions beyond the first context
        _rope("rope 16384 rows long", 16384, 16, 2, 128, "bfloat16", "long", False),
        # the rows of a step into the cache
        _append("append 64 rows neighbours", 64, 1, 16, 2, 128, 32, "float32", "neighbours"),
        _append("append 4x4093 rows long", 4, 4093, 16, 2, 128, 64, "bfloat16", "long"),
        # a decoding step: one row each, a page here and there
        _plan("plan 96x1", 96, 1, 1, 8000, 64, 8192, 0, 100),
        # prompts for a fifth of the sequences, whose predecessors ended; not all find room
        _plan("plan 256x0..2000", 256, 0, 2000, 4000, 16, 8192, 5, 80),
    ]


def _between(rng, lo, hi):
    """A whole number, spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rope", "append", "plan"])
    heads, kv, hd = rng.choice([(16, 2, 128), (16, 2, 128), (8, 8, 64), (8, 1, 128), (16, 4, 64), (12, 4, 96),
                                (16, 1, 128), (8, 2, 256), (20, 2, 128)])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["float32", "bfloat16"])
    if op == "attend":
        # as much as the largest listed case at most, were all sequences as long as the longest
        seqs = _between(rng, 1, 64)
        most = 16384 * 16384 // 2 * 16 * 128 // (heads * hd) // seqs
        hi = _between(rng, 1, min(12000, math.isqrt(most)))
        before = rng.choice([0, _between(rng, 1, max(1, min(100000 // seqs, most // hi - hi)))])
        return _attend("drawn", seqs, rng.choice([0, 1, hi]), hi, before, heads, kv, hd, page, dtype)
    rotation = rng.choice(sorted(ROTATIONS))
    if op == "rope":
        rows = _between(rng, 1, 16384 * 18 * 128 // ((heads + kv) * hd))
        return _rope("drawn", rows, heads, kv, hd, dtype, rotation, rng.random() < 0.4)
    if op == "append":
        seqs = _between(rng, 1, 128)
        rows = _between(rng, 1, max(1, 16000 * 256 // (kv * hd) // seqs))
        return _append("drawn", seqs, rows, heads, kv, hd, page, dtype, rotation)
    seqs = _between(rng, 1, 512)
    hi = _between(rng, 1, max(1, 500_000 // seqs))
    before = _between(rng, 1, max(1, 1_000_000 // seqs))
    slots = page * (-(-(hi + before) // page) + rng.choice([0, 3]))
    return _plan("drawn", seqs, rng.choice([0, 1, hi]), hi, before, page, slots, rng.choice([0, 1, 3]),
                 rng.choice([50, 100, 130]))


# ------------------------------------------------------------------ inputs

def _spread(n, lo, hi):
    """n whole numbers, evenly from hi down to lo (the same for every seed)."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _new_and_before(case):
    """The sequences' new rows and the entries before them: long parts of prompts stand behind short
    beginnings and the other way round, but for the first."""
    count = _spread(case["seqs"], case["lo"], case["hi"])
    before = _spread(case["seqs"], 0, case["before"])
    return count, before[:1] + before[:0:-1] if case["seqs"] > 1 else [case["before"]]


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _table(g, used, width):
    """Page numbers in a random order, -1 behind each sequence's last page, and how many there are."""
    total = max(1, sum(used))
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(used, device="cuda")
    first = count.cumsum(0) - count
    at = torch.arange(width, device="cuda")
    index = (first[:, None] + at).clamp(max=total - 1)
    return torch.where(at < count[:, None], perm[index], torch.full_like(perm[index], -1)).contiguous(), total


def _pools(g, total, page, kv, hd, filled):
    k = torch.zeros(total, page, kv, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    for t in (k, v) if filled else ():  # in parts, so that the fp32 draws stay small
        for i in range(0, total, 4096):
            t[i:i + 4096].copy_(torch.randn(t[i:i + 4096].shape, generator=g, device="cuda"))
    return k, v


def _frequencies(rotation, hd):
    """(turned dims, the pairs' angles of one position, the factor on the result), in 64 bits."""
    r = ROTATIONS[rotation]
    dims = int(hd * r["share"])
    f = THETA ** (-torch.arange(dims // 2, device="cuda", dtype=torch.float64) / (dims // 2))
    if r["scaling"] == "linear":
        f = f / FACTOR
    if r["scaling"] == "parts":
        turns = CONTEXT * f / (2 * math.pi)
        stay = ((turns - LOW) / (HIGH - LOW)).clamp(0, 1)
        f = f * (stay + (1 - stay) / FACTOR)
    return dims, f, 0.1 * math.log(FACTOR) + 1 if r["scaling"] == "parts" else 1.0


def _rope_of(rotation, hd):
    """The same as the package's plan of a rotation."""
    from quantized_moe_transformer_gb300 import binding as qb
    r = ROTATIONS[rotation]
    return qb.Rope(int(hd * r["share"]), THETA, layout=r["layout"], scaling=r["scaling"], factor=FACTOR, context=CONTEXT,
                   low=LOW, high=HIGH, scale=0.1 * math.log(FACTOR) + 1 if r["scaling"] == "parts" else 1.0)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"attend": _prepare_attend, "rope": _prepare_rope, "append": _prepare_append, "plan": _prepare_plan}[case["op"]](case, g)


def _prepare_attend(case, g):
    s = {"op": "attend"}
    seqs, heads, kv, hd, page = (case[n] for n in ("seqs", "heads", "kv", "hd", "page"))
    count, before = _new_and_before(case)
    order = torch.randperm(seqs, generator=g, device="cuda").tolist()
    count, before = [count[i] for i in order], [before[i] for i in order]
    lens = [a + b for a, b in zip(count, before)]
    used = [-(-m // page) for m in lens]
    s["table"], total = _table(g, used, max(1, max(used)))
    s["k"], s["v"] = _pools(g, total, page, kv, hd, True)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["count"] = torch.tensor(count, dtype=torch.int32, device="cuda")
    s["first"] = (s["count"].cumsum(0) - s["count"]).to(torch.int32)
    # rows are cut to a multiple of 8, as a program that keeps few shapes does: the last ones belong to nobody
    rows = max(8, -(-sum(count) // 8) * 8)
    # trained queries and keys give scores of a few units
    s["q"] = (_randn(g, rows, heads, hd) * 1.5).to(getattr(torch, case["dtype"]))
    s["out"] = torch.zeros_like(s["q"])
    s["most"], s["slots"] = max(count), s["table"].shape[1] * page
    if own:
        from quantized_moe_transformer_gb300 import binding as qb
        s["handle"] = qb.PagedCache(s["k"], s["v"], s["table"], s["lens"])
        s["ws"] = qb.paged_prefill_attention_workspace(s["handle"], rows, heads)
    return s


def _prepare_rope(case, g):
    rows, heads, kv, hd, dtype = (case[n] for n in ("rows", "heads", "kv", "hd", "dtype"))
    dtype = getattr(torch, dtype)
    s = {"op": "rope", "transpose": case["transpose"], "rotation": case["rotation"]}
    # queries and keys as a joint projection leaves them: queries, keys and values of a row side by side
    joint = _randn(g, rows, heads + 2 * kv, hd, dtype=dtype)
    s["q"], s["k"] = joint[:, :heads], joint[:, heads:heads + kv]
    s["pos"] = (torch.arange(rows, device="cuda") + torch.randint(0, 100000, (), generator=g, device="cuda")).to(torch.int32)
    s["q_out"] = torch.empty(rows, heads, hd, device="cuda", dtype=dtype)
    s["k_out"] = torch.empty(rows, kv, hd, device="cuda", dtype=dtype)
    s["turns"] = _frequencies(case["rotation"], hd)
    if own:
        s["rope"] = _rope_of(case["rotation"], hd)
    return s


def _prepare_append(case, g):
    seqs, rows, heads, kv, hd, page = (case[n] for n in ("seqs", "rows", "heads", "kv", "hd", "page"))
    dtype = getattr(torch, case["dtype"])
    s = {"op": "append", "rotation": case["rotation"]}
    before = [0 if rows > 16 else 37 * (i % 9) for i in range(seqs)]
    used = [-(-(m + rows) // page) for m in before]
    s["table"], total = _table(g, used, max(used))
    s["k"], s["v"] = _pools(g, total, page, kv, hd, False)
    s["lens"] = torch.tensor(before, dtype=torch.int32, device="cuda")
    n = seqs * rows
    at = torch.arange(n, device="cuda")
    s["seq"] = (at // rows).to(torch.int32)
    slot = s["lens"].long()[s["seq"].long()] + at % rows
    # one row in sixteen of a long call is padding (slot -1)
    pad = (at % 16 == 15) & (rows > 16)
    s["slot"] = torch.where(pad, torch.full_like(slot, -1), slot).to(torch.int32)
    ahead = torch.randint(0, 100000, (seqs,), generator=g, device="cuda")
    s["pos"] = (slot + ahead[s["seq"].long()]).to(torch.int32)
    s["kn"], s["vn"] = _randn(g, n, kv, hd, dtype=dtype), _randn(g, n, kv, hd, dtype=dtype)
    s["q"] = _randn(g, n, heads, hd, dtype=dtype)
    s["q_out"] = torch.empty_like(s["q"])
    s["turns"] = _frequencies(case["rotation"], hd)
    if own:
        from quantized_moe_transformer_gb300 import binding as qb
        s["handle"] = qb.PagedCache(s["k"], s["v"], s["table"], s["lens"])
        s["rope"] = _rope_of(case["rotation"], hd)
    return s


def _prepare_plan(case, g):
    seqs, page = case["seqs"], case["page"]
    s = {"op": "plan", "page": page}
    count, before = _new_and_before(case)
    order = torch.randperm(seqs, generator=g, device="cuda").tolist()
    ended = [case["ended"] > 0 and i % case["ended"] == 0 for i in order]
    count, before = [count[i] for i in order], [before[i] for i in order]
    used = [-(-m // page) for m in before]
    s["table"], total = _table(g, used, case["slots"] // page)
    asked = sum(-(-(c + (0 if e else b)) // page) - (0 if e else u) for c, b, u, e in zip(count, before, used, ended))
    given = sum(u for u, e in zip(used, ended) if e)
    free = max(0, asked * case["spare"] // 100 - given)
    s["pages"] = total + free
    s["free"] = torch.zeros(s["pages"], dtype=torch.int32, device="cuda")
    s["free"][:free] = total + torch.randperm(free, generator=g, device="cuda").to(torch.int32)
    s["n_free"] = torch.tensor([free], dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(before, dtype=torch.int32, device="cuda")
    # the others are cut to what they hold: a page that an earlier step took ahead goes back
    s["keep"] = torch.tensor([0 if e else b for b, e in zip(before, ended)], dtype=torch.int32, device="cuda")
    s["count"] = torch.tensor(count, dtype=torch.int32, device="cuda")
    s["next"] = s["keep"] + torch.randint(0, 100000, (seqs,), generator=g, device="cuda").to(torch.int32)
    rows = max(8, -(-sum(count) // 8) * 8)
    s["first"], s["granted"] = torch.empty_like(s["count"]), torch.empty_like(s["count"])
    s["seq"], s["slot"], s["pos"] = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(3))
    if own:
        from quantized_moe_transformer_gb300 import binding as qb
        k = torch.zeros(s["pages"], page, 1, 8, device="cuda", dtype=torch.bfloat16)
        s["handle"] = qb.PagedCache(k, torch.zeros_like(k), s["table"], s["lens"])
        s["pool"] = qb.PagePool(s["free"], s["n_free"])
        s["ws"] = qb.paged_plan_workspace(s["handle"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _run_own(state)
    return {"attend": _plain_attend, "rope": _plain_rope, "append": _plain_append, "plan": _plain_plan}[state["op"]](state)


def _run_own(s):
    from quantized_moe_transformer_gb300 import binding as qb
    if s["op"] == "attend":
        qb.paged_prefill_attention(s["handle"], s["q"], s["first"], s["count"], out=s["out"], ws=s["ws"])
        return {"out": s["out"]}
    if s["op"] == "rope":
        qb.rope(s["rope"], s["pos"], s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"], transpose=s["transpose"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "append":
        qb.paged_append(s["handle"], s["kn"], s["vn"], s["pos"], q=s["q"], q_out=s["q_out"], seq=s["seq"], slot=s["slot"],
                        rope=s["rope"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"], "lens": s["lens"]}
    qb.paged_plan(s["handle"], s["pool"], s["count"], keep=s["keep"], next_pos=s["next"], first=s["first"],
                  granted=s["granted"], seq=s["seq"], slot=s["slot"], pos=s["pos"], ws=s["ws"])
    return {n: s[n] for n in ("table", "lens", "free", "n_free", "first", "granted", "seq", "slot", "pos")}


def _plain_attend(s):
    q, lens, count = s["q"], s["lens"].long(), s["count"].long()
    rows, heads, hd = q.shape
    page, kv = s["k"].shape[1], s["k"].shape[2]
    n, slots, most = lens.shape[0], s["slots"], s["most"]
    if most == 0:
        return {"out": s["out"]}
    table = s["table"].long().clamp(min=0)
    there = torch.arange(slots, device=q.device) < lens[:, None]
    k = s["k"][table].reshape(n, slots, kv, hd).permute(0, 2, 3, 1).float()
    v = s["v"][table].reshape(n, slots, kv, hd).permute(0, 2, 1, 3).float()
    v = torch.where(there[:, None, :, None], v, torch.zeros_like(v))
    # the sequences' rows side by side, as long as the longest
    i = torch.arange(most, device=q.device)
    row = (s["first"].long()[:, None] + i).clamp(max=rows - 1)
    x = q.float()[row].reshape(n, most, kv, heads // kv, hd).permute(0, 2, 3, 1, 4).reshape(n, kv, -1, hd)
    x = (x @ k).mul_(1 / math.sqrt(hd)).view(n, kv, heads // kv, most, slots)
    sees = torch.arange(slots, device=q.device) < (lens - count)[:, None, None] + i[:, None] + 1
    x.masked_fill_(~(sees & there[:, None])[:, None, None], -math.inf)
    x.sub_(x.amax(dim=4, keepdim=True).clamp(min=-1e30)).exp_()
    total = x.sum(dim=4, keepdim=True)
    o = (x.view(n, kv, -1, slots) @ v).view(n, kv, heads // kv, most, hd) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, most, heads, hd).to(q.dtype)
    mine = i < count[:, None]
    s["out"][row[mine]] = o[mine]
    return {"out": s["out"]}


def _turned(x, pos, turns, layout, transpose=False):
    """x [rows][heads][hd], its pairs turned by their angles at ``pos``, in 32 bits."""
    dims, f, scale = turns
    angle = pos.double()[:, None] * f
    cos, sin = (angle.cos() * scale).float()[:, None], (angle.sin() * scale).float()[:, None]
    sin = -sin if transpose else sin
    x = x.float()
    if layout == "half":
        a, b = x[..., :dims // 2], x[..., dims // 2:dims]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., dims:]], dim=2)
    a, b = x[..., 0:dims:2], x[..., 1:dims:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2), x[..., dims:]], dim=2)


def _plain_rope(s):
    layout = ROTATIONS[s["rotation"]]["layout"]
    for x, y in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y.copy_(_turned(x, s["pos"], s["turns"], layout, s["transpose"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_append(s):
    page, layout = s["k"].shape[1], ROTATIONS[s["rotation"]]["layout"]
    real = (s["slot"] >= 0).nonzero()[:, 0]
    seq, slot = s["seq"].long()[real], s["slot"].long()[real]
    where = s["table"].long()[seq, slot // page], slot % page
    s["k"][where] = _turned(s["kn"], s["pos"], s["turns"], layout)[real].to(torch.bfloat16)
    s["v"][where] = s["vn"][real].to(torch.bfloat16)
    s["lens"].copy_(torch.zeros_like(s["lens"]).scatter_reduce(0, seq, (slot + 1).to(torch.int32), "amax").maximum(s["lens"]))
    s["q_out"].copy_(_turned(s["q"], s["pos"], s["turns"], layout))
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "lens": s["lens"]}


def _plain_plan(s):
    page, table, n = s["page"], s["table"].long(), s["count"].long().clamp(min=0)
    rows, width = s["seq"].shape[0], s["table"].shape[1]
    at = torch.arange(width, device=table.device)
    length = s["lens"].long().clamp(0, width * page)
    length = torch.where(s["keep"] >= 0, length.minimum(s["keep"].long()), length)
    s["lens"].copy_(torch.where(s["keep"] >= 0, length.to(torch.int32), s["lens"]))
    # pages behind what is kept go back, in the order of the sequences and of their pages
    owned = (table >= 0) & (table < s["pages"])
    back = owned & (s["keep"] >= 0)[:, None] & (at >= -(-length // page)[:, None])
    stack = torch.cat([s["free"][:int(s["n_free"])].long(), table[back]])
    table[back] = -1
    owned &= ~back
    # the pages that the new rows miss come off the stack, sequence by sequence, all of a sequence's or none
    need = ~owned & (at >= (length // page)[:, None]) & (at < -(-(length + n) // page)[:, None]) & (n > 0)[:, None]
    first = n.cumsum(0) - n
    fits = (length + n <= width * page) & (first + n <= rows)
    need &= fits[:, None]
    pages = need.sum(1)
    ok = fits & ((pages == 0) | (pages.cumsum(0) <= len(stack)))
    need &= ok[:, None]
    taken = int(need.sum())
    table[need] = stack.flip(0)[:taken]
    s["table"].copy_(table)
    left = stack[:len(stack) - taken]
    s["free"][:len(left)] = left.to(torch.int32)
    s["n_free"].fill_(len(left))
    s["first"].copy_(first)
    s["granted"].copy_(torch.where(ok, n, torch.zeros_like(n)))
    # the rows' maps; rows of nobody have neither sequence nor slot
    r = torch.arange(rows, device=table.device)
    b = torch.searchsorted(first + n, r, right=True)
    mine = b < len(n)
    b = b.clamp(max=len(n) - 1)
    i = r - first[b]
    s["seq"].copy_(torch.where(mine, b, torch.full_like(b, -1)))
    s["slot"].copy_(torch.where(mine & ok[b], length[b] + i, torch.full_like(b, -1)))
    s["pos"].copy_(torch.where(mine, s["next"].long()[b] + i, torch.zeros_like(b)))
    return {n: s[n] for n in ("table", "lens", "free", "n_free", "first", "granted", "seq", "slot", "pos")}


# ------------------------------------------------------------------ its work

def work(case):
    """Each entry, row and map read once and each result written once."""
    op = case["op"]
    size = 4 if case.get("dtype") == "float32" else 2
    if op == "attend":
        count, before = _new_and_before(case)
        entries = sum(b + c for b, c in zip(before, count) if c)
        visible = sum(c * b + c * (c + 1) // 2 for b, c in zip(before, count))
        moved = 4 * case["kv"] * case["hd"] * entries + 2 * sum(count) * case["heads"] * case["hd"] * size
        return {"bytes": moved + 12 * case["seqs"] + 4 * entries // case["page"], "flops": 4 * visible * case["heads"] * case["hd"]}
    if op == "rope":
        values = case["rows"] * (case["heads"] + case["kv"]) * case["hd"]
        return {"bytes": 2 * values * size + 4 * case["rows"], "flops": int(3 * values * ROTATIONS[case["rotation"]]["share"])}
    if op == "append":
        n, kv, hd = case["seqs"] * case["rows"], case["kv"], case["hd"]
        real = n - n // 16 if case["rows"] > 16 else n
        moved = real * 2 * kv * hd * (size + 2) + 2 * n * case["heads"] * hd * size + 12 * n + 4 * case["seqs"]
        return {"bytes": moved, "flops": int(3 * hd * (n * case["heads"] + real * kv) * ROTATIONS[case["rotation"]]["share"])}
    count, before = _new_and_before(case)
    page, every = case["page"], case["ended"]
    moved = 28 * case["seqs"] + 12 * max(8, -(-sum(count) // 8) * 8)
    back = sum(-(-b // page) for b in before) // every if every else 0
    new = sum(-(-c // page) for c in count)
    return {"bytes": moved + 8 * back + 8 * new, "flops": sum(count)}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None
    if case["op"] == "attend":
        out = s["out"].double()
        heads, kv, hd, page = case["heads"], case["kv"], case["hd"], case["page"]
        group = heads // kv
        for b, (m, n, first) in enumerate(zip(s["lens"].tolist(), s["count"].tolist(), s["first"].tolist())):
            pages = s["table"][b, :-(-m // page)].long()
            for g in range(kv if n else 0):
                k, v = (s[t][pages, :, g].flatten(0, 1)[:m].double() for t in "kv")
                for lo in range(0, n, 1024):
                    hi = min(n, lo + 1024)
                    end = m - n + hi
                    q = s["q"][first + lo:first + hi, g * group:(g + 1) * group].double()
                    x = torch.einsum("rhd,jd->hrj", q, k[:end]) * hd ** -0.5
                    hidden = torch.ones(hi - lo, end, dtype=torch.bool, device="cuda").triu_(m - n + lo + 1)
                    p = torch.softmax(x.masked_fill_(hidden, -math.inf), dim=2)
                    out[first + lo:first + hi, g * group:(g + 1) * group] = torch.einsum("hrj,jd->rhd", p, v[:end])
        return {"out": out}
    dims, f, scale = s["turns"]
    layout = ROTATIONS[case["rotation"]]["layout"]

    def turned(x, sign):
        """The turned part as complex numbers, times unit numbers."""
        head, rest = x.double()[..., :dims], x.double()[..., dims:]
        pairs = head.unflatten(2, (2, dims // 2)).transpose(2, 3) if layout == "half" else head.unflatten(2, (dims // 2, 2))
        angle = sign * s["pos"].double()[:, None, None] * f
        z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(angle, scale), angle)
        pairs = torch.view_as_real(z)
        return torch.cat([(pairs.transpose(2, 3) if layout == "half" else pairs).flatten(2), rest], dim=2)

    if case["op"] == "rope":
        sign = -1.0 if case["transpose"] else 1.0
        return {"q": turned(s["q"], sign), "k": turned(s["k"], sign)}
    k, v = s["k"].double(), s["v"].double()
    real = s["slot"] >= 0
    seq, slot = s["seq"][real].long(), s["slot"][real].long()
    flat = s["table"].long()[seq].gather(1, (slot // case["page"])[:, None])[:, 0] * case["page"] + slot % case["page"]
    k.view(-1, *k.shape[2:]).index_copy_(0, flat, turned(s["kn"], 1.0)[real])
    v.view(-1, *v.shape[2:]).index_copy_(0, flat, s["vn"][real].double())
    return {"q": turned(s["q"], 1.0), "k": k, "v": v, "lens": None}
