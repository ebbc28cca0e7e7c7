"""The paged key-value cache's operators against plain 64-bit implementations.

"CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
Now Splits": query heads share KV heads. The cases take the lengths at which
pages, tiles and work splits begin and end, empty sequences, several head
layouts, pools in three memory layouts, and pools that hold NaN wherever no
entry lies.

Tolerances. A score is a sum of hd products held in fp32: its rounding is at
most (hd + 8) 2^-24 of sum |q k| scale (the 8 for scaling, the maximum's
subtraction and the exponential). That moves a probability by at most twice its
relative size, and an output, which is a mean of values under the
probabilities, by at most 2 x that x max |v|. The probabilities and the partial
outputs add 2^-16 of max |v| (two bf16 parts of each probability, 2^-17, the
sums and the division). bf16 outputs are rounded once: 2^-8 of the value.
"""

import math

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


def handle(c, with_pos=True):
    return qb.PagedCache(c["k"], c["v"], c["table"], c["lens"], c["weight"], c["pos"] if with_pos else None)


def score_tol(hd, bound):
    return (hd + 8) * 2.0 ** -24 * bound


def close_out(got, want, bound, hd, v_max):
    tol = (2 * score_tol(hd, bound) + 2.0 ** -16) * v_max
    tol = tol + (2.0 ** -8 * want.abs() if got.dtype == torch.bfloat16 else 0.0)
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got.float()).all())
    assert bool((err <= tol).all()), float((err - tol).max())


def v_max(c):
    return float(torch.nan_to_num(c["v"].float(), nan=0.0).abs().max())


def check_attention(c, q, page, accumulate, scale=None, status=0):
    hd = q.shape[2]
    before = c["weight"].clone()
    out = qb.paged_attention(handle(c), q, accumulate=accumulate, scale=0.0 if scale is None else scale)
    torch.cuda.synchronize()
    assert qb.query_status() == status
    want, received, bound = ref.attention(q, c["k"], c["v"], c["table"], c["lens"], page, scale)
    close_out(out, want, bound, hd, max(v_max(c), 1e-30))
    if not accumulate:
        assert torch.equal(c["weight"], before)
        return out
    # every head's probability is off by 2 score roundings of its size; one
    # rounding for each of the sums over heads and the addition
    group = q.shape[1] // c["k"].shape[2]
    tol = received * (2 * score_tol(hd, bound) + (group + 8) * 2.0 ** -24) + (before.double() + received) * 2.0 ** -24
    err = (c["weight"].double() - before.double() - received).abs()
    assert bool((err <= tol + 1e-30).all()), float((err - tol).max())
    return out


LAYOUTS = [(16, 2, 128), (8, 8, 64), (12, 4, 96), (16, 1, 256), (20, 2, 128), (1, 1, 8), (33, 1, 40), (6, 2, 200)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,hd", LAYOUTS)
def test_attention_head_layouts(heads, kv, hd, dtype):
    c, g = ref.cache(1, [130, 1, 0, 77, 600], kv, hd, 16)
    q = torch.randn(5, heads, hd, generator=g, device="cuda").to(dtype)
    out = check_attention(c, q, 16, accumulate=True)
    assert bool((out[2] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,hd", [(16, 1, 256), (20, 2, 128), (33, 1, 40), (32, 2, 64), (48, 2, 128), (8, 4, 96)])
def test_attention_of_a_wide_table(heads, kv, hd, dtype):
    """A table for tens of thousands of slots a sequence (bf16 groups of more than
    8 heads take 16 at once there) with few entries, and with many."""
    lens = [130, 1, 0, 2077, 600]
    width = (1 << 25) // (4 * len(lens) * kv * hd * 16) + 1
    c, g = ref.cache(2, lens, kv, hd, 16, width=max(width, 200))
    q = torch.randn(5, heads, hd, generator=g, device="cuda").to(dtype)
    out = check_attention(c, q, 16, accumulate=True)
    assert bool((out[2] == 0).all())


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 512])
@pytest.mark.parametrize("around", [1, 8, 16, 32, 64, 128, 256, 512])
def test_attention_lengths_around_borders(page, around):
    lens = sorted({max(0, around + d) for d in (-9, -1, 0, 1, 7)})
    c, g = ref.cache(around, lens, 2, 128, page)
    q = torch.randn(len(lens), 16, 128, generator=g, device="cuda")
    check_attention(c, q, page, accumulate=True)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0], [1], [3000], [20000], [9000, 0, 1, 33, 4096, 2], list(range(0, 1300, 9)),
                                  [5] * 400])
@pytest.mark.parametrize("accumulate", [False, True])
def test_attention_batches(lens, accumulate):
    c, g = ref.cache(len(lens), lens, 2, 128, 32)
    q = (1.5 * torch.randn(len(lens), 16, 128, generator=g, device="cuda")).to(torch.bfloat16)
    check_attention(c, q, 32, accumulate)


@pytest.mark.parametrize("layout", ["heads", "both"])
@pytest.mark.parametrize("hd", [64, 128])
def test_attention_pool_layouts(layout, hd):
    c, g = ref.cache(3, [700, 31], 4, hd, 64, layout=layout)
    q = torch.randn(2, 8, hd, generator=g, device="cuda")
    check_attention(c, q, 64, accumulate=False)


def test_attention_contiguous_cache_as_pages():
    """A cache [ctx][kv][hd] as the block keeps it, seen as pages."""
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(1024, 2, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
    c = {"k": k.view(16, 64, 2, 128), "v": v.view(16, 64, 2, 128),
         "table": torch.arange(16, dtype=torch.int32, device="cuda")[None],
         "lens": torch.tensor([1000], dtype=torch.int32, device="cuda"),
         "weight": torch.zeros(1, 2, 1024, device="cuda"), "pos": torch.zeros(1, 2, 1024, dtype=torch.int32, device="cuda")}
    q = torch.randn(1, 16, 128, generator=g, device="cuda")
    check_attention(c, q, 64, accumulate=False)


@pytest.mark.parametrize("size", [0.0, 30.0])
def test_attention_flat_and_peaked(size):
    """Queries of zeros (the mean of the values) and scores of hundreds."""
    c, g = ref.cache(5, [900, 64], 2, 128, 64)
    q = size * torch.randn(2, 16, 128, generator=g, device="cuda")
    check_attention(c, q, 64, accumulate=True)


def test_attention_scale():
    c, g = ref.cache(6, [300], 2, 128, 64)
    q = torch.randn(1, 16, 128, generator=g, device="cuda")
    check_attention(c, q, 64, accumulate=False, scale=-0.03)


def test_attention_lowest_values():
    """Keys that drive scores to the lowest values: a row whose scores are all
    about -1e38 is a softmax like any other."""
    c, g = ref.cache(7, [40], 1, 64, 16)
    q = torch.zeros(1, 2, 64, device="cuda")
    q[..., 0] = 2.0 ** 60
    pages = c["table"][0, :3].long()
    c["k"][pages] = 0.0
    c["k"][pages, :, :, 0] = -(2.0 ** 60)
    c["k"][pages[1], 3, 0, 0] = -(2.0 ** 59)
    out = qb.paged_attention(handle(c), q)
    torch.cuda.synchronize()
    # the one entry with half the (negative) score takes everything
    want = c["v"][pages[1], 3, 0].float()
    assert torch.equal(out[0, 0], want) and torch.equal(out[0, 1], want)


def test_attention_bad_pages_hold_nothing():
    c, g = ref.cache(8, [200, 50, 64], 2, 128, 16)
    q = torch.randn(3, 16, 128, generator=g, device="cuda")
    c["table"][0, 3] = -1
    c["table"][0, 12] = c["k"].shape[0]
    c["table"][2, :4] = 1 << 30  # every page of a sequence
    out = check_attention(c, q, 16, accumulate=True, status=-8)
    assert bool((out[2] == 0).all())


def test_attention_length_beyond_the_table():
    c, g = ref.cache(9, [64, 48], 2, 128, 16)
    c["table"][1, 3] = c["table"][0, 0]
    c["k"][c["table"][0, 0].long()] = 0.25
    c["v"][c["table"][0, 0].long()] = -0.5
    c["lens"].copy_(torch.tensor([-5, 1000]))
    q = torch.randn(2, 16, 128, generator=g, device="cuda")
    out = check_attention(c, q, 16, accumulate=False)
    assert bool((out[0] == 0).all())


def test_attention_offsets_beyond_32_bits():
    """Pages whose element offsets pass 2^31 (and byte offsets 2^32)."""
    page, kv, hd = 256, 2, 128
    pages = (1 << 31) // (page * kv * hd) + 5
    k = torch.empty(pages, page, kv, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(10)
    far = [pages - 1, 0, pages - 3]
    for p in far:
        for t in (k, v):
            t[p] = torch.randn(page, kv, hd, generator=g, device="cuda").to(torch.bfloat16)
    c = {"k": k, "v": v, "table": torch.tensor([far], dtype=torch.int32, device="cuda"),
         "lens": torch.tensor([700], dtype=torch.int32, device="cuda"), "weight": torch.zeros(1, kv, 768, device="cuda"),
         "pos": torch.arange(768, device="cuda").to(torch.int32).expand(1, kv, 768).contiguous()}
    q = torch.randn(1, 16, hd, generator=g, device="cuda")
    out = qb.paged_attention(handle(c), q, accumulate=True)
    torch.cuda.synchronize()
    small = {"k": k[far], "v": v[far], "table": torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")}
    want, received, bound = ref.attention(q, small["k"], small["v"], small["table"], c["lens"], page)
    close_out(out, want, bound, hd, float(small["v"].float().abs().max()))
    # append to and evict from the far pages too
    row = torch.randn(1, kv, hd, generator=g, device="cuda")
    at = torch.tensor([700], dtype=torch.int32, device="cuda")
    qb.paged_append(handle(c), row, row, at)
    assert torch.equal(k[pages - 3, 700 - 512], row[0].to(torch.bfloat16))
    c["weight"][:] = 0.0
    c["weight"][:, :, 690:] = 1.0
    last = k[pages - 3, 690 - 512:701 - 512].clone()
    qb.cache_evict(handle(c), None, 256)
    assert torch.equal(k[pages - 1, 245:256], last)
    assert int(c["lens"][0]) == 256


def test_attention_repeats_and_streams():
    c, g = ref.cache(11, [5000, 77, 1200], 2, 128, 64)
    q = torch.randn(3, 16, 128, generator=g, device="cuda")
    weight = c["weight"].clone()
    first = qb.paged_attention(handle(c), q, accumulate=True)
    first_w = c["weight"].clone()
    c["weight"].copy_(weight)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ws = qb.paged_attention_workspace(handle(c), 16, True)
    ws.fill_(0xFF)  # nothing in the workspace has to start at a value
    out = torch.empty_like(q)
    side.wait_stream(torch.cuda.current_stream())
    qb.paged_attention(handle(c), q, out=out, accumulate=True, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(first, out) and torch.equal(first_w, c["weight"])
    # captured into a graph and replayed
    c["weight"].copy_(weight)
    graph, h = torch.cuda.CUDAGraph(), handle(c)
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qb.paged_attention(h, q, out=out, accumulate=True, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out) and torch.equal(first_w, c["weight"])


def test_attention_query_in_place():
    c, g = ref.cache(12, [400, 3], 2, 128, 64)
    q = torch.randn(2, 16, 128, generator=g, device="cuda")
    want = qb.paged_attention(handle(c), q)
    qb.paged_attention(handle(c), q, out=q)
    assert torch.equal(q, want)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,hd", LAYOUTS)
@pytest.mark.parametrize("theta", [0.0, 1e7])
def test_append_rows(heads, kv, hd, dtype, theta):
    lens = [0, 5, 16, 40]
    c, g = ref.cache(20, [80] * 4, kv, hd, 16)
    c["lens"].copy_(torch.tensor(lens))
    rows = [(b, s) for b, n in enumerate(lens) for s in range(n, n + 7)] + [(1, -1), (2, 79), (0, -7)]
    order = torch.randperm(len(rows), generator=g, device="cuda").tolist()
    rows = [rows[i] for i in order]
    seq = torch.tensor([r[0] for r in rows], dtype=torch.int32, device="cuda")
    slot = torch.tensor([r[1] for r in rows], dtype=torch.int32, device="cuda")
    pos = torch.randint(0, 1 << 20, (len(rows),), generator=g, device="cuda").to(torch.int32)
    pos[0] = 0
    k, v = (torch.randn(len(rows), kv, hd, generator=g, device="cuda").to(dtype) for _ in "kv")
    q = torch.randn(len(rows), heads, hd, generator=g, device="cuda").to(dtype)
    want = {name: t.clone() for name, t in c.items()}
    h = handle(c)
    q_out = qb.paged_append(h, k, v, pos, q=q, seq=seq, slot=slot, rope_theta=theta)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    # single-precision sine and cosine of an angle reduced in double: 2^-20
    # absolute covers the reduction's rounding to fp32 (2^-23 of pi) and the
    # functions; the products round once more; then the type's half step
    def near(got, exact):
        half = torch.finfo(got.dtype).eps / 2
        if theta == 0:
            tol = half * exact.abs()
        else:
            size = torch.cat([exact[..., :hd // 2].hypot(exact[..., hd // 2:])] * 2, dim=-1)
            tol = half * exact.abs() + (2.0 ** -20 + 2.0 ** -22) * 1.5 * size
        return bool(((got.double() - exact).abs() <= tol).all())

    assert near(q_out, ref.rotated(q, pos, theta))
    kr = ref.rotated(k, pos, theta)
    for i, (b, s) in enumerate(rows):
        if s < 0:
            continue
        p = int(c["table"][b, s // 16])
        assert near(c["k"][p, s % 16], kr[i])
        assert torch.equal(c["v"][p, s % 16], v[i].to(torch.bfloat16))
        want["k"][p, s % 16] = c["k"][p, s % 16]
        want["v"][p, s % 16] = v[i].to(torch.bfloat16)
        want["weight"][b, :, s] = 0
        want["pos"][b, :, s] = pos[i]
        want["lens"][b] = max(int(want["lens"][b]), s + 1)
    for name in c:  # and nothing else was written
        a, b = c[name], want[name]
        if a.dtype == torch.bfloat16:
            a, b = a.contiguous().view(torch.int16), b.contiguous().view(torch.int16)
        assert torch.equal(a, b), name


@pytest.mark.parametrize("n_seqs", [1, 3, 300])
def test_append_next_entries(n_seqs):
    """Without slots each sequence grows by one; q may be turned in place."""
    lens = [(7 * b) % 40 for b in range(n_seqs)]
    c, g = ref.cache(21, [64] * n_seqs, 2, 128, 16)
    c["lens"].copy_(torch.tensor(lens))
    h = handle(c)
    for step in range(3):
        k, v = (torch.randn(n_seqs, 2, 128, generator=g, device="cuda") for _ in "kv")
        q = torch.randn(n_seqs, 16, 128, generator=g, device="cuda")
        pos = torch.tensor([n + 1000 * step for n in lens], dtype=torch.int32, device="cuda")
        apart = qb.paged_append(h, k, v, pos, q=q, seq=torch.arange(n_seqs, dtype=torch.int32, device="cuda"),
                                slot=c["lens"].clone(), rope_theta=1e4)
        c["lens"].sub_(1)
        qb.paged_append(h, k, v, pos, q=q, q_out=q, rope_theta=1e4)
        assert torch.equal(q, apart)
        lens = [n + 1 for n in lens]
        assert c["lens"].tolist() == lens
        for b in (0, n_seqs - 1):
            p = int(c["table"][b, (lens[b] - 1) // 16])
            assert torch.equal(c["v"][p, (lens[b] - 1) % 16], v[b].to(torch.bfloat16))
    assert qb.query_status() == 0


def test_append_many_rows():
    """A prompt of every slot of its sequence, in order and shuffled."""
    n, page = 3001, 64
    c, g = ref.cache(22, [n, 10], 2, 128, page)
    c["lens"].zero_()
    for shuffled in (False, True):
        slot = torch.arange(n, device="cuda")
        if shuffled:
            slot = slot[torch.randperm(n, generator=g, device="cuda")]
        slot = slot.to(torch.int32)
        k, v = (torch.randn(n, 2, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
        seq = torch.zeros(n, dtype=torch.int32, device="cuda")
        c["lens"].zero_()
        qb.paged_append(handle(c), k, v, slot + 5, seq=seq, slot=slot)
        assert c["lens"].tolist() == [n, 0]
        where = c["table"][0].long()[slot.long() // page], slot.long() % page
        assert torch.equal(c["k"][where], k) and torch.equal(c["v"][where], v)
        assert torch.equal(c["pos"][0, 1, slot.long()], slot + 5)


def test_append_bad_rows():
    c, g = ref.cache(23, [30, 30], 2, 128, 16)
    c["table"][1, 0] = -1
    before = {name: t.clone() for name, t in c.items()}
    k = torch.randn(5, 2, 128, generator=g, device="cuda")
    seq = torch.tensor([2, -1, 0, 1, 0], dtype=torch.int32, device="cuda")
    slot = torch.tensor([0, 0, 32, 3, 1 << 30], dtype=torch.int32, device="cuda")
    qb.paged_append(handle(c), k, k, seq, seq=seq, slot=slot)
    torch.cuda.synchronize()
    assert qb.query_status() == -8
    for name in c:
        assert torch.equal(torch.nan_to_num(c[name].float()), torch.nan_to_num(before[name].float())), name
    # a full sequence has no next entry
    c["lens"].copy_(torch.tensor([32, 31]))
    c["table"][1] = c["table"][0]
    qb.paged_append(handle(c), k[:2], k[:2], seq[:2])
    torch.cuda.synchronize()
    assert qb.query_status() == -8
    assert c["lens"].tolist() == [32, 32]


# ---------------------------------------------------------------- evict

def check_evict(c, page, budget, recent, next_pos, in_place, with_pos=True):
    h = handle(c, with_pos)
    before = {name: t.clone() for name, t in c.items()}
    lens = before["lens"].tolist()
    if in_place:
        new = {"lens": c["lens"], "weight": c["weight"], "pos": c["pos"] if with_pos else None}
        qb.cache_evict(h, next_pos, budget, recent)
    else:
        new = {"lens": torch.full_like(c["lens"], -3), "weight": torch.full_like(c["weight"], -3.0),
               "pos": torch.full_like(c["pos"], -3) if with_pos else None}
        qb.cache_evict(h, next_pos, budget, recent, new["lens"], new["weight"], new["pos"])
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    want = {name: t.clone() for name, t in before.items()}
    slots = c["weight"].shape[2]
    for b, n in enumerate(lens):
        n = max(0, min(n, slots))
        m = min(n, budget)
        assert int(new["lens"][b]) == m
        for g in range(c["k"].shape[2]):
            first = int(next_pos[b]) - recent if recent else None
            _, moves = ref.evict(before["weight"][b, g], before["pos"][b, g], n, budget, first)
            for name in ("weight", "pos"):
                if new[name] is None:
                    continue
                row = before[name][b, g].clone()
                for src, dst in moves:
                    row[dst] = before[name][b, g, src]
                tail = before[name][b, g, m:] if in_place else torch.full_like(row[m:], -3)
                assert torch.equal(torch.nan_to_num(new[name][b, g, :m].float(), nan=-9.0), torch.nan_to_num(row[:m].float(), nan=-9.0))
                assert torch.equal(torch.nan_to_num(new[name][b, g, m:].float(), nan=-9.0), torch.nan_to_num(tail.float(), nan=-9.0))
            if moves:
                src, dst = (torch.tensor(x, device="cuda") for x in zip(*moves))
                t = before["table"][b].long()
                for name in ("k", "v"):
                    want[name][t[dst // page], dst % page, g] = before[name][t[src // page], src % page, g]
    for name in ("k", "v"):
        a, b = (x.contiguous().view(torch.int16) for x in (c[name], want[name]))
        assert torch.equal(a, b), name


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget,recent", [(0, 0), (1, 0), (1, 1), (64, 10), (100, 100), (257, 31), (5000, 64)])
def test_evict_budgets(budget, recent, in_place):
    lens = [0, 1, 63, 64, 65, 300, 1500]
    c, g = ref.cache(30, lens, 2, 64, 16)
    next_pos = torch.tensor([1500] * 7, dtype=torch.int32, device="cuda")
    check_evict(c, 16, budget, recent, next_pos, in_place)


@pytest.mark.parametrize("kind", ["equal", "few", "nan", "inf", "zeros", "negative", "tiny"])
def test_evict_ties_and_special_weights(kind):
    c, g = ref.cache(31, [700, 900, 40], 2, 64, 16)
    w = c["weight"]
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "few":
        w.copy_(torch.randint(0, 3, w.shape, generator=g, device="cuda").float())
    elif kind == "nan":
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.6] = math.nan
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.2] = -math.inf
    elif kind == "inf":
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.5] = math.inf
    elif kind == "zeros":
        w.copy_(torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.5, 0.0, -0.0))
    elif kind == "negative":
        w.sub_(0.5)
    else:  # denormal numbers differ in their order too
        w.mul_(1e-40)
    next_pos = torch.full((3,), 900, dtype=torch.int32, device="cuda")
    check_evict(c, 16, 333, 20, next_pos, in_place=False)


@pytest.mark.parametrize("n,budget", [(4097, 4096), (4100, 4096), (33000, 8192), (70001, 69000), (70001, 300), (100001, 2000)])
def test_evict_long(n, budget):
    c, g = ref.cache(32, [n], 1, 64, 64)
    next_pos = torch.tensor([c["pos"].shape[2]], dtype=torch.int32, device="cuda")
    check_evict(c, 64, budget, min(128, budget), next_pos, in_place=True)


@pytest.mark.parametrize("budget", [399990, 150000])
def test_evict_longest(budget):
    """More slots than a cluster's shared memory holds keys of, with equal weights
    on both sides of that border."""
    n = 400001
    c, g = ref.cache(37, [n], 1, 8, 64)
    c["weight"].copy_(torch.floor(c["weight"] * 50))
    next_pos = torch.tensor([c["pos"].shape[2]], dtype=torch.int32, device="cuda")
    check_evict(c, 64, budget, 1000, next_pos, in_place=False)
    c["weight"][0, 0, 100:] = 7.0
    check_evict(c, 64, budget, 0, None, in_place=True, with_pos=False)


@pytest.mark.parametrize("layout", ["heads", "both"])
@pytest.mark.parametrize("kv,hd", [(2, 128), (3, 200), (8, 8)])
def test_evict_layouts(layout, kv, hd):
    c, g = ref.cache(33, [90, 200], kv, hd, 8, layout=layout)
    check_evict(c, 8, 61, 0, None, in_place=True, with_pos=False)


def test_evict_many_sequences():
    lens = [(37 * b) % 300 for b in range(120)]
    c, g = ref.cache(34, lens, 2, 64, 16)
    next_pos = torch.full((120,), 304, dtype=torch.int32, device="cuda")
    check_evict(c, 16, 100, 25, next_pos, in_place=True)


def test_evict_bad_page():
    """An entry that should move but has no page stays out; the rest goes on."""
    c, g = ref.cache(35, [64], 1, 64, 16)
    c["weight"].zero_()
    c["weight"][0, 0, 30:34] = 1.0
    c["table"][0, 2] = -1  # slots 32..47
    pages = c["table"][0].long()
    moved = c["k"][pages[1], 14:16, 0].clone()
    qb.cache_evict(handle(c), None, 4)
    torch.cuda.synchronize()
    assert qb.query_status() == -8
    assert int(c["lens"][0]) == 4
    assert torch.equal(c["k"][pages[0], :2, 0], moved)


def test_evict_then_append_then_attend():
    """The operators in turn, as a bounded cache runs: after each eviction the
    attention equals that over the entries that stay."""
    n, page, budget = 200, 16, 150
    c, g = ref.cache(36, [n, 130], 2, 128, page)
    h = handle(c)
    c["weight"].zero_()
    c["pos"].copy_(torch.arange(c["pos"].shape[2], device="cuda").to(torch.int32).expand_as(c["pos"]))
    nxt = torch.tensor([n, 130], dtype=torch.int32, device="cuda")
    for step in range(6):
        if step:
            row = torch.randn(2, 2, 128, generator=g, device="cuda")
            qb.paged_append(h, row, row, nxt, rope_theta=1e6)
            nxt += 1
        q = torch.randn(2, 16, 128, generator=g, device="cuda")
        check_attention(c, q, page, accumulate=True)
        check_evict(c, page, budget, 16, nxt, in_place=True)
        for b in range(2):
            for kvh in range(2):
                held = c["pos"][b, kvh, :int(c["lens"][b])].tolist()
                assert len(set(held)) == len(held)
                assert set(range(int(nxt[b]) - 16, int(nxt[b]))) <= set(held)
    assert c["lens"].tolist() == [150, 135]
