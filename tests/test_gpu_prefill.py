"""Attention of packed rows over the paged cache against a plain 64-bit one.

The cases take the lengths at which pages, key blocks of 128, query tiles and the
split of long axes begin and end, sequences without rows and rows without
entries, several head layouts, pools in three memory layouts, rows of nobody, and
pools that hold NaN wherever no entry lies.

Tolerances. A score is a sum of hd products held in fp32: its rounding is at most
(hd + 8) 2^-24 of sum |q k| scale, which moves a probability by at most twice
that, relative to itself, and so an output by at most twice that times sum p |v|.
fp32 rows: probabilities are split into three bf16 parts (2^-24), sums of a block of
128 keys are cut off by the tensor cores at each of 24 steps (2^-23 each), the
blocks' sums rounded (n / 128 times 2^-24), all below 2^-16 of sum p |v| for the
lengths here. bf16 rows: a probability is rounded once, 2^-8 of itself; sums are
cut off at each of n / 16 steps (2^-23 each); the result is rounded once, 2^-8 of
itself.
"""

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from tests import prefill_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


def pool(total, page, kv, hd, layout):
    """A pool of NaN: contiguous, heads outside the slots, or inside a wider buffer."""
    nan = float("nan")
    if layout == "heads":
        return torch.full((total, kv, page, hd), nan, device="cuda", dtype=torch.bfloat16).permute(0, 2, 1, 3)
    if layout == "wide":
        return torch.full((total, page, kv, hd + 24), nan, device="cuda", dtype=torch.bfloat16)[..., 8:8 + hd]
    return torch.full((total, page, kv, hd), nan, device="cuda", dtype=torch.bfloat16)


def make(counts, lens, heads, kv, hd, page, dtype, layout="plain", seed=0, gap=0, spread=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000 * hd + len(counts))
    used = [-(-m // page) for m in lens]
    total = max(1, sum(used)) + 2
    perm = torch.randperm(total, generator=g, device="cuda").int()
    width = max(1, max(used)) + 1
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    k, v = pool(total, page, kv, hd, layout), pool(total, page, kv, hd, layout)
    at = 0
    for b, (m, u) in enumerate(zip(lens, used)):
        table[b, :u] = perm[at:at + u]
        table[b, u:] = 1 << 30  # behind the last page: not read
        for t in (k, v):
            for j in range(u):
                n = min(page, m - j * page)
                t[int(perm[at + j]), :n] = torch.randn(n, kv, hd, generator=g, device="cuda").to(torch.bfloat16)
        at += u
    first, r = [], gap
    for n in counts:
        first.append(r)
        r += max(n, 0) + gap
    q = (torch.randn(r + 3, heads, hd, generator=g, device="cuda") * spread).to(dtype)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return dict(k=k, v=v, table=table, lens=i32(lens), first=i32(first), count=i32(counts), q=q)


def run(c, **kw):
    cache = qb.PagedCache(c["k"], c["v"], c["table"], c["lens"])
    out = torch.full_like(c["q"], 7.0)
    qb.paged_prefill_attention(cache, c["q"], c["first"], c["count"], out=out, **kw)
    torch.cuda.synchronize()
    return out


def check(c, page, status=0, scale=None):
    out = run(c, scale=0.0 if scale is None else scale)
    assert qb.query_status() == status
    want, mean, bound = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["first"], c["count"], page, scale)
    mine = ~torch.isnan(want)
    assert bool((out[~mine] == 7.0).all()), "rows of nobody were written"
    got, want, mean = out.double()[mine], want[mine], mean[mine]
    hd, longest = c["q"].shape[2], int(c["lens"].max())
    tol = (2 * (hd + 8) * 2.0 ** -24 * bound + 2.0 ** -16) * mean
    if out.dtype == torch.bfloat16:
        tol = tol + (2.0 ** -8 + longest / 16 * 2.0 ** -23) * mean + 2.0 ** -8 * want.abs()
    assert bool(torch.isfinite(got).all())
    assert bool(((got - want).abs() <= tol + 1e-30).all()), float(((got - want).abs() / (tol + 1e-30)).max())
    return out


DTYPES = [torch.float32, torch.bfloat16]
HEADS = [(16, 2, 128), (8, 8, 64), (8, 1, 128), (12, 4, 96), (20, 2, 128), (4, 4, 8), (6, 2, 40), (8, 2, 256), (3, 1, 200),
         (2, 2, 72), (160, 1, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv,hd", HEADS)
def test_head_layouts(heads, kv, hd, dtype):
    check(make([37, 0, 1, 130], [37, 64, 300, 290], heads, kv, hd, 32, dtype), 32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [8, 16, 64, 128, 512])
@pytest.mark.parametrize("counts,lens", [
    ([1], [1]), ([128], [128]), ([129], [129]), ([127, 128, 1], [127, 257, 128]), ([16, 17, 15, 33], [16, 145, 143, 33]),
    ([300], [1000]), ([5, 0, 0, 2], [5, 0, 3, 900])])
def test_lengths_and_pages(page, counts, lens, dtype):
    check(make(counts, lens, 16, 2, 128, page, dtype, seed=page), page)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("layout", ["plain", "heads", "wide"])
@pytest.mark.parametrize("hd", [64, 128])
def test_pool_layouts(layout, hd, dtype):
    check(make([70, 9], [70, 200], 8, 2, hd, 16, dtype, layout), 16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,m", [(1, 5000), (16, 4100), (40, 9001), (700, 2500)])
def test_few_rows_on_a_long_axis(n, m, dtype):
    check(make([n], [m], 16, 2, 128, 64, dtype), 64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_sequences(dtype):
    counts = [(37 * i) % 23 if i % 3 else 1 for i in range(200)]
    lens = [n + (101 * i) % 400 for i, n in enumerate(counts)]
    check(make(counts, lens, 8, 2, 64, 16, dtype, gap=1), 16)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_without_entries_give_zeros(dtype):
    """More rows than entries: the first ones see nothing; a length below 0 or a sequence without
    entries leaves all rows with nothing."""
    c = make([6, 3, 4], [4, 0, 0], 16, 2, 128, 16, dtype)
    c["lens"][2] = -5
    out = check(c, 16)
    assert bool((out[0:2] == 0).all()) and bool((out[6:13] == 0).all()) and bool((out[2:6] != 0).any())


@pytest.mark.parametrize("dtype", DTYPES)
def test_padded_batch_and_rows_in_any_order(dtype):
    c = make([20, 150, 3], [20, 150, 90], 16, 2, 128, 32, dtype, gap=40)
    check(c, 32)
    order = torch.tensor([2, 0, 1], device="cuda")
    for n in ("table", "lens", "first", "count"):
        c[n] = c[n][order].contiguous()
    check(c, 32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_out_of_range_are_reported(dtype):
    c = make([20, 30, 5], [20, 60, 5], 16, 2, 128, 32, dtype)
    c["first"][1] = c["q"].shape[0] - 29
    check(c, 32, status=-8)
    c["first"][1] = -1
    check(c, 32, status=-8)
    c["count"][1] = -7
    check(c, 32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [16, 128])
def test_pages_out_of_range_hold_nothing(page, dtype):
    c = make([40, 10], [400, 10], 16, 2, 128, page, dtype)
    c["table"][0, 1] = -3
    c["table"][0, 2] = c["k"].shape[0]
    c["table"][1, 0] = 1 << 29
    out = check(c, page, status=-8)
    assert bool((out[40:50] == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1.0, -0.5, 1e-3])
def test_scales(scale, dtype):
    check(make([150], [333], 16, 2, 128, 32, dtype), 32, scale=scale)


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_scores(dtype):
    """Scores of thousands: the softmax is one entry, and its reference moves far."""
    check(make([200], [900], 16, 2, 128, 64, dtype, spread=300.0), 64)


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place_and_again(dtype):
    c = make([90, 7], [300, 500], 16, 2, 128, 64, dtype)
    want = run(c)
    again = run(c)
    assert torch.equal(want, again)
    cache = qb.PagedCache(c["k"], c["v"], c["table"], c["lens"])
    q = c["q"].clone()
    qb.paged_prefill_attention(cache, q, c["first"], c["count"], out=q)
    n = int(c["count"].sum())
    assert torch.equal(q[:n], want[:n]) and torch.equal(q[n:], c["q"][n:])


def test_on_a_stream_and_in_a_graph():
    """A captured call follows the lengths that its arrays hold when it is replayed; two graphs share a workspace in turn."""
    a = make([90, 7], [300, 500], 16, 2, 128, 64, torch.bfloat16)
    b = make([16], [4100], 16, 2, 128, 64, torch.bfloat16, seed=3)
    want = [run(c) for c in (a, b)]
    caches = [qb.PagedCache(c["k"], c["v"], c["table"], c["lens"]) for c in (a, b)]
    ws = max((qb.paged_prefill_attention_workspace(h, c["q"].shape[0], 16) for h, c in zip(caches, (a, b))), key=lambda t: t.numel())
    outs, graphs, side = [torch.full_like(c["q"], 7.0) for c in (a, b)], [], torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for h, c, o in zip(caches, (a, b), outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            qb.paged_prefill_attention(h, c["q"], c["first"], c["count"], out=o, ws=ws)
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            o.fill_(7.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    a["lens"][0], a["count"][0] = 250, 40
    shorter = run(a)
    outs[0].fill_(7.0)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], shorter)


def test_agrees_with_the_decoding_call():
    """One row of each sequence: paged_attention's outputs, up to both calls' roundings of fp32 rows."""
    c = make([1] * 5, [1, 64, 300, 1000, 77], 16, 2, 128, 64, torch.float32)
    cache = qb.PagedCache(c["k"], c["v"], c["table"], c["lens"])
    got = run(c)[:5]
    want = qb.paged_attention(cache, c["q"][:5].contiguous())
    _, mean, bound = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["first"], c["count"], 64)
    tol = 2 * (2 * 136 * 2.0 ** -24 * bound + 2.0 ** -16) * mean[:5]
    assert bool(((got - want).abs().double() <= tol).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,kv,hd", [(8, 2, 256), (6, 2, 200), (300, 2, 64), (40, 1, 144)])
def test_in_place_where_tiles_share_their_queries(heads, kv, hd, dtype):
    """Heads of more than 128 dims, or groups of more than a block's rows, are several tiles of the same rows."""
    c = make([150, 33], [700, 40], heads, kv, hd, 32, dtype, seed=4)
    want = run(c)
    cache = qb.PagedCache(c["k"], c["v"], c["table"], c["lens"])
    for _ in range(3):
        q = c["q"].clone()
        qb.paged_prefill_attention(cache, q, c["first"], c["count"], out=q)
        n = int(c["count"].sum())
        assert torch.equal(q[:n], want[:n]) and torch.equal(q[n:], c["q"][n:])
    q = c["q"].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qb.paged_prefill_attention(cache, q, c["first"], c["count"], out=q)
    for _ in range(3):
        q.copy_(c["q"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q[:n], want[:n]) and torch.equal(q[n:], c["q"][n:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs", [33, 600, 1100])
def test_a_batch_of_single_rows(seqs, dtype):
    """More sequences than lanes, than SMs and than 32 a lane, some without rows."""
    lens = [1 + (53 * i) % 90 for i in range(seqs)]
    check(make([0 if i % 7 == 3 else 1 for i in range(seqs)], lens, 4, 2, 64, 32, dtype), 32)


def test_two_streams_at_once():
    a = make([400, 90], [900, 90], 16, 2, 128, 64, torch.bfloat16)
    b = make([300], [3000], 16, 2, 128, 32, torch.float32, seed=9)
    want = [run(c) for c in (a, b)]
    caches = [qb.PagedCache(c["k"], c["v"], c["table"], c["lens"]) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for c, h, st in zip((a, b), caches, streams):
            with torch.cuda.stream(st):
                out = torch.full_like(c["q"], 7.0)
            outs.append(qb.paged_prefill_attention(h, c["q"], c["first"], c["count"], out=out, stream=st))
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert qb.query_status() == 0


def test_offsets_past_32_bits():
    """Rows and pages whose elements lie behind the first 2^31: as the same rows and pages at the front."""
    heads, kv, hd, page, many = 16, 2, 128, 64, 2 ** 17 + 9
    c = make([70, 5], [300, 5], heads, kv, hd, page, torch.bfloat16)
    want = run(c)
    rows = 2 ** 20 + 100
    shift, pages = rows - c["q"].shape[0], c["k"].shape[0]
    pools = [torch.empty(many + pages, page, kv, hd, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for big, small in zip(pools, (c["k"], c["v"])):
        big[many:] = small
    table = torch.where(c["table"] < pages, c["table"] + many, c["table"])
    q = torch.zeros(rows, heads, hd, dtype=torch.bfloat16, device="cuda")
    q[shift:] = c["q"]
    assert q.numel() > 2 ** 31 and pools[0].numel() > 2 ** 31
    out = qb.paged_prefill_attention(qb.PagedCache(*pools, table, c["lens"]), q, c["first"] + shift, c["count"])
    n = int(c["count"].sum())
    assert torch.equal(out[shift:shift + n], want[:n]) and not bool(out[:shift].any()) and not bool(out[shift + n:].any())


@pytest.mark.parametrize("dtype", DTYPES)
def test_pages_of_4096(dtype):
    check(make([200, 4097], [9000, 4097], 4, 2, 64, 4096, dtype), 4096)
