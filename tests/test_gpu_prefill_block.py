"""Prompts into the paged cache as a serving program brings them: plan, block over packed
rows, decoding, eviction, pages given back. Against the fp64 oracle, the contiguous path
and the decoding call.

"CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
Now Splits": the block (16 query heads, 2 KV heads, head_dim 128).
"""

import time

import numpy as np
import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from quantized_moe_transformer_gb300 import inputs
from tests.parity import GAP, TOL_GEMV, TOL_TC, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def blk_pair():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()
    arr = inputs.block(5, ctx=1024)
    return arr, qb.Block.from_arrays(arr, 8)


@pytest.fixture
def fp32_projections():
    old = qb.get_gemm_threshold()
    qb.set_gemm_threshold(1 << 20)
    yield
    qb.set_gemm_threshold(old)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """A cache, its pool and the sequences' next positions."""

    def __init__(self, n_seqs, pages, page=16, max_len=256):
        self.cache = qb.PagedCache.empty(n_seqs, max_len, 2, 128, page=page, n_pages=pages)
        self.pool = qb.PagePool.full(self.cache)
        self.next = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")

    def plan(self, counts, keep=None, n_rows=None):
        rows = sum(counts) if n_rows is None else n_rows
        got = qb.paged_plan(self.cache, self.pool, i32(counts), keep=None if keep is None else i32(keep), next_pos=self.next,
                            n_rows=rows)
        self.next += got[1]
        return got

    def step(self, blk, X, counts, **kw):
        first, granted, seq, slot, pos = self.plan(counts, n_rows=X.shape[0], **kw)
        return qb.block_prefill_paged(blk, self.cache, X, first, granted, seq, slot, pos)


def rows(seed, n):
    return torch.from_numpy(inputs.hidden(seed, n, 2048)).cuda()


def test_prompts_against_the_oracle(oracle, blk_pair, fp32_projections):
    """Sequences of 37, 0, 18 and 5 rows packed together; rows of each against the oracle's block for that sequence alone."""
    arr, blk = blk_pair
    counts = [37, 0, 18, 5]
    X = inputs.hidden(201, sum(counts), 2048)
    s = Server(4, 20)
    out = s.step(blk, torch.from_numpy(X).cuda(), counts).cpu().numpy()
    assert qb.query_status() == 0 and s.cache.lens.tolist() == counts
    at = 0
    for n in counts:
        if n:
            x = X[at:at + n]
            which = np.array(sorted({0, n // 2, n - 1}))
            kc, vc = (np.zeros((n, 2, 128)) for _ in "kv")
            ref, parts = oracle.block_forward_rows(x, arr, 8, 0, kc, vc, which)
            assert_close(out[at:at + n][which], ref, TOL_GEMV, rows=parts["gap"] >= GAP)
        at += n


def test_in_parts(blk_pair, fp32_projections):
    """A prompt in parts of 1, 40, 3 and 20 rows, beside another sequence's, equals the prompt at once: the same sums
    but for where the key blocks are cut (fp32)."""
    _, blk = blk_pair
    X, other = rows(202, 64), rows(203, 64)
    whole = Server(1, 8)
    want = whole.step(blk, X, [64])
    parts, at, got = Server(2, 12), 0, []
    for n in (1, 40, 3, 20):
        got.append(parts.step(blk, torch.cat([other[at:at + 5], X[at:at + n]]), [5, n])[5:])
        at += n
    assert qb.query_status() == 0
    assert_close(torch.cat(got).cpu().numpy(), want.cpu().numpy(), TOL_GEMV)
    a, b = (s.cache.k[s.cache.table[i, :4].long()].flatten(0, 1)[:64] for s, i in ((whole, 0), (parts, 1)))
    assert_close(a.float().cpu().numpy(), b.float().cpu().numpy(), TOL_GEMV)


@pytest.mark.parametrize("n", [40, 300])
def test_equals_the_contiguous_path(blk_pair, n):
    """Default projections on the tensor cores on both sides; the contiguous attention rounds its probabilities to bf16."""
    _, blk = blk_pair
    X = rows(204, n)
    kc, vc = (torch.zeros(n, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    want = qb.block_forward(blk, X, kc, vc, 0)
    s = Server(1, 40, max_len=512)
    got = s.step(blk, X, [n])
    assert qb.query_status() == 0
    flat = [t[s.cache.table[0, :-(-n // 16)].long()].flatten(0, 1)[:n] for t in (s.cache.k, s.cache.v)]
    assert torch.equal(flat[1], vc)
    # keys: the same projections turned by sines and cosines that both paths form in single precision, each off by
    # 2^-20 at most (two factors of a pair, on both sides: 2^-18 of the larger element of any pair), then two bf16
    # roundings of 2^-8 of the value each
    k, want_k = flat[0].double(), kc.double()
    assert bool(((k - want_k).abs() <= 2.0 ** -7 * want_k.abs() * (1 + 2.0 ** -7) + 2.0 ** -18 * want_k.abs().max() * 2).all())
    assert_close(got.cpu().numpy(), want.cpu().numpy(), TOL_TC)


def test_single_rows_equal_the_decoding_call(blk_pair):
    """One row of each sequence through both calls, then again: the same projections and experts, two attentions in fp32."""
    _, blk = blk_pair
    counts = [20, 3, 31]
    a, b = Server(3, 12), Server(3, 12)
    X = rows(205, sum(counts))
    for s in (a, b):
        s.step(blk, X, counts)
    for step in range(3):
        x = rows(206 + step, 3)
        got = a.step(blk, x, [1, 1, 1])
        first, granted, seq, slot, pos = b.plan([1, 1, 1])
        want = qb.block_decode_paged(blk, b.cache, x, pos)
        assert_close(got.cpu().numpy(), want.cpu().numpy(), TOL_GEMV)
        assert torch.equal(a.cache.lens, b.cache.lens) and torch.equal(a.cache.table, b.cache.table)
    assert qb.query_status() == 0


def test_rows_of_nobody_and_rows_not_granted(blk_pair):
    """Padding rows and a sequence that found no pages leave the cache alone and their rows come out without attention; the others are what they are without them."""
    _, blk = blk_pair
    X = rows(210, 60)
    s, alone = Server(3, 3), Server(3, 3)
    first, granted, seq, slot, pos = s.plan([20, 30, 2], n_rows=60)
    assert granted.tolist() == [20, 0, 0]
    got = qb.block_prefill_paged(blk, s.cache, X, first, granted, seq, slot, pos)
    want = alone.step(blk, X[:20].contiguous(), [20, 0, 0])
    assert s.cache.lens.tolist() == [20, 0, 0] and qb.query_status() == 0
    assert bool(torch.isfinite(got).all())
    assert_close(got[:20].cpu().numpy(), want.cpu().numpy(), TOL_TC)
    lone = qb.block_prefill_paged(blk, s.cache, X[20:].contiguous(), i32([0, 0, 0]), i32([0, 0, 0]), i32([-1] * 40), i32([-1] * 40), i32([0] * 40))
    assert_close(got[20:].cpu().numpy(), lone.cpu().numpy(), TOL_TC)


def test_a_descriptor_in_place_of_theta(blk_pair, fp32_projections):
    """The block's own rotation as a descriptor, and another one, which changes the result."""
    _, blk = blk_pair
    X = rows(211, 24)
    outs = []
    for r in (None, qb.Rope(128, 1e7), qb.Rope(128, 1e7, layout="interleaved")):
        s = Server(1, 4)
        plan = s.plan([24])
        outs.append(qb.block_prefill_paged(blk, s.cache, X, *plan, rope=r).cpu().numpy())
    assert_close(outs[1], outs[0], TOL_GEMV)
    assert np.abs(outs[2] - outs[0]).max() > 0.05 * np.abs(outs[0]).max()


def test_a_served_day(blk_pair):
    """Prompts, steps with accumulated weights and eviction, a sequence that ends and gives its pages to the next: lengths, pages
    and positions stay in order, and what a later prompt computes is what it computes alone."""
    _, blk = blk_pair
    s = Server(3, 14)
    s.step(blk, rows(220, 90), [60, 30, 0])
    for step in range(6):
        first, granted, seq, slot, pos = s.plan([1, 1, 0], keep=s.cache.lens.tolist())
        assert granted.tolist() == [1, 1, 0]
        first_pos = (s.next - granted).contiguous()
        out = qb.block_prefill_paged(blk, s.cache, rows(230 + step, 2), first, granted, seq, slot, pos)
        assert bool(torch.isfinite(out).all())
        qb.paged_attention(s.cache, torch.randn(3, 16, 128, device="cuda"), accumulate=True)
        qb.cache_evict(s.cache, s.next, 40, 8)
        assert int(first_pos[0]) == 60 + step
    assert s.cache.lens.tolist() == [40, 36, 0]
    X = rows(240, 50)
    # sequence 1 ends; 0 gives back what eviction left empty; 2 comes
    s.next[1] = 0
    out = s.step(blk, X, [0, 0, 50], keep=[40, 0, -1])
    assert s.cache.lens.tolist() == [40, 0, 50] and int(s.pool.n_free) == 14 - 3 - 4
    owned = s.cache.table[s.cache.table >= 0].tolist()
    assert len(owned) == 7 and len(set(owned + s.pool.free[:7].tolist())) == 14
    assert_close(out.cpu().numpy(), Server(1, 4).step(blk, X, [50]).cpu().numpy(), TOL_GEMV)
    assert qb.query_status() == 0


def test_step_in_a_graph(blk_pair):
    """Plan and block captured together; replays take the pages and lengths as they then are."""
    _, blk = blk_pair
    s, eager = Server(2, 10), Server(2, 10)
    X = rows(250, 12)
    counts, ends = i32([8, 4]), i32([-1, -1])
    for t in (s, eager):
        t.step(blk, X, [8, 4])
    ws = qb.block_prefill_paged_workspace(blk, s.cache, 12)
    pws = qb.paged_plan_workspace(s.cache)
    out = torch.empty_like(X)
    maps = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (2, 2, 12, 12, 12)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        qb.paged_plan(s.cache, s.pool, counts, keep=ends, n_rows=12, first=maps[0], granted=maps[1], seq=maps[2], slot=maps[3],
                      pos=maps[4], ws=pws)
        qb.block_prefill_paged(blk, s.cache, X, *maps, out=out, ws=ws)
    for step in range(3):
        X.copy_(rows(251 + step, 12))
        graph.replay()
        first, granted, seq, slot, pos = qb.paged_plan(eager.cache, eager.pool, counts, keep=ends, n_rows=12)
        want = qb.block_prefill_paged(blk, eager.cache, X, first, granted, seq, slot, pos)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.equal(s.cache.table, eager.cache.table) and s.cache.lens.tolist() == [32, 16]
    assert qb.query_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_withheld_copy_times_out(dtype):
    """Keys that never come end the waits after their limit: the status says so and the next call is right again."""
    cache = qb.PagedCache.empty(2, 1024, 2, 128)
    cache.k.normal_()
    cache.v.normal_()
    cache.lens[:] = i32([700, 300])
    q = torch.randn(400, 16, 128, device="cuda").to(dtype)
    args = (cache, q, i32([0, 300]), i32([300, 100]))
    want = qb.paged_prefill_attention(*args)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    qb.test_inject("prefill_copy", 2000)
    try:
        t0 = time.perf_counter()
        qb.paged_prefill_attention(*args)
        assert qb.query_status() == -7
        assert time.perf_counter() - t0 < 5.0
    finally:
        qb.test_inject("none")
    got = qb.paged_prefill_attention(*args)
    assert qb.query_status() == 0 and torch.equal(got, want)


def test_a_wait_that_runs_out_behind_the_first_warp_is_reported():
    """The second block of rows of a tile gives up when the first block's warps have stored theirs and left."""
    cache = qb.PagedCache.empty(1, 1024, 2, 128)
    cache.k.normal_()
    cache.v.normal_()
    cache.lens[:] = i32([32])
    q = torch.randn(32, 16, 128, device="cuda").to(torch.bfloat16)
    args = (cache, q, i32([0]), i32([32]))
    want = qb.paged_prefill_attention(*args)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    qb.test_inject("prefill_final", 2000)
    try:
        t0 = time.perf_counter()
        got = qb.paged_prefill_attention(*args)
        assert qb.query_status() == -7
        assert time.perf_counter() - t0 < 5.0
    finally:
        qb.test_inject("none")
    assert torch.equal(got[:16], want[:16])
    got = qb.paged_prefill_attention(*args)
    assert qb.query_status() == 0 and torch.equal(got, want)
