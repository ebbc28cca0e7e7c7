"""One new token for several sequences at once through the block and the paged
cache (append, attention, eviction) against the fp64 oracle and against plain
attention over the entries that stay.

"CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
Now Splits": the block (16 query heads, 2 KV heads, head_dim 128).
"""

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


def filled(arr, lens, page=64):
    """A paged cache whose sequence b holds the first lens[b] entries of the seeded
    contiguous cache rolled by b, and those contiguous caches."""
    cache = qb.PagedCache.empty(len(lens), 1024, 2, 128, page=page)
    kc, vc = (qb.cache_from_bits(arr[n]) for n in ("k_cache", "v_cache"))
    flat = []
    for b, n in enumerate(lens):
        k, v = kc.roll(b, 0).contiguous(), vc.roll(b, 0).contiguous()
        flat.append((k, v))
        if n:
            at = torch.arange(n, dtype=torch.int32, device="cuda")
            qb.paged_append(cache, k[:n].contiguous(), v[:n].contiguous(), at, seq=torch.full_like(at, b), slot=at)
    return cache, flat


MANY = [5, 900, 0, 17, 128, 300, 1, 64, 511, 33, 2, 77, 256, 40, 8, 100, 3, 9, 6, 21]


@pytest.fixture
def fp32_projections():
    old = qb.get_gemm_threshold()
    qb.set_gemm_threshold(1 << 20)
    yield
    qb.set_gemm_threshold(old)


@pytest.mark.parametrize("lens", [[1000], [0, 63, 64, 700], MANY])
def test_decode_of_several_sequences(oracle, blk_pair, fp32_projections, lens):
    """Each row equals the oracle's block for that sequence alone, with the fp32
    projections (the seeded weights' scores reach thousands, where bf16 queries
    of the tensor-core projections would move the softmax)."""
    arr, blk = blk_pair
    B = len(lens)
    cache, flat = filled(arr, lens)
    X = inputs.hidden(70 + B, B, 2048)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = qb.block_decode_paged(blk, cache, torch.from_numpy(X).cuda(), pos).cpu().numpy()
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    assert cache.lens.tolist() == [n + 1 for n in lens]
    for b in range(min(B, 6)):
        kc, vc = (oracle.bf16_bits_to_f64(np.roll(arr[n], b, axis=0)) for n in ("k_cache", "v_cache"))
        ref, parts = oracle.block_forward_rows(X[b:b + 1], arr, 8, lens[b], kc, vc, np.array([0]))
        assert_close(out[b:b + 1], ref, TOL_GEMV, rows=parts["gap"] >= GAP)


def test_decode_of_many_sequences_on_the_tensor_cores(blk_pair):
    """At the default threshold 20 rows take the tensor-core projections: the
    cached rows equal those of the fp32 projections up to the bf16 operands (as
    the block's own test bounds them), and every output is finite."""
    arr, blk = blk_pair
    assert len(MANY) > qb.get_gemm_threshold()
    X = torch.from_numpy(inputs.hidden(60, len(MANY), 2048)).cuda()
    pos = torch.tensor(MANY, dtype=torch.int32, device="cuda")
    rows = []
    old = qb.get_gemm_threshold()
    for threshold in (old, 1 << 20):
        qb.set_gemm_threshold(threshold)
        try:
            cache, _ = filled(arr, MANY)
            out = qb.block_decode_paged(blk, cache, X, pos, accumulate=True)
        finally:
            qb.set_gemm_threshold(old)
        assert bool(torch.isfinite(out).all())
        at = cache.table[torch.arange(len(MANY), device="cuda"), pos.long() // 64].long()
        rows.append(torch.stack([cache.k[at, pos.long() % 64], cache.v[at, pos.long() % 64]]).float())
    assert qb.query_status() == 0
    assert_close(rows[0].cpu().numpy(), rows[1].cpu().numpy(), TOL_TC)


def test_decode_equals_the_contiguous_path(blk_pair):
    """Several steps of two sequences against the block's own decode on contiguous
    caches: the projections and the experts are the same kernels, so only the
    attention's order of sums differs (fp32 on both sides)."""
    arr, blk = blk_pair
    lens = [130, 65]
    cache, flat = filled(arr, lens, page=16)
    pos = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for step in range(4):
        X = torch.from_numpy(inputs.hidden(90 + step, 2, 2048)).cuda()
        out = qb.block_decode_paged(blk, cache, X, pos, accumulate=True)
        for b in range(2):
            want = qb.block_forward(blk, X[b:b + 1].contiguous(), *flat[b], lens[b] + step)
            assert_close(out[b:b + 1].cpu().numpy(), want.cpu().numpy(), TOL_GEMV)
        pos += 1
    assert qb.query_status() == 0
    # the weights of a sequence add up to the query heads of a group per step
    for b in range(2):
        got = cache.weight[b].sum(dim=1)
        assert torch.allclose(got, torch.full_like(got, 32.0), rtol=1e-4)


def test_bounded_decode(blk_pair):
    """A prompt, then steps with eviction: the cache stays at its budget, the
    newest entries stay in it, and the result stays that of the contiguous path
    as long as nothing is evicted."""
    arr, blk = blk_pair
    budget, recent, n = 96, 32, 90
    cache, flat = filled(arr, [n])
    pos = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = qb.block_decode_paged_workspace(blk, cache, True)
    for step in range(20):
        X = torch.from_numpy(inputs.hidden(120 + step, 1, 2048)).cuda()
        out = qb.block_decode_paged(blk, cache, X, pos, accumulate=True, ws=ws)
        if n + step < budget:
            want = qb.block_forward(blk, X, *flat[0], n + step)
            assert_close(out.cpu().numpy(), want.cpu().numpy(), TOL_GEMV)
        pos += 1
        qb.cache_evict(cache, pos, budget, recent)
        held = int(cache.lens[0])
        assert held == min(n + step + 1, budget)
        for g in range(2):
            at = cache.pos[0, g, :held].tolist()
            assert len(set(at)) == held and set(range(n + step + 1 - recent, n + step + 1)) <= set(at)
        assert bool(torch.isfinite(out).all())
    assert qb.query_status() == 0


def test_full_sequence_is_reported(blk_pair):
    arr, blk = blk_pair
    cache, _ = filled(arr, [1024, 3])
    pos = torch.tensor([1024, 3], dtype=torch.int32, device="cuda")
    qb.block_decode_paged(blk, cache, torch.from_numpy(inputs.hidden(7, 2, 2048)).cuda(), pos)
    torch.cuda.synchronize()
    assert qb.query_status() == -8
    assert cache.lens.tolist() == [1024, 4]


def test_withheld_copy_times_out(blk_pair):
    """A copy that never comes ends the wait after its limit: the status says so
    and the next call is right again."""
    arr, _ = blk_pair
    cache, _ = filled(arr, [1000])
    q = torch.randn(1, 16, 128, device="cuda")
    want = qb.paged_attention(cache, q)
    torch.cuda.synchronize()
    qb.test_inject("paged_copy", 2000)
    try:
        qb.paged_attention(cache, q)
        assert qb.query_status() == -7
    finally:
        qb.test_inject("none")
    got = qb.paged_attention(cache, q)
    assert qb.query_status() == 0
    assert torch.equal(got, want)
