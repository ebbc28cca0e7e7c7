"""The paged cache at the edges of its ranges and beside the usual way of its
calls. Attention is compared with the plain 64-bit implementation at the tolerance
derived in test_gpu_paged.py.
"""

import math

import numpy as np
import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from quantized_moe_transformer_gb300 import inputs
from tests import paged_ref as ref
from tests.parity import TOL_TC, assert_close
from tests.test_gpu_paged import close_out, handle, score_tol, v_max
from tests.test_gpu_paged_block import MANY, filled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


#: one sequence with a table of at most 512 slots: (heads, KV heads, head dim, entries)
MANY_ROWS = [(160, 160, 64, 100), (153, 153, 128, 100), (153, 153, 128, 3), (152, 152, 64, 40), (1280, 20, 64, 512),
             (400, 400, 256, 130), (305, 305, 8, 0)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,kv,hd,n", MANY_ROWS)
def test_one_short_sequence_with_more_rows_than_sms(heads, kv, hd, n, dtype, accumulate):
    c, g = ref.cache(50, [n], kv, hd, 64, width=max(2, -(-n // 64)))
    q = torch.randn(1, heads, hd, generator=g, device="cuda").to(dtype)
    before = c["weight"].clone()
    out = torch.full_like(q, math.nan)
    qb.paged_attention(handle(c), q, out=out, accumulate=accumulate)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    want, received, bound = ref.attention(q, c["k"], c["v"], c["table"], c["lens"], 64)
    close_out(out, want, bound, hd, max(v_max(c), 1e-30))
    if not accumulate:
        assert torch.equal(c["weight"], before)
        return
    tol = received * (2 * score_tol(hd, bound) + (heads // kv + 8) * 2.0 ** -24) + (before.double() + received) * 2.0 ** -24
    assert bool(((c["weight"].double() - before.double() - received).abs() <= tol + 1e-30).all())


def test_append_to_a_length_below_zero():
    """A length below zero is taken as zero: the next entry is slot 0."""
    c, g = ref.cache(51, [32, 32, 32], 2, 128, 16)
    c["lens"].copy_(torch.tensor([-5, 3, -(1 << 31)]))
    row = torch.randn(3, 2, 128, generator=g, device="cuda")
    pos = torch.tensor([7, 8, 9], dtype=torch.int32, device="cuda")
    qb.paged_append(handle(c), row, row, pos)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    assert c["lens"].tolist() == [1, 4, 1]
    for b, slot in ((0, 0), (1, 3), (2, 0)):
        page = int(c["table"][b, 0])
        assert torch.equal(c["k"][page, slot], row[b].to(torch.bfloat16))
        assert torch.equal(c["v"][page, slot], row[b].to(torch.bfloat16))
        assert c["pos"][b, :, slot].tolist() == [7 + b] * 2 and c["weight"][b, :, slot].tolist() == [0.0] * 2


@pytest.fixture
def allocations(monkeypatch):
    """The stream that is current at each allocation."""
    seen = []
    for name in ("empty", "empty_like"):
        plain = getattr(torch, name)

        def noted(*a, plain=plain, **kw):
            seen.append(torch.cuda.current_stream().cuda_stream)
            return plain(*a, **kw)

        monkeypatch.setattr(torch, name, noted)
    return seen


def test_temporaries_of_a_call_on_another_stream(allocations):
    """Outputs and workspaces that a call allocates belong to the stream it runs
    on: released at its return, their bytes go to that stream's next calls, not to
    work that runs beside it."""
    c, g = ref.cache(52, [300, 20], 2, 128, 64)
    h = handle(c)
    q = torch.randn(2, 16, 128, generator=g, device="cuda")
    rows = torch.randn(2, 2, 128, generator=g, device="cuda")
    pos = torch.tensor([300, 20], dtype=torch.int32, device="cuda")
    arr = inputs.block(5, ctx=64)
    blk = qb.Block.from_arrays(arr, 8)
    X = torch.from_numpy(inputs.hidden(7, 2, 2048)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    allocations.clear()
    qb.paged_append(h, rows, rows, pos, q=q, rope_theta=1e4, stream=side)
    qb.paged_attention(h, q, accumulate=True, stream=side)
    qb.block_decode_paged(blk, h, X, pos + 1, accumulate=True, stream=side)
    qb.cache_evict(h, pos + 2, 200, 10, stream=side)
    side.synchronize()
    assert qb.query_status() == 0
    assert len(allocations) >= 6
    assert set(allocations) == {side.cuda_stream}


@pytest.mark.parametrize("n", [1000, 40000])
def test_withheld_copy_of_a_short_and_a_long_row(n):
    """The copies' warp gives up too: 1000 entries are one tile a warp; of 40000 the
    withheld copy's warp has tiles that it never comes to, whose copies wait for
    free places in its ring."""
    c, g = ref.cache(54, [n], 2, 128, 64)
    q = torch.randn(1, 16, 128, generator=g, device="cuda")
    h = handle(c)
    want = qb.paged_attention(h, q)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    qb.test_inject("paged_copy", 2000)
    try:
        qb.paged_attention(h, q)
        assert qb.query_status() == -7
    finally:
        qb.test_inject("none")
    got = qb.paged_attention(h, q)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("n", [1000, 40000])
def test_weights_survive_a_wait_that_runs_out(n):
    """A call that gives up reports it and leaves the accumulated weights alone (an
    infinite weight would hold its entry through every later eviction); the next
    call is right."""
    c, g = ref.cache(53, [n], 2, 128, 64)
    q = torch.randn(1, 16, 128, generator=g, device="cuda")
    h = handle(c)
    ws = qb.paged_attention_workspace(h, 16, True)
    before = c["weight"].clone()
    want = qb.paged_attention(h, q, accumulate=True, ws=ws)
    want_w = c["weight"].clone()
    c["weight"].copy_(before)
    ws.fill_(0x7F)  # whatever an earlier call left there
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    qb.test_inject("paged_copy", 2000)
    try:
        qb.paged_attention(h, q, accumulate=True, ws=ws)
        assert qb.query_status() == -7
    finally:
        qb.test_inject("none")
    assert torch.equal(c["weight"], before)
    got = qb.paged_attention(h, q, accumulate=True, ws=ws)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    assert torch.equal(got, want) and torch.equal(c["weight"], want_w)


# ---------------------------------------------------------------- the block

@pytest.fixture(scope="module")
def quiet():
    """A block whose scores are a few units (gains of 1/32 ahead of the
    projections, where the seeded weights' scores reach thousands), once with its
    experts and once with experts that give zero, whose output is the attention
    branch and the residual alone."""
    arr = inputs.block(5, ctx=1024)
    arr["g1"] = arr["g1"] / np.float32(32)
    whole = qb.Block.from_arrays(arr, 8)
    moe = dict(arr["moe"])
    for name in ("Wd", "Sd"):
        moe[name] = moe[name].copy()
        moe[name][..., :4] = 0  # the super-blocks' scale and minimum
    return arr, whole, qb.Block.from_arrays({**arr, "moe": moe}, 8)


@pytest.mark.parametrize("threshold", [None, 1 << 20])
def test_attention_branch_of_every_row(oracle, quiet, threshold):
    """20 sequences at once, on the tensor-core projections (the default threshold)
    and on the fp32 ones: every row's attention branch equals the oracle's for that
    sequence alone to the tensor-core tolerance of its own largest value."""
    arr, _, attn_only = quiet
    B = len(MANY)
    old = qb.get_gemm_threshold()
    assert B > old
    if threshold is not None:
        qb.set_gemm_threshold(threshold)
    try:
        cache, _ = filled(arr, MANY)
        X = inputs.hidden(60, B, 2048)
        pos = torch.tensor(MANY, dtype=torch.int32, device="cuda")
        out = qb.block_decode_paged(attn_only, cache, torch.from_numpy(X).cuda(), pos).cpu().numpy()
    finally:
        qb.set_gemm_threshold(old)
    assert qb.query_status() == 0
    for b, n in enumerate(MANY):
        kc, vc = (oracle.bf16_bits_to_f64(np.roll(arr[name], b, axis=0)) for name in ("k_cache", "v_cache"))
        want = X[b:b + 1] + oracle.attn_sublayer(X[b:b + 1], arr, n, kc, vc)
        assert_close(out[b:b + 1], want, TOL_TC)


@pytest.mark.parametrize("threshold", [None, 1 << 20])
def test_experts_follow_the_attention_branch(quiet, threshold):
    """The whole block equals norm and experts, by their own calls, on the attention
    branch's rows: the same kernels, so the same bits."""
    arr, whole, attn_only = quiet
    X = torch.from_numpy(inputs.hidden(61, len(MANY), 2048)).cuda()
    pos = torch.tensor(MANY, dtype=torch.int32, device="cuda")
    old = qb.get_gemm_threshold()
    if threshold is not None:
        qb.set_gemm_threshold(threshold)
    try:
        h1 = qb.block_decode_paged(attn_only, filled(arr, MANY)[0], X, pos)
        out = qb.block_decode_paged(whole, filled(arr, MANY)[0], X, pos)
        r2 = qb.rmsnorm(h1, whole.g2)
        want = qb.moe_forward(whole.moe, r2, R=h1)
    finally:
        qb.set_gemm_threshold(old)
    assert qb.query_status() == 0
    assert torch.equal(out, want)
