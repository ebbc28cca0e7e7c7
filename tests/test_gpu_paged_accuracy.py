"""How many bits paged attention keeps of its probabilities and sums, on inputs
that show one bit more or less.

bf16 rows are the fp32 rows of the same queries rounded once: the three parts of
a bf16 query are itself and two zeros, whose products add nothing, and where both
types cut the work alike (head dims up to 128, groups of up to 8 heads) every
other operation is the same, so the results are the same bits.

The other cases have keys of one non-zero head dim, so a score is one exact
product, and values that are the same in all counted entries, so that errors of
the probabilities add up instead of averaging out.
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


@pytest.mark.parametrize("heads,kv,hd", [(16, 2, 128), (8, 8, 64), (12, 4, 96), (8, 1, 128), (3, 1, 8)])
@pytest.mark.parametrize("lens", [[70000], [5000, 0, 1, 77, 1200], [300] * 40])
def test_bf16_rows_are_the_fp32_rows_rounded_once(heads, kv, hd, lens):
    c, g = ref.cache(40, lens, kv, hd, 64)
    q = (1.5 * torch.randn(len(lens), heads, hd, generator=g, device="cuda")).to(torch.bfloat16)
    before = c["weight"].clone()
    h = qb.PagedCache(c["k"], c["v"], c["table"], c["lens"], c["weight"], c["pos"])
    wide = qb.paged_attention(h, q.float(), accumulate=True)
    wide_w = c["weight"].clone()
    c["weight"].copy_(before)
    out = qb.paged_attention(h, q, accumulate=True)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    assert torch.equal(out, wide.to(torch.bfloat16))
    assert torch.equal(c["weight"], wide_w)


def two_part_rest(p):
    """What two bf16 parts leave of a number, relative to it."""
    hi = p.to(torch.bfloat16).float()
    mid = (p - hi).to(torch.bfloat16).float()
    return ((p - hi - mid) / p).abs()


def coherent_cache(n, kv, hd, page, a, n_seqs=1):
    """n entries: every 16th has score 0 and value 0, the others score -a (for a
    query of 1 in head dim 0 and scale 1) and one value in [1, 2) per head dim.
    All sequences have the same pages."""
    pages = -(-n // page)
    k = torch.zeros(pages, page, kv, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    j = torch.arange(n, device="cuda")
    counted = j[j % 16 != 0]
    k[counted // page, counted % page, :, 0] = -a
    value = (1 + torch.arange(hd, device="cuda") % 128 / 128).to(torch.bfloat16)
    v[counted // page, counted % page] = value
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(n_seqs, pages).contiguous()
    lens = torch.full((n_seqs,), n, dtype=torch.int32, device="cuda")
    share = len(counted) * math.exp(-a) / (len(counted) * math.exp(-a) + n - len(counted))
    return qb.PagedCache(k, v, table, lens), value.double() * share


@pytest.mark.parametrize("heads,kv,hd", [(16, 2, 128), (8, 8, 64), (8, 1, 256), (6, 2, 200)])
def test_probabilities_keep_their_bits(heads, kv, hd):
    """One sequence of 1000 entries, fp32 rows. Roundings of 2^-24: 8 of a tile's
    products (three instructions, cut off at 2^-23, and the alignment of their
    addends), 8 each of the sums of outputs and of denominators in a warp, 5 of
    the lanes' sums, 9 each of merging warps and joining CTAs, 3 of the division:
    50 in all. An error of a probability itself appears in numerator and
    denominator and is left by the share of the zero entries, at most 1/8 of
    (2^-22 for the exponential and 4 roundings of a score below 2): 1 more. Two
    parts of the probability would be off by 2^-17.5 and more, 90 such roundings."""
    a = torch.arange(26, 256, device="cpu").float() / 256
    rest = two_part_rest(torch.exp(-a.double()).float())
    picked = a[rest.argsort(descending=True)[:4]]
    assert bool((rest.sort(descending=True).values[:4] >= 2.0 ** -17.5).all())
    for x in picked.tolist():
        cache, want = coherent_cache(1000, kv, hd, 64, x)
        q = torch.zeros(1, heads, hd, device="cuda")
        q[..., 0] = 1.0
        out = qb.paged_attention(cache, q, scale=1.0)
        err = (out.double() - want).abs() / want
        assert float(err.max()) <= 51 * 2.0 ** -24, float(err.max()) * 2 ** 24


def test_sums_of_a_long_row_are_rounded():
    """A row of 16384 entries for each warp of the GPU, all probabilities 1. A
    tile of 16 slots adds 8 c - 2^-13, which from a sum of 4096 on is just below a
    step of fp32: a rounded sum is off by at most half a step each time, a sum
    that is cut off by 7/8 of one."""
    n, hd, page = 16384, 128, 64
    rows = torch.cuda.get_device_properties(0).multi_processor_count * 7
    k = torch.zeros(n // page, page, 1, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.full_like(k, -2.0 ** -16)
    c = (1 + torch.arange(hd, device="cuda") / 128).to(torch.bfloat16)
    v[:, ::2, 0] = c
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").expand(rows, n // page).contiguous()
    cache = qb.PagedCache(k, v, table, torch.full((rows,), n, dtype=torch.int32, device="cuda"))
    out = qb.paged_attention(cache, torch.zeros(rows, 8, hd, device="cuda"))
    total = (8 * c.double() - 2.0 ** -13)
    steps = torch.arange(1, n // 16 + 1, device="cuda", dtype=torch.float64)[:, None] * total
    half = torch.exp2(torch.floor(torch.log2(steps)) - 24).sum(0)  # half steps of the sums on the way
    # and 8 roundings of a tile's products, 3 of the division
    tol = half / n + 11 * 2.0 ** -24 * total / 16
    err = (out.double() - total / 16).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
