"""How many bits attention of packed rows keeps of its scores, probabilities and
sums, on inputs that show one bit more or less.

Key blocks are of 64 entries, and tiles may be cut between two CTAs from 512
entries on (parts of four key blocks at least), so the lengths lie about 64, 256
and 512, with few rows (tiles in parts) and many (whole tiles).
"""

import math

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from tests import prefill_ref as ref
from tests.test_gpu_paged_accuracy import two_part_rest
from tests.test_gpu_prefill import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


HEADS = [(16, 2, 128), (8, 8, 64), (12, 4, 96), (8, 2, 256), (3, 1, 200), (2, 2, 8)]


def make_exact(counts, lens, heads, kv, hd, page):
    """bf16 rows and keys of one non-zero head dim, at most 2 there: a score is one exact product of 4 at most,
    5.8 in units of log2."""
    c = make(counts, lens, heads, kv, hd, page, torch.bfloat16, spread=1.0)
    c["k"][..., 1:] = torch.where(torch.isnan(c["k"][..., 1:]), c["k"][..., 1:], 0.0)
    c["k"].clamp_(-2, 2)
    c["q"].clamp_(-2, 2)
    return c


def before_rounding(longest):
    """What an output is off before it is rounded, in parts of the sum of p |v|: a
    probability's two bf16 parts 2^-17; its argument 4 roundings of 2^-24 times 5.8, in numerator and denominator; n / 8
    products of 16 entries that the tensor cores cut off at 2^-23, and 64 more of those for the exponential,
    the denominator's sums, rescaling, joining parts and the division."""
    return 2.0 ** -17 + 8 * 5.8 * 2.0 ** -24 + (longest / 8 + 64) * 2.0 ** -23


@pytest.mark.parametrize("heads,kv,hd", HEADS)
@pytest.mark.parametrize("counts,lens", [
    ([37], [37]), ([63, 64, 65], [63, 64, 65]), ([300], [300]), ([5, 9, 7], [255, 256, 257]), ([3, 6, 20], [511, 512, 513]),
    ([16], [1000]), ([200], [1100])])
def test_bf16_rows_are_rounded_once(counts, lens, heads, kv, hd):
    """The rounding to bf16 takes the nearest: an output is off by what the right one's rounding is, and twice
    what it was off before. Probabilities of one bf16 part would be off by up to 2^-8, at random: 2^-10 / sqrt(n) of the
    sum of p |v|, 2^-13 at 100 entries."""
    page = 32
    c = make_exact(counts, lens, heads, kv, hd, page)
    out = run(c, scale=1.0)
    assert qb.query_status() == 0
    want, mean, _ = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["first"], c["count"], page, 1.0)
    mine = ~torch.isnan(want)
    got, want, mean = out.double()[mine], want[mine], mean[mine]
    tol = (want.to(torch.bfloat16).double() - want).abs() + 2 * before_rounding(max(lens)) * mean
    assert bool(((got - want).abs() <= tol + 1e-30).all()), float(((got - want).abs() / (tol + 1e-30)).max())


@pytest.mark.parametrize("heads,kv,hd", [(16, 2, 128), (8, 8, 64), (8, 2, 256)])
def test_bf16_single_rows_are_the_decoding_calls(heads, kv, hd):
    """One row of each sequence: the same as of paged_attention, but where the right output is so near to
    the middle between two bf16 numbers that what may be lost before the rounding decides. Of 1000 entries, the longest
    here, that is 2^-15 of the sum of p |v| to each side; an output is about 1 / sqrt(700) of it and a step 2^-7.5 of that:
    a quarter of the outputs, and less than half of all."""
    lens = [1, 64, 300, 1000, 77, 513]
    c = make_exact([1] * len(lens), lens, heads, kv, hd, 64)
    got = run(c, scale=1.0)[:len(lens)]
    cache = qb.PagedCache(c["k"], c["v"], c["table"], c["lens"])
    decoded = qb.paged_attention(cache, c["q"][:len(lens)].contiguous(), scale=1.0)
    want, mean, _ = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["first"], c["count"], 64, 1.0)
    want, e = want[:len(lens)], before_rounding(max(lens)) * mean[:len(lens)]
    clear = (want - e).to(torch.bfloat16) == (want + e).to(torch.bfloat16)
    assert float(clear.double().mean()) > 0.5
    assert torch.equal(got[clear], decoded[clear])


def parts(x, n):
    """The first n bf16 parts of fp32 numbers, together."""
    out, left = torch.zeros_like(x, dtype=torch.float64), x.float()
    for _ in range(n):
        part = left.to(torch.bfloat16).float()
        out, left = out + part.double(), left - part
    return out


def in_parts(c, page, q_parts, p_parts):
    """Rows of one sequence in 64 bits, of which queries and probabilities (relative to a row's largest) keep some bf16 parts."""
    (n,), (m,), (r0,) = c["count"].tolist(), c["lens"].tolist(), c["first"].tolist()
    heads, hd = c["q"].shape[1:]
    k, v = (ref.entries(c[t], c["table"], 0, m, page)[0] for t in "kv")
    hidden = torch.ones(n, m, dtype=torch.bool, device="cuda").triu_(m - n + 1)
    out = torch.empty(n, heads, hd, dtype=torch.float64, device="cuda")
    for h in range(heads):
        g = h // (heads // k.shape[1])
        x = parts(c["q"][r0:r0 + n, h], q_parts) @ k[:, g].T / math.sqrt(hd)
        x = x.masked_fill(hidden, -math.inf)
        p = torch.exp(x - x.max(1, keepdim=True).values)
        out[:, h] = parts(p.float(), p_parts) @ v[:, g] / p.sum(1, keepdim=True)
    return out


@pytest.mark.parametrize("heads,kv,hd", [(8, 8, 64), (16, 2, 128), (8, 2, 256), (6, 2, 200)])
@pytest.mark.parametrize("n,m", [(300, 300), (65, 513), (8, 1024), (16, 9000)])
def test_fp32_rows_in_norm(heads, kv, hd, n, m):
    """Whole tiles, tiles in two parts and in many. Random values: an output is off, relative to
    the outputs' norm, by what a weight is off, relative to itself. That is the score's error: hd / 16 products with the
    largest parts of the queries, each cut off by half a step on average, 2^-24 of a power of two below sums that grow to 1.5
    (two thirds of it in the mean, and three quarters of that); then 2^-22 for the exponential and its argument, and
    2^-25 for each key block that an output is a sum of, at random. Two parts of the queries
    leave 2^-17 to 2^-20 of each, two of the probabilities too: 1.3e-6 and more in norm, above the bound."""
    page = 64
    c = make([n], [m], heads, kv, hd, page, torch.float32, seed=7)
    out = run(c)
    assert qb.query_status() == 0
    want, _, _ = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["first"], c["count"], page)
    r0 = int(c["first"])
    want = want[r0:r0 + n]
    off = lambda x: float((x.double() - want).norm() / want.norm())
    bound = hd / 16 * 0.75 * 2.0 ** -24 + 2.0 ** -22 + math.sqrt(m / 64) * 2.0 ** -25
    assert off(out[r0:r0 + n]) <= bound, off(out[r0:r0 + n]) / bound
    assert off(in_parts(c, page, 3, 3)) < bound / 4
    assert off(in_parts(c, page, 2, 3)) > bound and off(in_parts(c, page, 3, 2)) > bound


def coherent(n, kv, hd, page, every, key):
    """n entries: one in ``every`` has score and value 0, the others ``key`` in head dim 0 and
    one value in [1, 2) per head dim; and how many they are."""
    k = torch.zeros(n // page, page, kv, hd, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    j = torch.arange(n, device="cuda")
    counted = j[j % every != 0]
    k[counted // page, counted % page, :, 0] = key
    value = (1 + torch.arange(hd, device="cuda") % 128 / 128).to(torch.bfloat16)
    v[counted // page, counted % page] = value
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    return qb.PagedCache(k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda")), value.double(), len(counted)


COHERENT = [(16, 2, 128), (8, 8, 64), (8, 1, 256), (6, 2, 200), (3, 1, 8)]


def one_row(cache, q):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out = qb.paged_prefill_attention(cache, q, i32([0]), i32([1]), scale=1.0)
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    return out.double()


@pytest.mark.parametrize("heads,kv,hd", COHERENT)
def test_fp32_rows_keep_the_bits_of_probabilities(heads, kv, hd):
    """One row that sees 256 entries, whose errors of a probability add up. Steps of 2^-24: 24 of a key block's
    products (twelve, cut off at 2^-23), 4 of the blocks' sums, 15 of the denominator's (chains of 8, three more, the
    blocks), 3 of the division, 1 of the exponential and its argument, by the share of the zero entries: 47 and
    1 to spare. Two parts of the probability would be off by 2^-17.5 and more, 90 steps."""
    a = torch.arange(26, 256).float() / 256
    rest = two_part_rest(torch.exp(-a.double()).float())
    picked = a[rest.argsort(descending=True)[:4]]
    assert bool((rest.sort(descending=True).values[:4] >= 2.0 ** -17.5).all())
    for x in picked.tolist():
        cache, value, many = coherent(256, kv, hd, 64, 16, -x)
        q = torch.zeros(1, heads, hd, device="cuda")
        q[..., 0] = 1.0
        want = value * (many * math.exp(-x) / (many * math.exp(-x) + 256 - many))
        err = (one_row(cache, q) - want).abs() / want
        assert float(err.max()) <= 48 * 2.0 ** -24, float(err.max()) * 2 ** 24


@pytest.mark.parametrize("heads,kv,hd", COHERENT)
def test_fp32_rows_keep_the_bits_of_queries(heads, kv, hd):
    """The same with queries of 24 bits, a score of -4 q for 63 entries in 64, exact in three parts. A score that is off moves
    the share of the entries counted by that of the others, 0.6 to 0.8 here. The steps above, and 8 more of a
    score's size in units of log2, 6 to 8: 64 more. Two parts of a query would be off by 2^-17.5 of 4 to 6, 200 steps and more."""
    g = torch.Generator()
    g.manual_seed(3)
    q0 = 1.1 + 0.3 * torch.rand(4096, generator=g)
    rest = two_part_rest(q0)
    picked = q0[rest.argsort(descending=True)[:4]]
    assert bool((rest.sort(descending=True).values[:4] >= 2.0 ** -17.5).all())
    for x in picked.tolist():
        cache, value, many = coherent(256, kv, hd, 64, 64, -4.0)
        q = torch.zeros(1, heads, hd, device="cuda")
        q[..., 0] = x
        want = value * (many * math.exp(-4 * x) / (many * math.exp(-4 * x) + 256 - many))
        err = (one_row(cache, q) - want).abs() / want
        assert float(err.max()) <= (47 + 64) * 2.0 ** -24, float(err.max()) * 2 ** 24
