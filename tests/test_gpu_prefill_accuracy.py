"""How many bits attention of packed rows keeps of its scores, probabilities and
sums, on inputs that show one bit more or less.

Key blocks are of 64 entries, and tiles may be cut between two CTAs from 512
entries on (parts of four key blocks at least), so the lengths lie about 64, 256
and 512, with few rows (tiles in parts) and many (whole tiles).
"""

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from tests import prefill_ref as ref
from tests.test_gpu_prefill import make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


HEADS = [(16, 2, 128), (8, 8, 64), (12, 4, 96), (8, 2, 256), (3, 1, 200), (2, 2, 8)]


@pytest.mark.parametrize("heads,kv,hd", HEADS)
@pytest.mark.parametrize("counts,lens", [
    ([37], [37]), ([63, 64, 65], [63, 64, 65]), ([300], [300]), ([5, 9, 7], [255, 256, 257]), ([3, 6, 20], [511, 512, 513]),
    ([16], [1000]), ([200], [1100])])
def test_bf16_rows_are_rounded_once(counts, lens, heads, kv, hd):
    """Keys of one non-zero head dim, at most 2 like the queries there: a score is one exact product of 4 at
    most, 5.8 in units of log2. What an output is off before it is rounded, in parts of the sum of p |v|: a
    probability's two bf16 parts 2^-17; its argument 4 roundings of 2^-24 times 5.8, in numerator and denominator; n / 8
    products of 16 entries that the tensor cores cut off at 2^-23, and 64 more of those for the exponential,
    the denominator's sums, rescaling, joining parts and the division. The rounding to bf16 takes the nearest: the output
    is off by what the right one's rounding is, and twice the rest. Probabilities of one bf16 part
    are off by up to 2^-8, at random: 2^-10 / sqrt(n) of the sum, 2^-13 at 100 entries."""
    page = 32
    c = make(counts, lens, heads, kv, hd, page, torch.bfloat16, spread=1.0)
    c["k"][..., 1:] = torch.where(torch.isnan(c["k"][..., 1:]), c["k"][..., 1:], 0.0)
    c["k"].clamp_(-2, 2)
    c["q"].clamp_(-2, 2)
    out = run(c, scale=1.0)
    assert qb.query_status() == 0
    want, mean, _ = ref.attention(c["q"], c["k"], c["v"], c["table"], c["lens"], c["first"], c["count"], page, 1.0)
    mine = ~torch.isnan(want)
    got, want, mean = out.double()[mine], want[mine], mean[mine]
    before = (2.0 ** -17 + 8 * 5.8 * 2.0 ** -24 + (max(lens) / 8 + 64) * 2.0 ** -23) * mean
    tol = (want.to(torch.bfloat16).double() - want).abs() + 2 * before
    assert bool(((got - want).abs() <= tol + 1e-30).all()), float(((got - want).abs() / (tol + 1e-30)).max())
