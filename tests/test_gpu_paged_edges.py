"""The paged cache at the edges of its ranges and beside the usual way of its
calls. Attention is compared with the plain 64-bit implementation at the tolerance
derived in test_gpu_paged.py.
"""

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from tests import paged_ref as ref
from tests.test_gpu_paged import handle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


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
