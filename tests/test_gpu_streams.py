"""What a call allocates for itself belongs to the stream that it runs on: released
at its return, the bytes go to that stream's next calls, not to work that runs
beside it. The results on another stream are those on the current one."""

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from quantized_moe_transformer_gb300 import inputs
from tests.test_gpu_paged_edges import allocations  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()
    arr = inputs.block(5, ctx=64)
    return arr, qb.Block.from_arrays(arr, 8)


def calls(block, stream):
    arr, blk = block
    X = torch.from_numpy(inputs.hidden(8, 3, 2048)).cuda()
    caches = [qb.cache_from_bits(arr[n]) for n in ("k_cache", "v_cache") * 2]
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    got = [*qb.moe_route(X, blk.moe.Wr, 8, stream=stream), qb.moe_forward(blk.moe, X, stream=stream),
           qb.moe_forward_noalloc(blk.moe, X, stream=stream), qb.rmsnorm(X, blk.g1, stream=stream),
           qb.attn_forward(blk, X, None, *caches[:2], 30, stream=stream), qb.block_forward(blk, X, *caches[2:], 30, stream=stream)]
    torch.cuda.synchronize()
    assert qb.query_status() == 0
    return got


def test_temporaries_of_the_layer_and_the_block(block, allocations):  # noqa: F811
    want = calls(block, None)
    assert set(allocations) == {torch.cuda.current_stream().cuda_stream}
    side = torch.cuda.Stream()
    allocations.clear()
    got = calls(block, side)
    assert len(allocations) >= 11
    assert set(allocations) == {side.cuda_stream}
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # host tensors: the output lies on the host, the workspace on the device
    X = torch.from_numpy(inputs.hidden(8, 3, 2048)).pin_memory()
    out = torch.zeros_like(X)
    allocations.clear()
    qb.moe_forward_host(block[1].moe, X, out=out, stream=side)
    assert allocations == [side.cuda_stream]
    assert torch.equal(out, want[2].cpu())
