"""Rotary positions of rows, alone and on their way into the paged cache, against 64 bits.

Tolerances. A sine or cosine is off by at most 2^-22 (the angle's rounding to fp32
after an exact reduction, and the function's), times the scale; a result is two
products and a sum in fp32, 3 roundings of 2^-24 of |a| + |b|. Together 2^-21 of the
pair's |a| + |b| times the scale bounds them; bf16 results are rounded once, 2^-8.
"""

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from tests import prefill_ref as ref

pytestmark = pytest.mark.gpu
LONG = dict(scaling="parts", factor=8.0, context=4096.0, low=1.0, high=32.0)
WAYS = [dict(), dict(layout="interleaved"), dict(layout="interleaved", scaling="linear", factor=4.0),
        dict(scale=1.25, **LONG), dict(layout="interleaved", theta=1e4, scale=0.5, **LONG)]


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from quantized_moe_transformer_gb300 import build
    build.build()


def freq(dims, way):
    return ref.frequencies(dims, **{k: v for k, v in way.items() if k not in ("layout", "scale")})


def close(got, x, pos, dims, way, transpose=False):
    layout, scale = way.get("layout", "half"), way.get("scale", 1.0)
    want = ref.turned(x, pos, freq(dims, way), layout, scale, transpose)
    n = dims // 2
    size = x.double().abs()
    both = size[..., :n] + size[..., n:dims] if layout == "half" else size[..., 0:dims:2] + size[..., 1:dims:2]
    tol = torch.zeros_like(want)
    tol[..., :dims] = 2.0 ** -21 * abs(scale) * (torch.cat([both, both], 2) if layout == "half" else both.repeat_interleave(2, 2))
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    assert bool(((got.double() - want).abs() <= tol).all()), float((got.double() - want).abs().max())
    assert torch.equal(got[..., dims:], x[..., dims:].to(got.dtype)), "elements behind the turned ones changed"


def rows(n, heads, hd, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, heads, hd, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("way", range(len(WAYS)))
@pytest.mark.parametrize("hd,dims", [(128, 128), (128, 64), (256, 256), (96, 24), (8, 8), (72, 40)])
@pytest.mark.parametrize("transpose", [False, True])
def test_rows(hd, dims, way, dtype, transpose):
    way = WAYS[way]
    q, k = rows(37, 5, hd, dtype), rows(37, 2, hd, dtype, 1)
    pos = (torch.arange(37, device="cuda") * 3571 - 7).int()
    pos[3], pos[4], pos[5] = 2 ** 31 - 1, -2 ** 31, 0
    qo, ko = qb.rope(qb.Rope(dims, **way), pos, q, k, transpose=transpose)
    close(qo, q, pos, dims, way, transpose)
    close(ko, k, pos, dims, way, transpose)
    assert torch.equal(qb.rope(qb.Rope(dims, **way), pos, q, transpose=transpose), qo)


@pytest.mark.parametrize("n", [1, 2, 31, 33, 700, 5000])
def test_row_counts_and_strides(n):
    """Parts of a joint projection, heads outside the rows, in place."""
    way = WAYS[3]
    r = qb.Rope(64, **way)
    joint = rows(n, 8, 128, torch.bfloat16)
    q, k = joint[:, :4], joint[:, 4:6]
    pos = torch.arange(n, dtype=torch.int32, device="cuda") + 70000
    qo, ko = qb.rope(r, pos, q, k)
    close(qo, q, pos, 64, way)
    close(ko, k, pos, 64, way)
    across = torch.empty(4, n, 128, dtype=torch.bfloat16, device="cuda").permute(1, 0, 2)
    qb.rope(r, pos, q, q_out=across)
    assert torch.equal(across, qo)
    rest = joint[:, 6:].clone()
    qb.rope(r, pos, q, k, q_out=q, k_out=k)
    assert torch.equal(joint[:, :4], qo) and torch.equal(joint[:, 4:6], ko) and torch.equal(joint[:, 6:], rest)


def test_gradient():
    """The transpose is the gradient: <rope(x), y> = <x, transpose(y)>, and against differences along one direction
    (the map is linear: exact but for roundings, 2^-20 of the sum of absolute products)."""
    r = qb.Rope(96, **WAYS[4])
    x, y, e = (rows(50, 3, 128, torch.float32, s) for s in (1, 2, 3))
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 977
    back = qb.rope(r, pos, y, transpose=True)
    fwd = qb.rope(r, pos, x)
    left, right = (fwd.double() * y.double()).sum(), (x.double() * back.double()).sum()
    size = float((fwd.double() * y.double()).abs().sum() + (x.double() * back.double()).abs().sum())
    assert abs(float(left - right)) <= 2.0 ** -20 * size
    diff = ((qb.rope(r, pos, x + e).double() - qb.rope(r, pos, x - e).double()) * y.double()).sum() / 2
    size = float(((x.double().abs() + e.double().abs()) * back.double().abs()).sum() + (fwd.double().abs() * y.double().abs()).sum()) * 2
    assert abs(float(diff - (e.double() * back.double()).sum())) <= 2.0 ** -20 * size


def test_frequencies_of_its_own():
    f = [0.5, 7.0, 1e-3, 0.0]
    x = rows(9, 2, 16, torch.float32)
    pos = torch.arange(9, dtype=torch.int32, device="cuda") * 100
    got = qb.rope(qb.Rope(8, frequencies=f), pos, x)
    want = ref.turned(x, pos, f)
    assert float((got.double() - want).abs().max()) <= 2.0 ** -21 * 2 * float(x.abs().max())
    assert torch.equal(got[..., [3, 7]], x[..., [3, 7]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("way", range(len(WAYS)))
@pytest.mark.parametrize("hd,dims,n", [(128, 128, 3), (128, 32, 200), (64, 64, 1), (256, 128, 40), (8, 8, 5)])
def test_append(hd, dims, n, way, dtype):
    way = WAYS[way]
    cache = qb.PagedCache.empty(2, 256, 2, hd, page=16)
    q, k, v = rows(n, 6, hd, dtype), rows(n, 2, hd, dtype, 1), rows(n, 2, hd, dtype, 2)
    pos = torch.arange(n, dtype=torch.int32, device="cuda") + 40000
    seq = torch.ones(n, dtype=torch.int32, device="cuda")
    slot = torch.arange(n, dtype=torch.int32, device="cuda")
    r = qb.Rope(dims, **way)
    qo = qb.paged_append(cache, k, v, pos, q=q, seq=seq, slot=slot, rope=r)
    close(qo, q, pos, dims, way)
    flat = lambda t: t.view(2, 256, 2, hd)[1, :n]
    wide = qb.rope(r, pos, k.float())
    assert torch.equal(flat(cache.k), wide.to(torch.bfloat16))
    assert torch.equal(flat(cache.v), v.to(torch.bfloat16))
    assert cache.lens.tolist() == [0, n] and torch.equal(qo, qb.rope(r, pos, q))
    assert qb.query_status() == 0


def test_append_as_theta_does():
    """A plain descriptor turns as rope_theta does, up to the latter's sines (2^-20)."""
    k, v = rows(30, 2, 128, torch.float32), rows(30, 2, 128, torch.float32, 1)
    pos = torch.arange(30, dtype=torch.int32, device="cuda") * 5000
    seq, slot = torch.zeros_like(pos), torch.arange(30, dtype=torch.int32, device="cuda")
    q = [qb.paged_append(qb.PagedCache.empty(1, 64, 2, 128), k, v, pos, q=k, seq=seq, slot=slot, **kw)
         for kw in (dict(rope_theta=1e7), dict(rope=qb.Rope(128, 1e7)))]
    assert float((q[0] - q[1]).abs().max()) <= 2.0 ** -19 * 2 * float(k.abs().max())


@pytest.mark.parametrize("n", [2 ** 29 + 5, 2 ** 31 - 1])
def test_offsets_and_rows_past_32_bits(n):
    """More elements than 32 bits count, and as many rows as they do: the last rows equal a small call's."""
    turn = qb.Rope(8, theta=100.0)
    y = torch.empty(n, 1, 8, dtype=torch.bfloat16, device="cuda")
    x = torch.randn(1, 1, 8, device="cuda").to(torch.bfloat16)
    pos = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    pos[-4:] = torch.tensor([1, 2, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    qb.rope(turn, pos, x.expand(n, 1, 8), q_out=y)
    few = qb.rope(turn, pos[-9:].contiguous(), x.repeat(9, 1, 1))
    assert torch.equal(y[-9:], few) and torch.equal(y[n // 2:n // 2 + 4], few[:4]) and torch.equal(y[:4], few[:4])
