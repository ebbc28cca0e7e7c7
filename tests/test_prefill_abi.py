"""The entry points that bring prompts into the paged cache refuse bad arguments on the
host, before any GPU work; a rotation's frequencies are those of its formulas."""

import ctypes
import math

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from quantized_moe_transformer_gb300 import build
from tests import prefill_ref as ref
from tests.test_paged_abi import ALIGN, ARG, CACHE_FAULTS, FAKE, NULL, WORKSPACE, desc


@pytest.fixture(scope="module")
def lib():
    build.build()
    return qb._paged_lib()


def rope_desc(**kw):
    d = qb.RopeDesc(0, 64, 1.0)
    for name, value in kw.items():
        setattr(d, name, value)
    return d


def rows(**kw):
    r = qb.RopeRows(FAKE, FAKE, 16, 2048, 128, 2048, 128)
    for name, value in kw.items():
        setattr(r, name, value)
    return r


def init(lib, layout=0, dims=64, theta=1e7, scaling=2, factor=4.0, context=4096.0, low=1.0, high=32.0, scale=1.0):
    return lib.qmoe_rope_init(ctypes.byref(qb.RopeDesc()), layout, dims, theta, scaling, factor, context, low, high, scale)


def rope(lib, d=None, q=None, k=None, dtype=0, pos=FAKE, n_rows=3, hd=128):
    return lib.qmoe_rope(ctypes.byref(d or rope_desc()), ctypes.byref(q or rows()), ctypes.byref(k) if k else None, dtype,
                         pos, n_rows, hd, 0, None)


def append(lib, d=None, rope=None, rows=3, dtype=0):
    return lib.qmoe_paged_append_rope(ctypes.byref(d or desc()), FAKE, FAKE, FAKE, FAKE, dtype, None, None, FAKE, rows, 16,
                                      ctypes.byref(rope or rope_desc()), None)


def plan(lib, d=None, free=FAKE, n_free=FAKE, count=FAKE, keep=FAKE, nxt=FAKE, n_rows=5, first=FAKE, granted=FAKE, seq=FAKE,
         slot=FAKE, pos=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return lib.qmoe_paged_plan(ctypes.byref(d or desc()), free, n_free, count, keep, nxt, n_rows, first, granted, seq, slot,
                               pos, ws, ws_bytes, None)


def attend(lib, d=None, q=FAKE, out=FAKE, dtype=0, first=FAKE, count=FAKE, n_rows=5, heads=16, scale=0.0, ws=FAKE,
           ws_bytes=1 << 40):
    return lib.qmoe_paged_prefill_attention(ctypes.byref(d or desc()), q, out, dtype, first, count, n_rows, heads, scale, ws,
                                            ws_bytes, None)


@pytest.mark.parametrize("call", [append, plan, attend])
@pytest.mark.parametrize("field,value,status", CACHE_FAULTS)
def test_cache_descriptor(lib, call, field, value, status):
    d = desc(**{field: value})
    assert call(lib, d) == status
    assert lib.qmoe_paged_plan_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.qmoe_paged_prefill_attention_workspace_bytes(ctypes.byref(d), 10, 16) == 0


@pytest.mark.parametrize("kw", [
    {"layout": 2}, {"layout": -1}, {"dims": 0}, {"dims": 4}, {"dims": 60}, {"dims": 264}, {"theta": 0.0}, {"theta": -1e4},
    {"theta": float("nan")}, {"theta": float("inf")}, {"scaling": 3}, {"scaling": -1}, {"factor": 0.5}, {"factor": float("nan")},
    {"scaling": 1, "factor": 1e7}, {"context": 0.0}, {"context": float("inf")}, {"low": -1.0}, {"high": 1.0},
    {"high": float("inf")}, {"scale": float("nan")}, {"scale": float("inf")}])
def test_rotations(lib, kw):
    assert init(lib, **kw) == ARG


def test_what_a_scaling_does_not_read_is_not_looked_at(lib):
    bad = dict(factor=0.0, context=-1.0, low=5.0, high=float("nan"))
    assert init(lib, scaling=0, **bad) == 0
    assert init(lib, scaling=1, **(bad | {"factor": 2.0})) == 0
    assert lib.qmoe_rope_init(None, 0, 64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, 1.0) == NULL


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.0), dict(theta=5e5),
                                dict(scaling="parts", factor=8.0, context=8192.0, low=1.0, high=4.0)])
def test_frequencies(kw):
    """turns[i] / 2^64 is f_i / (2 pi), whole turns left out, to 2^-50 of a turn."""
    r = qb.Rope(96, **kw)
    for t, f in zip(r.desc.turns, ref.frequencies(96, **kw)):
        assert abs(t / 2.0 ** 64 - f / (2 * math.pi)) < 2.0 ** -50


@pytest.mark.parametrize("d,status", [({"layout": 5}, ARG), ({"dims": 136}, ARG), ({"dims": 12}, ARG), ({"dims": 0}, ARG),
                                      ({"scale": float("inf")}, ARG)])
def test_descriptors(lib, d, status):
    assert rope(lib, rope_desc(**d)) == status
    assert append(lib, rope=rope_desc(**d)) == status


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, ARG), ({"n_rows": -1}, ARG), ({"hd": 0}, ARG), ({"hd": 100}, ARG), ({"hd": 264}, ARG), ({"hd": 56}, ARG),
    ({"pos": None}, NULL), ({"pos": FAKE + 2}, ALIGN)])
def test_rope_arguments(lib, kw, status):
    assert rope(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"x": None}, NULL), ({"y": None}, NULL), ({"x": FAKE + 8}, ALIGN), ({"y": FAKE + 4}, ALIGN), ({"n_heads": 0}, ARG),
    ({"n_heads": 1 << 17}, ARG), ({"x_row_stride": -8}, ARG), ({"x_head_stride": 12}, ARG), ({"y_row_stride": 4}, ARG),
    ({"y_head_stride": 129}, ARG)])
def test_rope_rows(lib, kw, status):
    assert rope(lib, q=rows(**kw)) == status
    assert rope(lib, k=rows(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    ({"n_rows": -1}, ARG), ({"free": None}, NULL), ({"n_free": None}, NULL), ({"count": None}, NULL), ({"first": None}, NULL),
    ({"granted": None}, NULL), ({"seq": None}, NULL), ({"slot": None}, NULL), ({"pos": None}, NULL), ({"ws": None}, NULL),
    ({"free": FAKE + 2}, ALIGN), ({"keep": FAKE + 1}, ALIGN), ({"nxt": FAKE + 2}, ALIGN), ({"pos": FAKE + 3}, ALIGN),
    ({"ws": FAKE + 16}, ALIGN), ({"ws_bytes": 64}, WORKSPACE)])
def test_plan_arguments(lib, kw, status):
    assert plan(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 3}, ARG), ({"n_rows": -2}, ARG), ({"heads": 0}, ARG), ({"heads": 15}, ARG), ({"heads": 1 << 17}, ARG),
    ({"scale": float("nan")}, ARG), ({"q": None}, NULL), ({"out": None}, NULL), ({"first": None}, NULL), ({"count": None}, NULL),
    ({"ws": None}, NULL), ({"q": FAKE + 8}, ALIGN), ({"out": FAKE + 4}, ALIGN), ({"first": FAKE + 2}, ALIGN),
    ({"count": FAKE + 1}, ALIGN), ({"ws": FAKE + 128}, ALIGN), ({"ws_bytes": 8}, WORKSPACE)])
def test_attention_arguments(lib, kw, status):
    assert attend(lib, **kw) == status


def test_no_rows_is_a_no_op(lib):
    assert attend(lib, n_rows=0, q=None, out=None, ws=None) == 0
    assert rope(lib, n_rows=0) == 0
    assert append(lib, rows=0) == 0


def test_attention_workspace_refuses_what_the_call_refuses(lib):
    f = lib.qmoe_paged_prefill_attention_workspace_bytes
    assert f(ctypes.byref(desc()), 5, 16) > 0 and f(ctypes.byref(desc()), 0, 16) > 0
    assert f(ctypes.byref(desc()), -1, 16) == 0 and f(ctypes.byref(desc()), 5, 15) == 0 and f(ctypes.byref(desc()), 5, 0) == 0


def test_two_ways_to_turn_are_refused(monkeypatch):
    from tests.test_paged_binding import Counted, On, cache, ints
    r = qb.Rope(64)
    seen = Counted()
    monkeypatch.setattr(qb, "_paged_lib", lambda: seen)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 16)
    new = torch.zeros(3, 2, 64)
    with pytest.raises(qb.QmoeError, match="two ways"):
        qb.paged_append(cache(), On(new), On(new), On(ints(3)), rope=r, rope_theta=1e7)
    assert not seen.calls
    qb.paged_append(cache(), On(new), On(new), On(ints(3)), rope=r)
    assert seen.calls == ["qmoe_paged_append_rope"]


def test_python_names_of_a_rotation():
    for kw in (dict(layout="both"), dict(scaling="log"), dict(frequencies=[1.0] * 3), dict(dims=0), dict(frequencies=[float("nan")] * 32)):
        with pytest.raises(qb.QmoeError):
            qb.Rope(**(dict(dims=64) | kw))


def block_desc(**kw):
    d = qb.BlockDesc(2048, 16, 2, 128, 1e7, 1e-6, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                     qb.MoeDesc(2048, 256, 8, 512, 0, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE))
    for name, value in kw.items():
        setattr(d, name, value)
    return d


def prefill(lib, b=None, d=None, X=FAKE, out=2 * FAKE, n_rows=5, first=FAKE, count=FAKE, seq=FAKE, slot=FAKE, pos=FAKE, rope=None,
            ws=FAKE, ws_bytes=1 << 40):
    return lib.qmoe_block_prefill_paged(ctypes.byref(b or block_desc()), ctypes.byref(d or desc()), X, out, n_rows, first, count,
                                        seq, slot, pos, ctypes.byref(rope) if rope else None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    ({"n_rows": -1}, ARG), ({"X": None}, NULL), ({"out": None}, NULL), ({"first": None}, NULL), ({"count": None}, NULL),
    ({"seq": None}, NULL), ({"slot": None}, NULL), ({"pos": None}, NULL), ({"ws": None}, NULL), ({"out": FAKE}, ARG),
    ({"X": FAKE + 8}, ALIGN), ({"out": FAKE + 4}, ALIGN), ({"first": FAKE + 2}, ALIGN), ({"pos": FAKE + 1}, ALIGN),
    ({"ws": FAKE + 64}, ALIGN), ({"ws_bytes": 4096}, WORKSPACE)])
def test_block_arguments(lib, kw, status):
    assert prefill(lib, **kw) == status


def test_block_of_another_cache(lib):
    assert prefill(lib, d=desc(n_kv=4)) == ARG and prefill(lib, d=desc(head_dim=64)) == ARG
    assert prefill(lib, rope=rope_desc(dims=136)) == ARG and prefill(lib, n_rows=0, ws=None) == 0
    assert lib.qmoe_block_prefill_paged_workspace_bytes(ctypes.byref(block_desc()), ctypes.byref(desc(n_kv=4)), 5) == 0
    assert lib.qmoe_block_prefill_paged_workspace_bytes(ctypes.byref(block_desc()), ctypes.byref(desc()), 0) == 0


@pytest.mark.parametrize("kw", [{"granted": 3}, {"count": 3}, {"keep": 3}, {"nxt": 3}, {"free": 3}, {"seq": 3}, {"slot": 3},
                                {"first": "lens"}, {"granted": "lens"}, {"pos": "table"}, {"n_free": "lens"}, {"count": "lens"}])
def test_a_plan_does_not_write_what_it_reads(lib, kw):
    """Two arrays of a plan in one place: ``first`` with another, or one with the cache's own."""
    names = ["free", "n_free", "count", "keep", "nxt", "first", "granted", "seq", "slot", "pos"]
    apart = {n: FAKE + 4096 * (i + 1) for i, n in enumerate(names)}
    own = desc()
    own.lens, own.table = FAKE + 4096 * 20, FAKE + 4096 * 21
    (name, where), = kw.items()
    at = {"lens": own.lens, "table": own.table}.get(where, apart["first"])
    assert plan(lib, own, **{**apart, name: at}) == ARG


@pytest.mark.parametrize("name", ["keep", "nxt"])
def test_a_plan_may_read_the_lengths(lib, name):
    names = ["free", "n_free", "count", "keep", "nxt", "first", "granted", "seq", "slot", "pos"]
    apart = {n: FAKE + 4096 * (i + 1) for i, n in enumerate(names)}
    own = desc()
    own.lens, own.table = FAKE + 4096 * 20, FAKE + 4096 * 21
    if torch.cuda.is_available():
        pytest.skip("the call would run")
    assert plan(lib, own, **{**apart, name: own.lens}) not in (0, NULL, ARG, ALIGN, WORKSPACE)


@pytest.mark.parametrize("kw,n_rows", [({"y_row_stride": 0}, 2), ({"y_head_stride": 0}, 1)])
def test_rows_that_would_be_written_over_one_another(lib, kw, n_rows):
    assert rope(lib, q=rows(**kw), n_rows=n_rows) == ARG
    assert rope(lib, k=rows(**kw), n_rows=n_rows) == ARG


@pytest.mark.parametrize("n_rows", [2 ** 30 + 1, 2 ** 31 - 256, 2 ** 31 - 1])
def test_more_rows_than_32_bits_count(lib, n_rows):
    """A sequence's rows rounded up to whole tiles, and a tile's last place, have to stay below 2^31."""
    assert attend(lib, n_rows=n_rows) == ARG and attend(lib, n_rows=n_rows, dtype=1, d=desc(n_kv=2), heads=6) == ARG
    assert lib.qmoe_paged_prefill_attention_workspace_bytes(ctypes.byref(desc()), n_rows, 16) == 0
    assert lib.qmoe_paged_prefill_attention_workspace_bytes(ctypes.byref(desc()), 2 ** 30, 16) > 0
    assert lib.qmoe_block_prefill_paged_workspace_bytes(ctypes.byref(block_desc()), ctypes.byref(desc()), n_rows) == 0
    assert prefill(lib, n_rows=n_rows, ws_bytes=1 << 62) == ARG


@pytest.mark.parametrize("seqs,pages", [(1, 1), (96, 12000), (5000, 77)])
def test_plan_workspace(lib, seqs, pages):
    """Six numbers a sequence and one a page, each array to 256 bytes, and a head."""
    up = lambda n: -(-n // 256) * 256
    d = desc(n_seqs=seqs, n_pages=pages)
    assert lib.qmoe_paged_plan_workspace_bytes(ctypes.byref(d)) == 256 + 6 * up(4 * seqs) + up(4 * pages)


A, B, C, D = (FAKE + (1 << 20) * i for i in range(4))


@pytest.mark.parametrize("q,k", [
    (dict(x=A, y=A, y_row_stride=4096), None), (dict(x=A, y=A, y_head_stride=256), None), (dict(x=A, y=A, x_row_stride=0), None),
    (dict(x=A, y=B), dict(x=C, y=C, x_head_stride=0)), (dict(x=A, y=B), dict(x=C, y=B)), (dict(x=A, y=B), dict(x=B, y=C)),
    (dict(x=A, y=B), dict(x=C, y=A)), (dict(x=A, y=A), dict(x=A, y=A))])
def test_rows_that_are_written_while_they_are_read(lib, q, k):
    """In place with other strides, or one array's rows where the other's lie."""
    assert rope(lib, q=rows(**q), k=rows(**k) if k else None) == ARG


@pytest.mark.parametrize("q,k", [
    (dict(x=A, y=A), dict(x=B, y=B)), (dict(x=A, y=B), dict(x=A, y=C)), (dict(x=A, y=A, n_heads=1, y_head_stride=64), None),
    (dict(x=A, y=B, x_row_stride=0), dict(x=C, y=D, n_heads=2))])
def test_rows_in_place_and_apart_are_taken(lib, q, k):
    if torch.cuda.is_available():
        pytest.skip("the call would run")
    assert rope(lib, q=rows(**q), k=rows(**k) if k else None) not in (0, NULL, ARG, ALIGN)


@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2)])
def test_outputs_over_a_part_of_the_rows(lib, dtype, size):
    """Rows are read and written in no order: out is q, or apart from it."""
    total = 5 * 16 * 128 * size
    for off in (16, total // 5, total - 16):
        assert attend(lib, q=A, out=A + off, dtype=dtype) == ARG and attend(lib, q=A + off, out=A, dtype=dtype) == ARG
    total = 5 * 2048 * 4
    for off in (16, total - 16):
        assert prefill(lib, X=A, out=A + off) == ARG and prefill(lib, X=A + off, out=A) == ARG


@pytest.mark.parametrize("dtype,size", [(0, 4), (1, 2)])
def test_outputs_in_place_and_apart_are_taken(lib, dtype, size):
    if torch.cuda.is_available():
        pytest.skip("the call would run")
    total = 5 * 16 * 128 * size
    for out in (A, A + total, A - total):
        assert attend(lib, q=A, out=out, dtype=dtype) not in (0, NULL, ARG, ALIGN, WORKSPACE)
