"""The paged cache's entry points refuse bad arguments on the host, before any
GPU work: sizes and types, missing and misaligned pointers, small workspaces."""

import ctypes

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb
from quantized_moe_transformer_gb300 import build

ARG, NULL, ALIGN, WORKSPACE = -1, -2, -3, -4
FAKE = 1 << 20  # never dereferenced by the host checks


@pytest.fixture(scope="module")
def lib():
    build.build()
    return qb._paged_lib()


def desc(**kw):
    d = qb.PagedCacheDesc(3, 2, 128, 64, 40, 10, 64 * 256, 256, 128, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    for name, value in kw.items():
        setattr(d, name, value)
    return d


def append(lib, d=None, q=FAKE, q_out=FAKE, k=FAKE, v=FAKE, dtype=0, seq=None, slot=None, pos=FAKE, rows=3, heads=16,
           theta=1e7):
    return lib.qmoe_paged_append(ctypes.byref(d or desc()), q, q_out, k, v, dtype, seq, slot, pos, rows, heads, theta, None)


def attend(lib, d=None, q=FAKE, out=FAKE, dtype=0, heads=16, scale=0.0, accumulate=1, ws=FAKE, ws_bytes=1 << 40):
    return lib.qmoe_paged_attention(ctypes.byref(d or desc()), q, out, dtype, heads, scale, accumulate, ws, ws_bytes, None)


def evict(lib, d=None, nxt=FAKE, budget=100, recent=10, lens=FAKE, weight=FAKE, pos=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return lib.qmoe_cache_evict(ctypes.byref(d or desc()), nxt, budget, recent, lens, weight, pos, ws, ws_bytes, None)


CACHE_FAULTS = [("n_seqs", 0, ARG), ("n_kv", 0, ARG), ("n_kv", 65536, ARG), ("head_dim", 4, ARG), ("head_dim", 100, ARG),
                ("head_dim", 264, ARG), ("page", 4, ARG), ("page", 48, ARG), ("page", 8192, ARG), ("n_pages", 0, ARG),
                ("max_pages", 0, ARG), ("max_pages", (1 << 24) + 1, ARG), ("page_stride", -8, ARG), ("slot_stride", 12, ARG),
                ("head_stride", 130, ARG), ("k", None, NULL), ("v", None, NULL), ("table", None, NULL),
                ("lens", None, NULL), ("k", FAKE + 8, ALIGN), ("v", FAKE + 2, ALIGN), ("table", FAKE + 2, ALIGN),
                ("weight", FAKE + 4, ALIGN)]


@pytest.mark.parametrize("call", [append, attend, evict])
@pytest.mark.parametrize("field,value,status", CACHE_FAULTS)
def test_cache_descriptor(lib, call, field, value, status):
    d = desc(**{field: value})
    assert call(lib, d) == status
    assert lib.qmoe_cache_evict_workspace_bytes(ctypes.byref(d)) == 0
    assert lib.qmoe_paged_attention_workspace_bytes(ctypes.byref(d), 16, 0) == 0


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 2}, ARG), ({"dtype": -1}, ARG), ({"rows": -1}, ARG), ({"theta": -1.0}, ARG), ({"theta": float("nan")}, ARG),
    ({"theta": float("inf")}, ARG), ({"heads": 0}, ARG), ({"rows": 4}, ARG), ({"q_out": None}, NULL), ({"q": None}, NULL),
    ({"seq": FAKE}, NULL), ({"slot": FAKE}, NULL), ({"k": None}, NULL), ({"v": None}, NULL), ({"pos": None}, NULL),
    ({"q": FAKE + 8}, ALIGN), ({"k": FAKE + 4}, ALIGN), ({"v": FAKE + 2}, ALIGN), ({"pos": FAKE + 1}, ALIGN)])
def test_append_arguments(lib, kw, status):
    assert append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    ({"dtype": 5}, ARG), ({"heads": 0}, ARG), ({"heads": 15}, ARG), ({"heads": 1 << 17}, ARG), ({"scale": float("nan")}, ARG),
    ({"scale": float("inf")}, ARG), ({"q": None}, NULL), ({"out": None}, NULL), ({"ws": None}, NULL),
    ({"q": FAKE + 8}, ALIGN), ({"out": FAKE + 4}, ALIGN), ({"ws": FAKE + 128}, ALIGN), ({"ws_bytes": 16}, WORKSPACE)])
def test_attention_arguments(lib, kw, status):
    assert attend(lib, **kw) == status


def test_attention_without_weights(lib):
    assert attend(lib, desc(weight=None), accumulate=1) == NULL


@pytest.mark.parametrize("kw,status", [
    ({"budget": -1}, ARG), ({"recent": -1}, ARG), ({"recent": 101}, ARG), ({"lens": None}, NULL), ({"weight": None}, NULL),
    ({"pos": None}, NULL), ({"nxt": None}, NULL), ({"ws": None}, NULL), ({"weight": FAKE + 8}, ALIGN),
    ({"pos": FAKE + 4}, ALIGN), ({"lens": FAKE + 1}, ALIGN), ({"ws": FAKE + 16}, ALIGN), ({"ws_bytes": 64}, WORKSPACE)])
def test_evict_arguments(lib, kw, status):
    assert evict(lib, **kw) == status


def test_evict_without_weights_or_positions(lib):
    assert evict(lib, desc(weight=None)) == NULL
    assert evict(lib, desc(pos=None), pos=None) == NULL  # recent needs positions


def test_no_rows_is_a_no_op(lib):
    assert append(lib, rows=0, seq=FAKE, slot=FAKE) == 0


def test_workspaces_grow_with_the_cache(lib):
    small, big = desc(), desc(n_seqs=64, max_pages=256)
    for size in (lib.qmoe_cache_evict_workspace_bytes, lambda d: lib.qmoe_paged_attention_workspace_bytes(d, 16, 1)):
        assert 0 < size(ctypes.byref(small)) <= size(ctypes.byref(big))


def test_binding_refuses_tensors_of_another_kind():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(qb.QmoeError, match="CUDA"):
        qb.PagedCache(k, k.clone(), table, lens)
    with pytest.raises(qb.QmoeError, match="strides"):
        qb.PagedCache(k, k[:2], table, lens)
    with pytest.raises(qb.QmoeError, match="strides"):
        qb.PagedCache(k.transpose(2, 3), k.transpose(2, 3), table, lens)


def block_desc(**kw):
    moe = qb.MoeDesc(2048, 256, 8, 512, 0, 1, FAKE, FAKE, FAKE, FAKE, None, None, None)
    d = qb.BlockDesc(2048, 16, 2, 128, 1e7, 1e-6, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, moe)
    for name, value in kw.items():
        setattr(d, name, value)
    return d


@pytest.mark.parametrize("block_kw,cache_kw,call_kw,status", [
    ({"n_kv": 4}, {}, {}, ARG), ({"head_dim": 64, "n_heads": 32}, {}, {}, ARG), ({"H": 300}, {}, {}, ARG),
    ({}, {"page": 48}, {}, ARG), ({}, {"k": None}, {}, NULL), ({}, {"weight": None}, {}, NULL), ({}, {}, {"X": None}, NULL),
    ({}, {}, {"nxt": None}, NULL), ({}, {}, {"ws": None}, NULL), ({}, {}, {"out": FAKE}, ARG), ({}, {}, {"X": FAKE + 4}, ALIGN),
    ({}, {}, {"ws_bytes": 1000}, WORKSPACE)])
def test_block_decode_arguments(lib, block_kw, cache_kw, call_kw, status):
    a = {"X": FAKE, "out": 2 * FAKE, "nxt": FAKE, "ws": FAKE, "ws_bytes": 1 << 40, **call_kw}
    r = lib.qmoe_block_decode_paged(ctypes.byref(block_desc(**block_kw)), ctypes.byref(desc(**cache_kw)), a["X"], a["out"],
                                    a["nxt"], 1, a["ws"], a["ws_bytes"], None)
    assert r == status


def test_block_decode_workspace(lib):
    b, c = block_desc(), desc()
    n = lib.qmoe_block_decode_paged_workspace_bytes(ctypes.byref(b), ctypes.byref(c), 0)
    assert n > lib.qmoe_paged_attention_workspace_bytes(ctypes.byref(c), 16, 0) > 0
    assert lib.qmoe_block_decode_paged_workspace_bytes(ctypes.byref(b), ctypes.byref(desc(n_kv=1)), 0) == 0
