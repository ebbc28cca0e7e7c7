"""What the paged cache's Python calls refuse before the library is called: tensors,
streams and a current device other than the cache's. The tensors say that they are
on a device; the library is one that counts its calls."""

from types import SimpleNamespace

import pytest
import torch

from quantized_moe_transformer_gb300 import binding as qb


class On:
    """A host tensor that says it is on CUDA device ``index``."""

    def __init__(self, t, index=1):
        self.t, self.index, self.is_cuda, self.device = t, index, True, SimpleNamespace(index=index)

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Counted:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def fake(monkeypatch):
    """The calls made to the library; the current device is 1 of 2."""
    seen = Counted()
    monkeypatch.setattr(qb, "_paged_lib", lambda: seen)
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 16 + device)
    return seen


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache_tensors():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    return {"k": k, "v": k.clone(), "table": ints(3, 2), "lens": ints(3), "weight": torch.zeros(3, 2, 32), "pos": ints(3, 2, 32)}


def cache():
    return qb.PagedCache(**{name: On(t) for name, t in cache_tensors().items()})


def arguments(call):
    rows, ws = torch.zeros(3, 2, 64), torch.zeros(256, dtype=torch.uint8)
    q, X = torch.zeros(3, 8, 64), torch.zeros(3, 256)
    return {"append": {"k": rows, "v": rows, "pos": ints(3), "q": q, "q_out": q, "seq": ints(3), "slot": ints(3)},
            "attend": {"q": q, "out": q, "ws": ws},
            "evict": {"next_pos": ints(3), "lens_out": ints(3), "weight_out": torch.zeros(3, 2, 32), "pos_out": ints(3, 2, 32),
                      "ws": ws},
            "decode": {"X": X, "next_pos": ints(3), "out": X, "ws": ws}}[call]


def run(call, a, stream=None):
    c = cache()
    if call == "append":
        return qb.paged_append(c, a.pop("k"), a.pop("v"), a.pop("pos"), **a, stream=stream)
    if call == "attend":
        return qb.paged_attention(c, a.pop("q"), **a, stream=stream)
    if call == "evict":
        return qb.cache_evict(c, a.pop("next_pos"), 10, **a, stream=stream)
    block = SimpleNamespace(H=256, Wq=a.pop("block", On(torch.zeros(1))), desc=qb.BlockDesc())
    return qb.block_decode_paged(block, c, a.pop("X"), a.pop("next_pos"), **a, stream=stream)


CALLS = ["append", "attend", "evict", "decode"]


@pytest.mark.parametrize("call", CALLS)
def test_calls_on_the_caches_device(fake, call):
    run(call, {name: On(t) for name, t in arguments(call).items()})
    run(call, {name: On(t) for name, t in arguments(call).items()}, SimpleNamespace(device_index=1, cuda_stream=5))
    assert len(fake.calls) == 2


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in arguments(c)] + [("decode", "block")])
@pytest.mark.parametrize("index", [0, -1])
def test_a_tensor_elsewhere(fake, call, name, index):
    a = {n: On(t) for n, t in arguments(call).items()}
    t = torch.zeros(1) if name == "block" else arguments(call)[name]
    a[name] = On(t, 0) if index == 0 else t
    with pytest.raises(qb.QmoeError, match="cuda:0, the cache on cuda:1" if index == 0 else "CUDA device"):
        run(call, a)
    assert not fake.calls


@pytest.mark.parametrize("name", ["v", "table", "lens", "weight", "pos"])
def test_a_cache_over_two_devices(fake, name):
    tensors = {n: On(t) for n, t in cache_tensors().items()}
    tensors[name].index = 0
    with pytest.raises(qb.QmoeError, match="cuda:0, the cache on cuda:1"):
        qb.PagedCache(**tensors)


@pytest.mark.parametrize("call", CALLS)
def test_another_current_device(fake, monkeypatch, call):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(qb.QmoeError, match="current device is cuda:0"):
        run(call, {name: On(t) for name, t in arguments(call).items()})
    assert not fake.calls


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device(fake, call):
    with pytest.raises(qb.QmoeError, match="stream is of cuda:0"):
        run(call, {name: On(t) for name, t in arguments(call).items()}, SimpleNamespace(device_index=0, cuda_stream=5))
    assert not fake.calls


@pytest.mark.parametrize("call,name", [("append", "k"), ("append", "q"), ("attend", "q")])
@pytest.mark.parametrize("shape", [(), (3,), (3, 8), (3, 8, 64, 1)])
def test_rows_of_another_rank(fake, call, name, shape):
    a = {n: On(t) for n, t in arguments(call).items()}
    a[name] = On(torch.zeros(shape))
    with pytest.raises(qb.QmoeError, match="has shape"):
        run(call, a)
    assert not fake.calls
