"""What the Python calls around packed rows refuse before the library is called: tensors,
streams and a current device other than the cache's (for ``rope``, than the positions').
The tensors say that they are on a device; the library is one that counts its calls."""

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


def arguments(call):
    """Five rows of three sequences."""
    q, X, ws = torch.zeros(5, 8, 64), torch.zeros(5, 256), torch.zeros(256, dtype=torch.uint8)
    maps = {"seq": ints(5), "slot": ints(5), "pos": ints(5)}
    return {"plan": {"free": ints(4), "n_free": ints(1), "count": ints(3), "keep": ints(3), "next_pos": ints(3), "first": ints(3),
                     "granted": ints(3), **maps, "ws": ws},
            "attend": {"q": q, "first": ints(3), "count": ints(3), "out": q, "ws": ws},
            "block": {"X": X, "first": ints(3), "count": ints(3), **maps, "out": X, "ws": ws},
            "append": {"k": q[:, :2].contiguous(), "v": q[:, :2].contiguous(), **maps, "q": q, "q_out": q},
            "rope": {"pos": ints(5), "q": q, "k": q[:, :2], "q_out": q, "k_out": q[:, :2]}}[call]


CALLS = ["plan", "attend", "block", "append", "rope"]


def run(call, a, stream=None):
    a = dict(a)
    turn = qb.Rope(64)
    qb._paged_lib().calls.clear()
    if call == "rope":
        return qb.rope(turn, **a, stream=stream)
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    c = qb.PagedCache(On(k), On(k.clone()), On(ints(3, 2)), On(ints(3)))
    if call == "plan":
        return qb.paged_plan(c, qb.PagePool(a.pop("free"), a.pop("n_free")), **a, n_rows=5, stream=stream)
    if call == "attend":
        return qb.paged_prefill_attention(c, **a, stream=stream)
    if call == "append":
        return qb.paged_append(c, **a, rope=turn, stream=stream)
    block = SimpleNamespace(H=256, Wq=a.pop("block", On(torch.zeros(1))), desc=qb.BlockDesc())
    return qb.block_prefill_paged(block, c, **a, rope=turn, stream=stream)


def on(call):
    return {name: On(t) for name, t in arguments(call).items()}


@pytest.mark.parametrize("call", CALLS)
def test_calls_on_the_device(fake, call):
    run(call, on(call))
    assert len(fake.calls) == 1
    run(call, on(call), SimpleNamespace(device_index=1, cuda_stream=5))
    assert len(fake.calls) == 1


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in arguments(c)] + [("block", "block")])
@pytest.mark.parametrize("index", [0, -1])
def test_a_tensor_elsewhere(fake, call, name, index):
    a = on(call)
    t = torch.zeros(1) if name == "block" else arguments(call)[name]
    a[name] = On(t, 0) if index == 0 else t
    with pytest.raises(qb.QmoeError, match="cuda:|CUDA device"):
        run(call, a)
    assert not fake.calls


@pytest.mark.parametrize("call", CALLS)
def test_another_current_device(fake, monkeypatch, call):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(qb.QmoeError, match="current device is cuda:0"):
        run(call, on(call))
    assert not fake.calls


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device(fake, call):
    with pytest.raises(qb.QmoeError, match="stream is of cuda:0"):
        run(call, on(call), SimpleNamespace(device_index=0, cuda_stream=5))
    assert not fake.calls


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in arguments(c) if n != "ws"])
def test_another_type(fake, call, name):
    a = on(call)
    t = arguments(call)[name]
    a[name] = On(t.to(torch.float16 if t.dtype is torch.float32 else torch.int64))
    with pytest.raises(qb.QmoeError, match="type"):
        run(call, a)
    assert not fake.calls


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in arguments(c) if n != "ws"])
def test_another_shape(fake, call, name):
    for shape in ((), (7,), (5, 3, 64), (5, 8, 64, 1)):
        t = arguments(call)[name]
        if (call, name, len(shape)) in {("rope", "q", 3), ("rope", "k", 3), ("attend", "q", 3), ("append", "q", 3)}:
            continue  # another number of heads is another call
        a = on(call)
        a[name] = On(torch.zeros(shape, dtype=t.dtype))
        with pytest.raises(qb.QmoeError, match="shape|dimension"):
            run(call, a)
        assert not fake.calls


@pytest.mark.parametrize("name", ["q", "q_out", "k", "k_out"])
def test_heads_whose_elements_lie_apart(fake, name):
    a = on("rope")
    a[name] = On(torch.zeros(5, 64, 8 if name[0] == "q" else 2).transpose(1, 2))
    with pytest.raises(qb.QmoeError, match="one after the other"):
        run("rope", a)
    assert not fake.calls


def test_outputs_of_nothing(fake):
    with pytest.raises(qb.QmoeError, match="without k"):
        run("rope", {n: t for n, t in on("rope").items() if n != "k"})
    a = {n: t for n, t in on("plan").items() if n != "seq"}
    with pytest.raises(qb.QmoeError, match="n_rows"):
        c = qb.PagedCache(*[On(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)) for _ in "kv"], On(ints(3, 2)), On(ints(3)))
        qb.paged_plan(c, qb.PagePool(a.pop("free"), a.pop("n_free")), **a)
    assert not fake.calls
