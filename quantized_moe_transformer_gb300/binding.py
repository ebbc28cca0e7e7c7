"""Thin ctypes binding of libqmoe.so (argument marshalling only).

Every step of the layer runs in the library's CUDA kernels; PyTorch supplies
device memory and the current stream. There is no fallback: if the library is
missing or the device is not a GB300, the calls raise.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmoe.so")

Q4K, Q5K, Q6K, MXFP4 = 0, 1, 2, 3
QTYPE = {"q4k": Q4K, "q5k": Q5K, "q6k": Q6K, "mxfp4": MXFP4}
PATH_NAMES = {0: "none", 1: "gemv", 2: "gemm_tc", 3: "decode"}

_c_int, _c_size, _vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p


class MoeDesc(ctypes.Structure):
    _fields_ = [("H", _c_int), ("E", _c_int), ("k", _c_int), ("F", _c_int),
                ("gate_type", _c_int), ("down_type", _c_int),
                ("Wr", _vp), ("Wg", _vp), ("Wu", _vp), ("Wd", _vp),
                ("Sg", _vp), ("Su", _vp), ("Sd", _vp)]


class MoeWsLayout(ctypes.Structure):
    _fields_ = [("ids", _c_size), ("w", _c_size), ("offsets", _c_size), ("perm", _c_size),
                ("y", _c_size)]


class QmoeError(RuntimeError):
    pass


_lib = None


def lib() -> ctypes.CDLL:
    """Loads libqmoe.so (built in-tree by ``quantized_moe_transformer_gb300.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise QmoeError(f"{LIB_PATH} is not built; run quantized_moe_transformer_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER
        L.qmoe_status_str.restype = ctypes.c_char_p
        L.qmoe_status_str.argtypes = [_c_int]
        L.qmoe_query_status.argtypes = [_vp]
        L.qmoe_get_gemm_threshold.argtypes = []
        L.qmoe_set_gemm_threshold.argtypes = [_c_int]
        L.qmoe_set_gemm_threshold.restype = None
        L.qmoe_last_path.argtypes = []
        L.qmoe_moe_route_workspace_bytes.restype = _c_size
        L.qmoe_moe_route_workspace_bytes.argtypes = [_c_int] * 4
        L.qmoe_moe_route.argtypes = [_vp, _vp, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                                     _c_size, _vp]
        L.qmoe_moe_workspace_bytes.restype = _c_size
        L.qmoe_moe_workspace_bytes.argtypes = [P(MoeDesc), _c_int]
        L.qmoe_moe_workspace_layout.argtypes = [P(MoeDesc), _c_int, P(MoeWsLayout)]
        L.qmoe_moe_forward.argtypes = [P(MoeDesc), _vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_size,
                                       _vp]
        L.qmoe_moe_forward_host_workspace_bytes.restype = _c_size
        L.qmoe_moe_forward_host_workspace_bytes.argtypes = [P(MoeDesc), _c_int]
        L.qmoe_moe_forward_host.argtypes = [P(MoeDesc), _vp, _vp, _vp, _c_int, _vp, _c_size, _vp]
        L.qmoe_launch_count.restype = ctypes.c_longlong
        L.qmoe_launch_count.argtypes = []
        L.qmoe_profile_start.argtypes = [_c_int]
        L.qmoe_profile_stop.argtypes = [P(ctypes.c_double), P(_c_int)]
        L.qmoe_profile_read.argtypes = [P(ctypes.c_double), P(_c_int)]
        L.qmoe_moe_forward_noalloc.argtypes = [P(MoeDesc), _vp, _vp, _vp, _c_int, _vp]
        L.qmoe_last_cuda_error.argtypes = []
        L.qmoe_get_decode_max_rows.argtypes = []
        L.qmoe_set_decode_max_rows.argtypes = [_c_int]
        L.qmoe_set_decode_max_rows.restype = None
        L.qmoe_test_inject.argtypes = [_c_int, _c_int]
        _lib = L
    return _lib


def exported_symbols() -> list[str]:
    """Names of the entry points include/qmoe.h declares."""
    return ["qmoe_status_str", "qmoe_query_status", "qmoe_get_gemm_threshold",
            "qmoe_set_gemm_threshold", "qmoe_last_path", "qmoe_moe_route_workspace_bytes",
            "qmoe_moe_route", "qmoe_moe_workspace_bytes", "qmoe_moe_workspace_layout",
            "qmoe_moe_forward", "qmoe_moe_forward_host_workspace_bytes", "qmoe_moe_forward_host",
            "qmoe_launch_count", "qmoe_profile_start", "qmoe_profile_stop", "qmoe_profile_read",
            "qmoe_moe_forward_noalloc", "qmoe_get_decode_max_rows", "qmoe_set_decode_max_rows",
            "qmoe_last_cuda_error", "qmoe_rmsnorm", "qmoe_attn_workspace_bytes", "qmoe_attn_forward", "qmoe_block_workspace_bytes",
            "qmoe_block_forward", "qmoe_test_inject",
            "qmoe_paged_append", "qmoe_paged_attention_workspace_bytes", "qmoe_paged_attention",
            "qmoe_cache_evict_workspace_bytes", "qmoe_cache_evict", "qmoe_block_decode_paged_workspace_bytes",
            "qmoe_block_decode_paged", "qmoe_rope_init", "qmoe_rope", "qmoe_paged_append_rope",
            "qmoe_paged_plan_workspace_bytes", "qmoe_paged_plan", "qmoe_paged_prefill_attention_workspace_bytes",
            "qmoe_paged_prefill_attention", "qmoe_block_prefill_paged_workspace_bytes", "qmoe_block_prefill_paged"]


def _check(status: int):
    if status != 0:
        msg = f"qmoe status {status}: {lib().qmoe_status_str(status).decode()}"
        if status == -6:
            msg += f" (cudaError {int(lib().qmoe_last_cuda_error())})"
        raise QmoeError(msg)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise QmoeError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise QmoeError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _allocating(stream):
    """Where a call allocates its own tensors: under the stream that it runs on. A
    workspace is released at the call's return, and its bytes then go to that
    stream's next work, not to work beside it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


class MoeLayer:
    """Device-resident weights of one routed-MoE layer plus its descriptor."""

    def __init__(self, H, E, k, F, Wr, Wg, Wu, Wd, Sg=None, Su=None, Sd=None,
                 gate_type="q4k", down_type="q5k"):
        self.H, self.E, self.k, self.F = H, E, k, F
        self.gate_type, self.down_type = gate_type, down_type
        self.Wr, self.Wg, self.Wu, self.Wd = Wr, Wg, Wu, Wd
        self.Sg, self.Su, self.Sd = Sg, Su, Sd
        self._desc = MoeDesc(H, E, k, F, QTYPE[gate_type], QTYPE[down_type],
                             _ptr(Wr), _ptr(Wg), _ptr(Wu), _ptr(Wd),
                             _ptr(Sg), _ptr(Su), _ptr(Sd))
        self._desc_ref = ctypes.byref(self._desc)

    @classmethod
    def from_arrays(cls, layer: dict, k: int, device="cuda"):
        """From the numpy dict of ``inputs.moe_layer``."""
        dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(device)
        return cls(layer["H"], layer["E"], k, layer["F"], dev(layer["Wr"]), dev(layer["Wg"]),
                   dev(layer["Wu"]), dev(layer["Wd"]), dev(layer.get("Sg")), dev(layer.get("Su")),
                   dev(layer.get("Sd")), layer["gate_type"], layer["down_type"])

    @property
    def desc(self) -> MoeDesc:
        return self._desc

    def workspace_bytes(self, T: int) -> int:
        return int(lib().qmoe_moe_workspace_bytes(ctypes.byref(self._desc), T))

    def workspace_layout(self, T: int) -> MoeWsLayout:
        out = MoeWsLayout()
        _check(lib().qmoe_moe_workspace_layout(ctypes.byref(self._desc), T, ctypes.byref(out)))
        return out

    def workspace(self, T: int) -> torch.Tensor:
        return torch.empty(max(self.workspace_bytes(T), 256), dtype=torch.uint8,
                           device=self.Wr.device)


def moe_route(X: torch.Tensor, Wr: torch.Tensor, k: int, ws: torch.Tensor | None = None,
              stream=None):
    """ids [T,k] int32 and w [T,k] fp32 of rows X [T,H] under router Wr [H,E]."""
    T, H = X.shape
    E = Wr.shape[1]
    need = int(lib().qmoe_moe_route_workspace_bytes(T, H, E, k))
    with _allocating(stream):
        ids = torch.empty((T, k), dtype=torch.int32, device=X.device)
        w = torch.empty((T, k), dtype=torch.float32, device=X.device)
        if ws is None:
            ws = torch.empty(max(need, 256), dtype=torch.uint8, device=X.device)
    _check(lib().qmoe_moe_route(_ptr(X), _ptr(Wr), T, H, E, k, _ptr(ids), _ptr(w), _ptr(ws),
                                ws.numel(), _stream(stream)))
    return ids, w


def moe_forward(layer: MoeLayer, X: torch.Tensor, R: torch.Tensor | None = None,
                ids: torch.Tensor | None = None, w: torch.Tensor | None = None,
                out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """out = R + shared(X) + sum_s w_s expert_{ids_s}(X), enqueued on ``stream``."""
    T = X.shape[0]
    if out is None or ws is None:
        with _allocating(stream):
            out = torch.empty_like(X) if out is None else out
            ws = layer.workspace(T) if ws is None else ws
    _check(lib().qmoe_moe_forward(ctypes.byref(layer.desc), _ptr(X), _ptr(R), _ptr(ids), _ptr(w),
                                  _ptr(out), T, _ptr(ws), ws.numel(), _stream(stream)))
    return out


FAULT_SITES = {"none": 0, "decode_copy": 1, "tc_arrive": 2, "attn_final": 3, "paged_copy": 4, "prefill_copy": 5,
               "prefill_final": 6}


def test_inject(site: str, wait_us: int = 0):
    """Test-only: make the next calls withhold one copy, arrival or signal at
    ``site`` so that one bounded device wait runs out after ``wait_us``."""
    _check(lib().qmoe_test_inject(FAULT_SITES[site], int(wait_us)))


def query_status(stream=None) -> int:
    return int(lib().qmoe_query_status(_stream(stream)))


def last_path() -> str:
    return PATH_NAMES[int(lib().qmoe_last_path())]


def set_gemm_threshold(rows: int):
    lib().qmoe_set_gemm_threshold(int(rows))


def get_gemm_threshold() -> int:
    return int(lib().qmoe_get_gemm_threshold())


def set_decode_max_rows(rows: int):
    lib().qmoe_set_decode_max_rows(int(rows))


def get_decode_max_rows() -> int:
    return int(lib().qmoe_get_decode_max_rows())


STAGES = {"router": 1, "route": 2, "gateup": 3, "down": 4, "combine": 5, "decode": 6}


def moe_forward_host(layer: MoeLayer, X: torch.Tensor, R: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """The layer on HOST tensors (pinned for asynchronous copies): the library
    copies X (and R) in, runs the layer and copies the result back, then waits."""
    T = X.shape[0]
    if out is None:
        out = torch.empty_like(X)
    if ws is None:
        n = int(lib().qmoe_moe_forward_host_workspace_bytes(ctypes.byref(layer.desc), T))
        with _allocating(stream):
            ws = torch.empty(max(n, 256), dtype=torch.uint8, device=layer.Wr.device)
    for t in (X, R, out):
        if t is not None and (t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous()):
            raise QmoeError("moe_forward_host takes contiguous fp32 host tensors")
    if not ws.is_cuda:
        raise QmoeError("the workspace must be on a CUDA device")
    # (a per-call path: integer addresses and the layer's cached descriptor
    # reference, converted by the argument types declared in lib())
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(lib().qmoe_moe_forward_host(layer._desc_ref, X.data_ptr(), None if R is None else R.data_ptr(),
                                       out.data_ptr(), T, ws.data_ptr(), ws.numel(), s.cuda_stream))
    return out


def host_workspace_bytes(layer: MoeLayer, T: int) -> int:
    return int(lib().qmoe_moe_forward_host_workspace_bytes(ctypes.byref(layer.desc), T))


def launch_count() -> int:
    return int(lib().qmoe_launch_count())


def profile_start(stage: str):
    _check(lib().qmoe_profile_start(STAGES[stage]))


def profile_read():
    """(summed kernel milliseconds, launches) of the profiled launches as the
    last replay of a graph captured with profiling on left them."""
    ms = ctypes.c_double()
    n = _c_int()
    _check(lib().qmoe_profile_read(ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def profile_stop():
    """(summed kernel milliseconds, launches) of the profiled stage."""
    ms = ctypes.c_double()
    n = _c_int()
    _check(lib().qmoe_profile_stop(ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def moe_forward_noalloc(layer: MoeLayer, X: torch.Tensor, R: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The layer with the library's fixed device scratch instead of a caller
    workspace (for callers that cannot allocate); raises for T beyond it."""
    T = X.shape[0]
    if out is None:
        with _allocating(stream):
            out = torch.empty_like(X)
    _check(lib().qmoe_moe_forward_noalloc(ctypes.byref(layer.desc), _ptr(X), _ptr(R), _ptr(out), T,
                                          _stream(stream)))
    return out


# ---------------------------------------------------------------- block

class BlockDesc(ctypes.Structure):
    _fields_ = [("H", _c_int), ("n_heads", _c_int), ("n_kv", _c_int), ("head_dim", _c_int),
                ("rope_theta", ctypes.c_float), ("eps", ctypes.c_float),
                ("g1", _vp), ("g2", _vp), ("Wq", _vp), ("Wk", _vp), ("Wv", _vp), ("Wo", _vp),
                ("moe", MoeDesc)]


def _block_lib():
    L = lib()
    if not getattr(L, "_block_declared", False):
        P = ctypes.POINTER
        L.qmoe_rmsnorm.argtypes = [_vp, _vp, ctypes.c_float, _vp, _c_int, _c_int, _vp]
        L.qmoe_attn_workspace_bytes.restype = _c_size
        L.qmoe_attn_workspace_bytes.argtypes = [P(BlockDesc), _c_int, _c_int]
        L.qmoe_attn_forward.argtypes = [P(BlockDesc), _vp, _vp, _vp, _c_int, _vp, _vp, _c_int, _c_int, _vp,
                                        _c_size, _vp]
        L.qmoe_block_workspace_bytes.restype = _c_size
        L.qmoe_block_workspace_bytes.argtypes = [P(BlockDesc), _c_int, _c_int]
        L.qmoe_block_forward.argtypes = [P(BlockDesc), _vp, _vp, _c_int, _vp, _vp, _c_int, _c_int, _vp,
                                         _c_size, _vp]
        L._block_declared = True
    return L


class Block:
    """Device-resident weights of one attention + MoE block and its descriptor."""

    def __init__(self, H, n_heads, n_kv, head_dim, g1, g2, Wq, Wk, Wv, Wo, moe: MoeLayer,
                 rope_theta=1e7, eps=1e-6):
        self.H, self.n_heads, self.n_kv, self.head_dim = H, n_heads, n_kv, head_dim
        self.g1, self.g2, self.Wq, self.Wk, self.Wv, self.Wo = g1, g2, Wq, Wk, Wv, Wo
        self.moe = moe
        self._desc = BlockDesc(H, n_heads, n_kv, head_dim, rope_theta, eps, _ptr(g1), _ptr(g2), _ptr(Wq),
                               _ptr(Wk), _ptr(Wv), _ptr(Wo), moe.desc)

    @classmethod
    def from_arrays(cls, blk: dict, k: int, device="cuda"):
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)
        moe = MoeLayer.from_arrays(blk["moe"], k, device)
        return cls(blk["H"], blk["n_heads"], blk["n_kv"], blk["head_dim"], dev(blk["g1"]), dev(blk["g2"]),
                   dev(blk["Wq"]), dev(blk["Wk"]), dev(blk["Wv"]), dev(blk["Wo"]), moe)

    @property
    def desc(self) -> BlockDesc:
        return self._desc

    def attn_workspace(self, T, pos0):
        n = int(_block_lib().qmoe_attn_workspace_bytes(ctypes.byref(self._desc), T, pos0))
        return torch.empty(max(n, 256), dtype=torch.uint8, device=self.Wq.device)

    def workspace(self, T, pos0):
        n = int(_block_lib().qmoe_block_workspace_bytes(ctypes.byref(self._desc), T, pos0))
        return torch.empty(max(n, 256), dtype=torch.uint8, device=self.Wq.device)


def cache_from_bits(bits: np.ndarray, device="cuda") -> torch.Tensor:
    """bf16 cache tensor from uint16 bit patterns (same bytes)."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).to(device).view(torch.bfloat16)


def rmsnorm(X: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, out=None, stream=None):
    T, H = X.shape
    if out is None:
        with _allocating(stream):
            out = torch.empty_like(X)
    _check(_block_lib().qmoe_rmsnorm(_ptr(X), _ptr(gamma), eps, _ptr(out), T, H, _stream(stream)))
    return out


def attn_forward(block: Block, X: torch.Tensor, R: torch.Tensor | None, k_cache: torch.Tensor,
                 v_cache: torch.Tensor, pos0: int, out=None, ws=None, stream=None):
    """out = R + O(attention(...)) for rows at positions pos0..pos0+T-1 (R may be None)."""
    T = X.shape[0]
    if out is None or ws is None:
        with _allocating(stream):
            out = torch.empty_like(X) if out is None else out
            ws = block.attn_workspace(T, pos0) if ws is None else ws
    _check(_block_lib().qmoe_attn_forward(ctypes.byref(block.desc), _ptr(X), _ptr(R), _ptr(out), T,
                                          _ptr(k_cache), _ptr(v_cache), pos0, k_cache.shape[0], _ptr(ws),
                                          ws.numel(), _stream(stream)))
    return out


def block_forward(block: Block, X: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, pos0: int,
                  out=None, ws=None, stream=None):
    T = X.shape[0]
    if out is None or ws is None:
        with _allocating(stream):
            out = torch.empty_like(X) if out is None else out
            ws = block.workspace(T, pos0) if ws is None else ws
    _check(_block_lib().qmoe_block_forward(ctypes.byref(block.desc), _ptr(X), _ptr(out), T, _ptr(k_cache),
                                           _ptr(v_cache), pos0, k_cache.shape[0], _ptr(ws), ws.numel(),
                                           _stream(stream)))
    return out


# ---------------------------------------------------------------- paged cache

class PagedCacheDesc(ctypes.Structure):
    _fields_ = [("n_seqs", _c_int), ("n_kv", _c_int), ("head_dim", _c_int), ("page", _c_int), ("n_pages", _c_int),
                ("max_pages", _c_int), ("page_stride", ctypes.c_longlong), ("slot_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("k", _vp), ("v", _vp), ("table", _vp), ("lens", _vp),
                ("weight", _vp), ("pos", _vp)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("layout", _c_int), ("dims", _c_int), ("scale", ctypes.c_float), ("turns", ctypes.c_uint64 * 128)]


class RopeRows(ctypes.Structure):
    _fields_ = [("x", _vp), ("y", _vp), ("n_heads", _c_int), ("x_row_stride", ctypes.c_longlong),
                ("x_head_stride", ctypes.c_longlong), ("y_row_stride", ctypes.c_longlong),
                ("y_head_stride", ctypes.c_longlong)]


_DTYPE = {torch.float32: 0, torch.bfloat16: 1}


_paged = None


def _paged_lib():
    global _paged
    if _paged is None:
        L = lib()
        P = ctypes.POINTER(PagedCacheDesc)
        L.qmoe_paged_append.argtypes = [P, _vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp, _c_int, _c_int, ctypes.c_float,
                                        _vp]
        L.qmoe_paged_attention_workspace_bytes.restype = _c_size
        L.qmoe_paged_attention_workspace_bytes.argtypes = [P, _c_int, _c_int]
        L.qmoe_paged_attention.argtypes = [P, _vp, _vp, _c_int, _c_int, ctypes.c_float, _c_int, _vp, _c_size, _vp]
        L.qmoe_cache_evict_workspace_bytes.restype = _c_size
        L.qmoe_cache_evict_workspace_bytes.argtypes = [P]
        L.qmoe_cache_evict.argtypes = [P, _vp, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_size, _vp]
        L.qmoe_block_decode_paged_workspace_bytes.restype = _c_size
        L.qmoe_block_decode_paged_workspace_bytes.argtypes = [ctypes.POINTER(BlockDesc), P, _c_int]
        L.qmoe_block_decode_paged.argtypes = [ctypes.POINTER(BlockDesc), P, _vp, _vp, _vp, _c_int, _vp, _c_size, _vp]
        R = ctypes.POINTER(RopeDesc)
        L.qmoe_rope_init.argtypes = [R, _c_int, _c_int, ctypes.c_double, _c_int] + [ctypes.c_double] * 4 + [ctypes.c_float]
        L.qmoe_rope.argtypes = [R, ctypes.POINTER(RopeRows), ctypes.POINTER(RopeRows), _c_int, _vp, _c_int, _c_int, _c_int,
                                _vp]
        L.qmoe_paged_append_rope.argtypes = [P, _vp, _vp, _vp, _vp, _c_int, _vp, _vp, _vp, _c_int, _c_int, R, _vp]
        L.qmoe_paged_plan_workspace_bytes.restype = _c_size
        L.qmoe_paged_plan_workspace_bytes.argtypes = [P]
        L.qmoe_paged_plan.argtypes = [P] + [_vp] * 5 + [_c_int] + [_vp] * 6 + [_c_size, _vp]
        L.qmoe_paged_prefill_attention_workspace_bytes.restype = _c_size
        L.qmoe_paged_prefill_attention_workspace_bytes.argtypes = [P, _c_int, _c_int]
        L.qmoe_paged_prefill_attention.argtypes = [P, _vp, _vp, _c_int, _vp, _vp, _c_int, _c_int, ctypes.c_float, _vp,
                                                   _c_size, _vp]
        L.qmoe_block_prefill_paged_workspace_bytes.restype = _c_size
        L.qmoe_block_prefill_paged_workspace_bytes.argtypes = [ctypes.POINTER(BlockDesc), P, _c_int]
        L.qmoe_block_prefill_paged.argtypes = [ctypes.POINTER(BlockDesc), P, _vp, _vp, _c_int] + [_vp] * 5 + [R, _vp, _c_size,
                                                                                                       _vp]
        _paged = L
    return _paged


def _need(t, what, shape, dtype, device):
    """The address of one tensor argument, checked: on this CUDA device,
    contiguous, of this shape and type (one line where all is well: it runs for
    each argument of each call)."""
    if t.get_device() == device and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _need_device(t, what, device)
    if t.dtype is not dtype:
        raise QmoeError(f"{what} has type {t.dtype}, not {dtype}")
    if t.shape != shape:
        raise QmoeError(f"{what} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise QmoeError(f"{what} must be contiguous")


def _need_device(t, what, device):
    if not t.is_cuda:
        raise QmoeError(f"{what} must be on a CUDA device")
    if t.get_device() != device:
        raise QmoeError(f"{what} is on cuda:{t.get_device()}, the cache on cuda:{device}")


def _need_ws(ws, device):
    if not ws.is_cuda or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise QmoeError("the workspace must be a contiguous uint8 tensor on a CUDA device")
    _need_device(ws, "the workspace", device)
    return ws.data_ptr()


def _size(t, dim, what):
    """One size of an argument whose other sizes are checked with its type."""
    try:
        return t.shape[dim]
    except IndexError:
        raise QmoeError(f"{what} has shape {tuple(t.shape)}, not three dimensions") from None


class PagedCache:
    """Keys and values of many sequences in pages, and what eviction goes by.

    k, v [pages][page][kv heads][head dim] bf16 (any strides but the last, the
    same for both), table [sequences][pages of a sequence] int32, lens
    [sequences] int32, weight (fp32) and pos (int32) [sequences][kv heads][slots]
    or None. The cache refers to these tensors; the calls below write them.
    """

    def __init__(self, k, v, table, lens, weight=None, pos=None):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise QmoeError("k and v must be [pages][page][kv heads][head dim] with the same strides, the last 1")
        for t, what in ((k, "k"), (v, "v")):
            if not t.is_cuda:
                raise QmoeError(f"{what} must be on a CUDA device")
            if t.dtype != torch.bfloat16:
                raise QmoeError(f"{what} has type {t.dtype}, not {torch.bfloat16}")
        self.device = dev = k.get_device()  # the calls run on this device
        self.one_of_many = torch.cuda.device_count() > 1
        _need_device(v, "v", dev)
        self.n_pages, self.page, self.n_kv, self.head_dim = k.shape
        if table.dim() != 2:
            raise QmoeError("the table must be [sequences][pages of a sequence]")
        self.n_seqs, self.max_pages = table.shape
        self.slots = self.max_pages * self.page
        per_slot = (self.n_seqs, self.n_kv, self.slots)
        self.k, self.v, self.table, self.lens, self.weight, self.pos = k, v, table, lens, weight, pos
        self._desc = PagedCacheDesc(
            self.n_seqs, self.n_kv, self.head_dim, self.page, self.n_pages, self.max_pages, k.stride(0), k.stride(1),
            k.stride(2), k.data_ptr(), v.data_ptr(), _need(table, "table", table.shape, torch.int32, dev),
            _need(lens, "lens", (self.n_seqs,), torch.int32, dev),
            None if weight is None else _need(weight, "weight", per_slot, torch.float32, dev),
            None if pos is None else _need(pos, "pos", per_slot, torch.int32, dev))
        self._desc_ref = ctypes.byref(self._desc)

    @classmethod
    def empty(cls, n_seqs, max_len, n_kv, head_dim, page=64, n_pages=None, device="cuda"):
        """An empty cache. Without ``n_pages`` every sequence owns the pages of
        ``max_len`` entries; with it the pool has that many and the table is
        filled with -1 for the caller to hand pages out."""
        width = -(-max_len // page)
        if n_pages is None:
            table = torch.arange(n_seqs * width, dtype=torch.int32, device=device).view(n_seqs, width)
            n_pages = n_seqs * width
        else:
            table = torch.full((n_seqs, width), -1, dtype=torch.int32, device=device)
        k = torch.zeros((n_pages, page, n_kv, head_dim), dtype=torch.bfloat16, device=device)
        return cls(k, torch.zeros_like(k), table, torch.zeros(n_seqs, dtype=torch.int32, device=device),
                   torch.zeros((n_seqs, n_kv, width * page), dtype=torch.float32, device=device),
                   torch.zeros((n_seqs, n_kv, width * page), dtype=torch.int32, device=device))

    @property
    def desc(self) -> PagedCacheDesc:
        return self._desc


def _raw_stream(stream, cache):
    """The stream's handle; without one, that of the device's current stream (by
    PyTorch's accessor of the bare handle: 0.1 us against 2.9 us through a
    torch.cuda.Stream object on the GB300's host). The library launches on the
    current device, which has to be the cache's (asked where there is another:
    0.4 us)."""
    return _stream_on(stream, cache.device, "the cache", cache.one_of_many)


def _stream_on(stream, device, what, one_of_many):
    if one_of_many and torch._C._cuda_getDevice() != device:
        raise QmoeError(f"{what} is on cuda:{device}, the current device is cuda:{torch._C._cuda_getDevice()}")
    if stream is not None:
        if stream.device_index != device:
            raise QmoeError(f"the stream is of cuda:{stream.device_index}, {what} on cuda:{device}")
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device)


ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {None: 0, "linear": 1, "parts": 2}


class Rope:
    """How heads turn by their positions: the first ``dims`` elements, in pairs half
    of them apart ("half") or of neighbours ("interleaved"), by theta^(-2i/dims) a
    position, scaled for long contexts ("linear": divided by ``factor``; "parts":
    only where a pair turns less than ``high`` times within ``context`` positions,
    in full below ``low``, and between them by how often it turns; models that blend by
    the pair's number need ``frequencies``), the result times ``scale``. ``frequencies``
    (an angle of one position for each pair) take the place of theta and the scaling."""

    def __init__(self, dims, theta=1e7, layout="half", scaling=None, factor=1.0, context=0.0, low=0.0, high=0.0,
                 scale=1.0, frequencies=None):
        if layout not in ROPE_LAYOUTS or scaling not in ROPE_SCALINGS:
            raise QmoeError(f"no rotary layout {layout!r} with scaling {scaling!r}")
        self.dims, self.desc = dims, RopeDesc()
        self.one_of_many = torch.cuda.device_count() > 1
        kind = ROPE_SCALINGS[scaling if frequencies is None else None]
        _check(_paged_lib().qmoe_rope_init(ctypes.byref(self.desc), ROPE_LAYOUTS[layout], dims, theta, kind, factor, context,
                                           low, high, scale))
        if frequencies is not None:
            if len(frequencies) != dims // 2:
                raise QmoeError(f"{len(frequencies)} frequencies for {dims // 2} pairs")
            for i, f in enumerate(frequencies):
                turn = float(f) / (2 * math.pi)
                if not math.isfinite(turn):
                    raise QmoeError("frequencies must be finite")
                self.desc.turns[i] = int((turn - math.floor(turn)) * 2.0 ** 64) & (2 ** 64 - 1)
        self._ref = ctypes.byref(self.desc)


def _rope_rows(x, y, what, rows, hd, dtype, dev):
    """One array of rows of ``rope`` and where it goes: on this device, of this
    type, [rows][heads][hd] with elements one after the other (one condition where all
    is well, as in _need)."""
    heads = _size(x, 1, what)
    shape, xs, ys = (rows, heads, hd), x.stride(), y.stride()
    if (x.shape == shape and y.shape == shape and x.dtype is dtype and y.dtype is dtype and x.get_device() == dev
            and y.get_device() == dev and xs[2] == 1 and ys[2] == 1):
        return RopeRows(x.data_ptr(), y.data_ptr(), heads, xs[0], xs[1], ys[0], ys[1])
    for t, name in ((x, what), (y, f"{what}_out")):
        if not t.is_cuda or t.get_device() != dev:
            raise QmoeError(f"{name} must be on cuda:{dev}, as pos is")
        if t.dtype is not dtype:
            raise QmoeError(f"{name} has type {t.dtype}, not {dtype}")
        if t.shape != shape:
            raise QmoeError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    raise QmoeError(f"the elements of a head of {what} or {what}_out must be one after the other")


def rope(rope: Rope, pos, q, k=None, q_out=None, k_out=None, transpose: bool = False, stream=None):
    """Rows q [rows][heads][hd] and k [rows][kv heads][hd] (fp32 or bf16; any row and
    head strides that are multiples of 8, such as parts of a joint projection) turned
    by their positions ``pos`` [rows] int32; ``transpose``: turned back (times the
    scale), which takes gradients of the results to those of the rows. Returns q_out
    and k_out, new tensors by default; they may be q and k."""
    dtype, dev, hd = q.dtype, pos.get_device(), _size(q, 2, "q")
    rows = q.shape[0]
    if dtype not in _DTYPE:
        raise QmoeError(f"q has type {dtype}, not fp32 or bf16")
    at = _need(pos, "pos", (rows,), torch.int32, dev)
    if not pos.is_cuda:
        raise QmoeError("pos must be on a CUDA device")
    if k is None and k_out is not None:
        raise QmoeError("k_out without k")
    if q_out is None or (k is not None and k_out is None):
        with _allocating(stream):
            q_out = torch.empty(q.shape, dtype=dtype, device=q.device) if q_out is None else q_out
            k_out = torch.empty(k.shape, dtype=dtype, device=k.device) if k is not None and k_out is None else k_out
    rq = _rope_rows(q, q_out, "q", rows, hd, dtype, dev)
    rk = None if k is None else ctypes.byref(_rope_rows(k, k_out, "k", rows, hd, dtype, dev))
    _check(_paged_lib().qmoe_rope(rope._ref, ctypes.byref(rq), rk, _DTYPE[dtype], at, rows, hd, int(transpose),
                                  _stream_on(stream, dev, "pos", rope.one_of_many)))
    return q_out if k is None else (q_out, k_out)


def paged_append(cache: PagedCache, k, v, pos, q=None, q_out=None, seq=None, slot=None, rope_theta: float = 0.0,
                 stream=None, rope: Rope | None = None):
    """Rows k, v [rows][kv heads][hd] (fp32 or bf16) into the cache: row n to
    slot ``slot[n]`` of sequence ``seq[n]`` (both None: row n is the next entry
    of sequence n; a slot below 0: not cached), at position ``pos[n]``, keys (and
    the queries q [rows][heads][hd], returned) rotated when ``rope_theta`` > 0,
    or as ``rope`` says."""
    rows = _size(k, 0, "k")
    dtype, dev = k.dtype, cache.device
    if dtype not in _DTYPE:
        raise QmoeError(f"k has type {dtype}, not fp32 or bf16")
    kv_shape = (rows, cache.n_kv, cache.head_dim)
    heads = 0
    if q is not None:
        heads = _size(q, 1, "q")
        if q_out is None:
            with _allocating(stream):
                q_out = torch.empty_like(q)
        q_shape = (rows, heads, cache.head_dim)
        qp, qo = _need(q, "q", q_shape, dtype, dev), _need(q_out, "q_out", q_shape, dtype, dev)
    elif q_out is not None:
        raise QmoeError("q_out without q")
    else:
        qp = qo = None
    args = (cache._desc_ref, qp, qo, _need(k, "k", kv_shape, dtype, dev), _need(v, "v", kv_shape, dtype, dev), _DTYPE[dtype],
            None if seq is None else _need(seq, "seq", (rows,), torch.int32, dev),
            None if slot is None else _need(slot, "slot", (rows,), torch.int32, dev),
            _need(pos, "pos", (rows,), torch.int32, dev), rows, heads)
    if rope is None:
        _check(_paged_lib().qmoe_paged_append(*args, rope_theta, _raw_stream(stream, cache)))
    elif rope_theta:
        raise QmoeError("rope_theta and rope are two ways to say how rows turn: give one")
    else:
        _check(_paged_lib().qmoe_paged_append_rope(*args, rope._ref, _raw_stream(stream, cache)))
    return q_out


def paged_attention_workspace(cache: PagedCache, n_heads: int, accumulate: bool = False) -> torch.Tensor:
    n = int(_paged_lib().qmoe_paged_attention_workspace_bytes(cache._desc_ref, n_heads, int(accumulate)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.k.device)


def paged_attention(cache: PagedCache, q, out=None, scale: float = 0.0, accumulate: bool = False, ws=None,
                    stream=None):
    """Attention of one new token q [sequences][heads][hd] (fp32 or bf16) for
    each sequence over its cached entries; with ``accumulate`` every entry's
    weight grows by the attention it received. scale 0: 1/sqrt(hd)."""
    dtype = q.dtype
    if dtype not in _DTYPE:
        raise QmoeError(f"q has type {dtype}, not fp32 or bf16")
    heads = _size(q, 1, "q")
    shape = (cache.n_seqs, heads, cache.head_dim)
    if out is None or ws is None:
        with _allocating(stream):
            out = torch.empty_like(q) if out is None else out
            ws = paged_attention_workspace(cache, heads, accumulate) if ws is None else ws
    dev = cache.device
    _check(_paged_lib().qmoe_paged_attention(
        cache._desc_ref, _need(q, "q", shape, dtype, dev), _need(out, "out", shape, dtype, dev), _DTYPE[dtype], heads,
        scale, int(accumulate), _need_ws(ws, dev), ws.numel(), _raw_stream(stream, cache)))
    return out


def paged_prefill_attention_workspace(cache: PagedCache, n_rows: int, n_heads: int) -> torch.Tensor:
    n = int(_paged_lib().qmoe_paged_prefill_attention_workspace_bytes(cache._desc_ref, n_rows, n_heads))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.k.device)


def paged_prefill_attention(cache: PagedCache, q, first, count, out=None, scale: float = 0.0, ws=None, stream=None):
    """Causal attention of packed rows q [rows][heads][hd] (fp32 or bf16): rows
    first[b] .. first[b] + count[b] - 1 are the last count[b] entries of sequence b,
    appended before, and each sees the entries up to its own. Rows of no sequence
    are not written (a new ``out`` holds zeros there). scale 0: 1/sqrt(hd)."""
    dtype = q.dtype
    if dtype not in _DTYPE:
        raise QmoeError(f"q has type {dtype}, not fp32 or bf16")
    rows, heads = _size(q, 0, "q"), _size(q, 1, "q")
    shape = (rows, heads, cache.head_dim)
    if out is None or ws is None:
        with _allocating(stream):
            out = torch.zeros_like(q) if out is None else out
            ws = paged_prefill_attention_workspace(cache, rows, heads) if ws is None else ws
    dev = cache.device
    _check(_paged_lib().qmoe_paged_prefill_attention(
        cache._desc_ref, _need(q, "q", shape, dtype, dev), _need(out, "out", shape, dtype, dev), _DTYPE[dtype],
        _need(first, "first", (cache.n_seqs,), torch.int32, dev), _need(count, "count", (cache.n_seqs,), torch.int32, dev),
        rows, heads, scale, _need_ws(ws, dev), ws.numel(), _raw_stream(stream, cache)))
    return out


class PagePool:
    """The free pages of a cache's pools, a stack: ``free`` [pages] int32, of which the
    first ``n_free`` [1] int32 are free, the last of them the next to go."""

    def __init__(self, free, n_free):
        self.free, self.n_free = free, n_free

    @classmethod
    def full(cls, cache: PagedCache):
        """All pages of a cache free, page 0 the first to go. The cache's table must name none."""
        n = cache.n_pages
        return cls(torch.arange(n - 1, -1, -1, dtype=torch.int32, device=cache.k.device),
                   torch.full((1,), n, dtype=torch.int32, device=cache.k.device))


def paged_plan_workspace(cache: PagedCache) -> torch.Tensor:
    n = int(_paged_lib().qmoe_paged_plan_workspace_bytes(cache._desc_ref))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.k.device)


def paged_plan(cache: PagedCache, pool: PagePool, count, keep=None, next_pos=None, n_rows: int | None = None, first=None,
               granted=None, seq=None, slot=None, pos=None, ws=None, stream=None):
    """The pages and slots of a step's new rows, count[b] for each sequence, after
    sequence b was cut to its first keep[b] entries (below 0, or without ``keep``: left as it
    is) and the pages behind them went back to ``pool``. Returns (first, granted, seq, slot,
    pos): each sequence's first row of ``n_rows`` and how many rows it was granted (all
    or none), each row's sequence, slot (-1: not granted) and position (next_pos[b] and on). The
    length of ``seq`` is n_rows where it is given."""
    dev, seqs = cache.device, (cache.n_seqs,)
    if n_rows is None:
        if seq is None:
            raise QmoeError("a plan needs n_rows or an array of that length for seq")
        n_rows = _size(seq, 0, "seq")
    rows = (n_rows,)
    if first is None or granted is None or seq is None or slot is None or pos is None or ws is None:
        if n_rows < 0:
            raise QmoeError("n_rows is below 0")
        with _allocating(stream):
            new = lambda t, n: torch.empty(n, dtype=torch.int32, device=cache.k.device) if t is None else t
            first, granted = new(first, seqs), new(granted, seqs)
            seq, slot, pos = new(seq, rows), new(slot, rows), new(pos, rows)
            ws = paged_plan_workspace(cache) if ws is None else ws
    i32 = torch.int32
    _check(_paged_lib().qmoe_paged_plan(
        cache._desc_ref, _need(pool.free, "the pool's pages", (cache.n_pages,), i32, dev),
        _need(pool.n_free, "the pool's count", (1,), i32, dev), _need(count, "count", seqs, i32, dev),
        None if keep is None else _need(keep, "keep", seqs, i32, dev),
        None if next_pos is None else _need(next_pos, "next_pos", seqs, i32, dev), n_rows, _need(first, "first", seqs, i32, dev),
        _need(granted, "granted", seqs, i32, dev), _need(seq, "seq", rows, i32, dev), _need(slot, "slot", rows, i32, dev),
        _need(pos, "pos", rows, i32, dev), _need_ws(ws, dev), ws.numel(), _raw_stream(stream, cache)))
    return first, granted, seq, slot, pos


def cache_evict_workspace(cache: PagedCache) -> torch.Tensor:
    n = int(_paged_lib().qmoe_cache_evict_workspace_bytes(cache._desc_ref))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.k.device)


def cache_evict(cache: PagedCache, next_pos, budget: int, recent: int = 0, lens_out=None, weight_out=None,
                pos_out=None, ws=None, stream=None):
    """Brings every sequence to at most ``budget`` entries for each KV head: those
    at positions >= next_pos - recent and the heaviest of the others. Without
    outputs the cache's own lens, weight and pos are updated; (lens, weight, pos)
    are returned."""
    lens_out = cache.lens if lens_out is None else lens_out
    weight_out = cache.weight if weight_out is None else weight_out
    pos_out = cache.pos if pos_out is None else pos_out
    if weight_out is None:
        raise QmoeError("the cache has no weights to evict by")
    per_slot, dev = (cache.n_seqs, cache.n_kv, cache.slots), cache.device
    if ws is None:
        with _allocating(stream):
            ws = cache_evict_workspace(cache)
    _check(_paged_lib().qmoe_cache_evict(
        cache._desc_ref, None if next_pos is None else _need(next_pos, "next_pos", (cache.n_seqs,), torch.int32, dev),
        budget, recent, _need(lens_out, "lens_out", (cache.n_seqs,), torch.int32, dev),
        _need(weight_out, "weight_out", per_slot, torch.float32, dev),
        None if pos_out is None else _need(pos_out, "pos_out", per_slot, torch.int32, dev), _need_ws(ws, dev),
        ws.numel(), _raw_stream(stream, cache)))
    return lens_out, weight_out, pos_out


def block_decode_paged_workspace(block: Block, cache: PagedCache, accumulate: bool = False) -> torch.Tensor:
    n = int(_paged_lib().qmoe_block_decode_paged_workspace_bytes(ctypes.byref(block.desc), cache._desc_ref,
                                                                 int(accumulate)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.k.device)


def block_decode_paged(block: Block, cache: PagedCache, X, next_pos, out=None, accumulate: bool = False, ws=None,
                       stream=None):
    """The block for one new token X [sequences][H] fp32 of each sequence: its key
    and value become the sequence's next entry (at position ``next_pos``), its
    query attends to every entry; the lengths grow by one."""
    shape = (cache.n_seqs, block.H)
    if out is None or ws is None:
        with _allocating(stream):
            out = torch.empty_like(X) if out is None else out
            ws = block_decode_paged_workspace(block, cache, accumulate) if ws is None else ws
    dev = cache.device
    _need_device(block.Wq, "the block", dev)
    _check(_paged_lib().qmoe_block_decode_paged(
        ctypes.byref(block.desc), cache._desc_ref, _need(X, "X", shape, torch.float32, dev),
        _need(out, "out", shape, torch.float32, dev), _need(next_pos, "next_pos", (cache.n_seqs,), torch.int32, dev),
        int(accumulate), _need_ws(ws, dev), ws.numel(), _raw_stream(stream, cache)))
    return out


def block_prefill_paged_workspace(block: Block, cache: PagedCache, n_rows: int) -> torch.Tensor:
    n = int(_paged_lib().qmoe_block_prefill_paged_workspace_bytes(ctypes.byref(block.desc), cache._desc_ref, n_rows))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=cache.k.device)


def block_prefill_paged(block: Block, cache: PagedCache, X, first, count, seq, slot, pos, rope: Rope | None = None,
                        out=None, ws=None, stream=None):
    """The block for packed rows X [rows][H] fp32 of many sequences' prompts, parts of
    prompts and single tokens, placed as ``paged_plan`` says (``count``: the rows granted): their
    keys and values are appended, and each row attends to its sequence's entries up to
    its own. ``rope``: how queries and keys turn, by the block's theta without it."""
    rows, dev = X.shape[0] if X.dim() else 0, cache.device
    shape, seqs, per_row, i32 = (rows, block.H), (cache.n_seqs,), (rows,), torch.int32
    if out is None or ws is None:
        with _allocating(stream):
            out = torch.empty_like(X) if out is None else out
            ws = block_prefill_paged_workspace(block, cache, rows) if ws is None else ws
    _need_device(block.Wq, "the block", dev)
    _check(_paged_lib().qmoe_block_prefill_paged(
        ctypes.byref(block.desc), cache._desc_ref, _need(X, "X", shape, torch.float32, dev),
        _need(out, "out", shape, torch.float32, dev), rows, _need(first, "first", seqs, i32, dev),
        _need(count, "count", seqs, i32, dev), _need(seq, "seq", per_row, i32, dev), _need(slot, "slot", per_row, i32, dev),
        _need(pos, "pos", per_row, i32, dev), None if rope is None else rope._ref, _need_ws(ws, dev), ws.numel(),
        _raw_stream(stream, cache)))
    return out
