"""Thin Python binding of the C ABI in include/bitnet.h.

Argument marshalling only: PyTorch provides device memory and the current
stream; every step of the computation runs in the library's CUDA kernels.
The binding refuses to run when the shared library is missing (there is no
fallback of any kind).

Function names match the C entry points.  Tensors must live on the CUDA
device; bf16 arrays may be passed as torch.bfloat16 or as 16-bit integer
tensors holding the bit patterns.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbitnet_b200.so")

STATUS = {
    0: "BITNET_OK", 1: "BITNET_ERR_INVALID_ARG", 2: "BITNET_ERR_SHAPE", 3: "BITNET_ERR_ALIGN",
    4: "BITNET_ERR_WORKSPACE", 5: "BITNET_ERR_UNSUPPORTED", 6: "BITNET_ERR_CUDA",
    7: "BITNET_ERR_TIMEOUT", 8: "BITNET_ERR_NONFINITE", 9: "BITNET_ERR_PAGES",
}

# name -> (restype, argtypes)
_P, _I64, _SZ, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "bitnet_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "bitnet_version": (ctypes.c_int, []),
    "bitnet_pack_workspace_size": (_SZ, [_I64, _I64]),
    "bitnet_pack_weights": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "bitnet_quant_act": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, _P]),
    "bitnet_linear_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bitnet_linear": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "bitnet_ffn_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bitnet_ffn": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _F,
                                  _P, _P, _P, _SZ, _P]),
    "bitnet_last_device_status": (ctypes.c_int, [_P]),
    "bitnet_linear_noalloc": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _I64, _P, _P]),
    "bitnet_linear_chain_workspace_size": (_SZ, [_I64, _P, _P, _I64]),
    "bitnet_linear_chain": (ctypes.c_int, [_I64, _P, _P, _P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "bitnet_linear_multi_workspace_size": (_SZ, [_I64, _P, _I64, _I64]),
    "bitnet_linear_multi": (ctypes.c_int, [_I64, _P, _P, _P, _I64, _P, _I64, _P, _P, _SZ, _P]),
    "bitnet_pack_w1_workspace_size": (_SZ, [_I64, _I64]),
    "bitnet_pack_weights_w1": (ctypes.c_int, [_P, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "bitnet_linear_w1_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bitnet_linear_w1": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "bitnet_linear_tl2": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _P, _P, _P, _P]),
    "bitnet_quant_act_a48": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "bitnet_linear_a48_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bitnet_linear_a48": (ctypes.c_int, [_P, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P,
                                         _SZ, _P]),
    "bitnet_ffn_tp_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "bitnet_ffn_tp_gate_up": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P,
                                             _P, _P, _P, _SZ, _P]),
    "bitnet_ffn_tp_down": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "bitnet_ffn_tp_finish": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _F, _P, _P,
                                            _P]),
    "bitnet_attn_prompt": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64,
                                          _I64, _I64, _I64, _F, _P, _I64, _P, _P]),
    "bitnet_attn_decode_workspace_size": (_SZ, [_I64, _I64, _I64, _I64]),
    "bitnet_attn_decode": (ctypes.c_int, [_P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _F,
                                          _P, _I64, _P, _P, _SZ, _P]),
    "bitnet_kv_workspace_size": (_SZ, [_I64, _I64]),
    "bitnet_kv_extend": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _SZ, _P]),
    "bitnet_kv_append": (ctypes.c_int, [_P, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _P,
                                        _P, _P, _P]),
    "bitnet_kv_fork": (ctypes.c_int, [_P, _P, _P, _I64, _P, _P, _P, _P, _SZ, _P]),
    "bitnet_kv_free": (ctypes.c_int, [_P, _P, _I64, _P]),
    "bitnet_kv_compact": (ctypes.c_int, [_P, _P, _P, _P, _P, _SZ, _P]),
    "bitnet_kv_copy_pages": (ctypes.c_int, [_I64, _P, _P, _I64, _I64, _P, _P, _I64, _P]),
}


class FfnDebug(ctypes.Structure):
    _fields_ = [("xq1", _P), ("acc_gate", _P), ("acc_up", _P), ("h", _P), ("xq2", _P),
                ("acc_down", _P), ("y_f32", _P)]


class KvTables(ctypes.Structure):
    _fields_ = [("table", _P), ("lens", _P), ("refs", _P), ("n_slots", _I64), ("max_pages", _I64),
                ("n_pages", _I64), ("page_size", _I64)]


class BitnetError(RuntimeError):
    def __init__(self, func: str, status: int):
        super().__init__(f"{func} failed: {STATUS.get(status, status)}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "ternary_weight_linear_int8_b200/build.py (nvcc, sm_100a)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(name, st):
    if st != 0:
        raise BitnetError(name, st)


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _bits16(t, name):
    _dev(t, name)
    if t.element_size() != 2:
        raise ValueError(f"{name} must hold 16-bit (bf16) elements")
    return t


def _workspace(nbytes, device, ws=None):
    if nbytes == 0:
        return None
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return torch.empty(int(nbytes), dtype=torch.uint8, device=device)


def bitnet_status_string(status: int) -> str:
    return lib().bitnet_status_string(status).decode()


def bitnet_version() -> int:
    return lib().bitnet_version()


def bitnet_pack_weights(W: torch.Tensor, packed=None, gamma=None, workspace=None):
    """W fp32 [N,K] -> (packed uint8 [N,K/4], gamma fp32 [1])."""
    _dev(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    N, K = W.shape
    packed = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device) if packed is None else packed
    gamma = torch.empty(1, dtype=torch.float32, device=W.device) if gamma is None else gamma
    nb = lib().bitnet_pack_workspace_size(N, K)
    ws = _workspace(nb, W.device, workspace)
    st = lib().bitnet_pack_weights(_ptr(W), N, K, _ptr(packed), _ptr(gamma), _ptr(ws), nb, _stream())
    _check("bitnet_pack_weights", st)
    return packed, gamma


def bitnet_quant_act(x: torch.Tensor, with_rowsum: bool = True, xq=None, scale=None,
                     rowsum=None):
    """x bf16 [M,K] -> (x_q int8 [M,K], scale fp32 [M], rowsum int32 [M] or None).
    The outputs may be given as preallocated tensors."""
    _bits16(x, "x")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device) if xq is None else _dev(xq, "xq")
    s = torch.empty(M, dtype=torch.float32, device=x.device) if scale is None else _dev(scale, "scale")
    rs = rowsum if rowsum is not None else (
        torch.empty(M, dtype=torch.int32, device=x.device) if with_rowsum else None)
    st = lib().bitnet_quant_act(_ptr(x), M, K, _ptr(xq), _ptr(s), _ptr(rs), _stream())
    _check("bitnet_quant_act", st)
    return xq, s, rs


def bitnet_linear_workspace_size(M: int, N: int, K: int) -> int:
    return lib().bitnet_linear_workspace_size(M, N, K)


def bitnet_linear(packed: torch.Tensor, gamma: torch.Tensor, x: torch.Tensor, y=None,
                  want_f32: bool = False, want_acc: bool = False, workspace=None,
                  y_f32=None, acc=None):
    """y = BitLinear(x) on packed weights.  Returns (y bf16 [M,N], y_f32, acc).
    `y`, `y_f32` and `acc` may be given as preallocated [M,N] tensors."""
    _dev(packed, "packed")
    _dev(gamma, "gamma")
    _bits16(x, "x")
    N, Kb = packed.shape
    M, K = x.shape
    if K != 4 * Kb:
        raise ValueError("x and packed disagree on K")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    y32 = y_f32 if y_f32 is not None else (
        torch.empty((M, N), dtype=torch.float32, device=x.device) if want_f32 else None)
    acc = acc if acc is not None else (
        torch.empty((M, N), dtype=torch.int32, device=x.device) if want_acc else None)
    for t, name in ((y, "y"), (y32, "y_f32"), (acc, "acc")):
        if t is not None:
            _dev(t, name)
            if tuple(t.shape) != (M, N):
                raise ValueError(f"{name} must have shape [M, N]")
    nb = lib().bitnet_linear_workspace_size(M, N, K)
    ws = _workspace(nb, x.device, workspace)
    st = lib().bitnet_linear(_ptr(packed), _ptr(gamma), N, K, _ptr(x), M, _ptr(y), _ptr(y32),
                             _ptr(acc), _ptr(ws), nb, _stream())
    _check("bitnet_linear", st)
    return y, y32, acc


def bitnet_ffn_workspace_size(M: int, H: int, I: int) -> int:
    return lib().bitnet_ffn_workspace_size(M, H, I)


@dataclass
class FfnWeights:
    gate: torch.Tensor
    gamma_gate: torch.Tensor
    up: torch.Tensor
    gamma_up: torch.Tensor
    down: torch.Tensor
    gamma_down: torch.Tensor
    norm1_w: torch.Tensor | None = None
    norm2_w: torch.Tensor | None = None


def bitnet_ffn(x: torch.Tensor, w: FfnWeights, eps: float = 1e-5, y=None, debug=False,
               workspace=None):
    """Fused FFN block.  Returns (y bf16 [M,H], dict of debug outputs or None).
    `debug` is False, True (the binding allocates the debug outputs) or a dict
    of preallocated tensors with the keys below."""
    _bits16(x, "x")
    M, H = x.shape
    I = w.gate.shape[0]
    dev = x.device
    y = torch.empty((M, H), dtype=torch.bfloat16, device=dev) if y is None else y
    dbg = None
    dstruct = None
    if isinstance(debug, dict):
        dbg = debug
    elif debug:
        dbg = {
            "xq1": torch.empty((M, H), dtype=torch.int8, device=dev),
            "acc_gate": torch.empty((M, I), dtype=torch.int32, device=dev),
            "acc_up": torch.empty((M, I), dtype=torch.int32, device=dev),
            "h": torch.empty((M, I), dtype=torch.float32, device=dev),
            "xq2": torch.empty((M, I), dtype=torch.int8, device=dev),
            "acc_down": torch.empty((M, H), dtype=torch.int32, device=dev),
            "y_f32": torch.empty((M, H), dtype=torch.float32, device=dev),
        }
    if dbg is not None:
        dstruct = FfnDebug(*[_ptr(dbg[k]) for k in
                             ("xq1", "acc_gate", "acc_up", "h", "xq2", "acc_down", "y_f32")])
    nb = lib().bitnet_ffn_workspace_size(M, H, I)
    ws = _workspace(nb, dev, workspace)
    st = lib().bitnet_ffn(_ptr(x), M, H, I, _ptr(w.norm1_w), _ptr(w.gate), _ptr(w.gamma_gate),
                          _ptr(w.up), _ptr(w.gamma_up), _ptr(w.norm2_w), _ptr(w.down),
                          _ptr(w.gamma_down), float(eps), _ptr(y),
                          ctypes.byref(dstruct) if dstruct is not None else None,
                          _ptr(ws), nb, _stream())
    _check("bitnet_ffn", st)
    return y, dbg


def _host_arrays(packs, gammas, ys, x):
    L = len(packs)
    Ns = (ctypes.c_int64 * L)(*[int(p.shape[0]) for p in packs])
    Ks = (ctypes.c_int64 * L)(*[int(p.shape[1]) * 4 for p in packs])
    P = (ctypes.c_void_p * L)(*[p.data_ptr() for p in packs])
    G = (ctypes.c_void_p * L)(*[g.data_ptr() for g in gammas])
    Y = (ctypes.c_void_p * L)(*[y.data_ptr() for y in ys])
    return L, Ns, Ks, P, G, Y


def bitnet_linear_chain_workspace_size(Ns, Ks, M: int) -> int:
    L = len(Ns)
    n = (ctypes.c_int64 * L)(*Ns)
    k = (ctypes.c_int64 * L)(*Ks)
    return lib().bitnet_linear_chain_workspace_size(L, n, k, M)


def bitnet_linear_chain(packs, gammas, x: torch.Tensor, ys=None, workspace=None):
    """Layers l = 0..L-1: y[l] = BitLinear(packs[l], gammas[l])(y[l-1]), y[-1] = x.
    `ys` (optional) are the output tensors, one per layer; a layer's output
    may not be its own input (ping-pong buffers are fine).  Returns ys."""
    _bits16(x, "x")
    if len(packs) != len(gammas) or not packs:
        raise ValueError("packs and gammas must be non-empty lists of equal length")
    M = x.shape[0]
    for p, g in zip(packs, gammas):
        _dev(p, "packed")
        _dev(g, "gamma")
    if ys is None:
        ys = [torch.empty((M, p.shape[0]), dtype=torch.bfloat16, device=x.device) for p in packs]
    for y in ys:
        _bits16(y, "y")
    L, Ns, Ks, P, G, Y = _host_arrays(packs, gammas, ys, x)
    nb = lib().bitnet_linear_chain_workspace_size(L, Ns, Ks, M)
    ws = _workspace(nb, x.device, workspace)
    st = lib().bitnet_linear_chain(L, P, G, Ns, Ks, _ptr(x), M, Y, _ptr(ws), nb, _stream())
    _check("bitnet_linear_chain", st)
    return ys


def bitnet_linear_multi_workspace_size(Ns, K: int, M: int) -> int:
    L = len(Ns)
    n = (ctypes.c_int64 * L)(*Ns)
    return lib().bitnet_linear_multi_workspace_size(L, n, K, M)


def bitnet_linear_multi(packs, gammas, x: torch.Tensor, ys=None, workspace=None):
    """Matrices l = 0..L-1 on one input: y[l] = BitLinear(packs[l], gammas[l])(x)
    (e.g. query/key/value or gate/up projections).  All matrices share K;
    `ys` (optional) are the output tensors, one per matrix, none overlapping
    x or each other.  Returns ys."""
    _bits16(x, "x")
    if len(packs) != len(gammas) or not packs:
        raise ValueError("packs and gammas must be non-empty lists of equal length")
    M, K = x.shape
    for p, g in zip(packs, gammas):
        _dev(p, "packed")
        _dev(g, "gamma")
        if int(p.shape[1]) * 4 != K:
            raise ValueError("every packed matrix must have K/4 columns")
    if ys is None:
        ys = [torch.empty((M, p.shape[0]), dtype=torch.bfloat16, device=x.device) for p in packs]
    for y in ys:
        _bits16(y, "y")
    L, Ns, _, P, G, Y = _host_arrays(packs, gammas, ys, x)
    nb = lib().bitnet_linear_multi_workspace_size(L, Ns, K, M)
    ws = _workspace(nb, x.device, workspace)
    st = lib().bitnet_linear_multi(L, P, G, Ns, K, _ptr(x), M, Y, _ptr(ws), nb, _stream())
    _check("bitnet_linear_multi", st)
    return ys


class PreparedChain:
    """bitnet_linear_chain with its argument arrays and workspace built once:
    calling it enqueues the whole chain with one C call (the layers' device
    pointers, shapes and output buffers are fixed; only x and the stream
    change from call to call)."""

    def __init__(self, packs, gammas, ys, workspace=None):
        if len(packs) != len(gammas) or len(packs) != len(ys) or not packs:
            raise ValueError("packs, gammas and ys must be non-empty lists of equal length")
        for p, g, y in zip(packs, gammas, ys):
            _dev(p, "packed")
            _dev(g, "gamma")
            _bits16(y, "y")
        self.M = ys[0].shape[0]
        self.K0 = packs[0].shape[1] * 4
        self._keep = (list(packs), list(gammas), list(ys))
        self.L, self.Ns, self.Ks, self.P, self.G, self.Y = _host_arrays(packs, gammas, ys, None)
        nb = lib().bitnet_linear_chain_workspace_size(self.L, self.Ns, self.Ks, self.M)
        self.nb = nb
        self.ws = _workspace(nb, ys[0].device, workspace)
        self.ys = ys
        self._fn = lib().bitnet_linear_chain
        self._ws_ptr = _ptr(self.ws)

    def __call__(self, x: torch.Tensor):
        if x.shape[0] != self.M or x.shape[1] != self.K0:
            raise ValueError("x does not match the prepared chain")
        st = self._fn(self.L, self.P, self.G, self.Ns, self.Ks, ctypes.c_void_p(x.data_ptr()),
                      self.M, self.Y, self._ws_ptr, self.nb, _stream())
        _check("bitnet_linear_chain", st)
        return self.ys[-1]

    def capture(self, x: torch.Tensor):
        """Record the chain on the input buffer x into a CUDA graph (one
        eager call first, so that every kernel is loaded) and return a
        function that replays it on the current stream: one launch for the
        whole chain.  New inputs are written into x between replays; the
        result is self.ys[-1].  The graph holds the buffers it was recorded
        on (x, the outputs, the workspace)."""
        if x.shape[0] != self.M or x.shape[1] != self.K0:
            raise ValueError("x does not match the prepared chain")
        side = torch.cuda.Stream(device=x.device)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self(x)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            self(x)
        self._graph = graph
        self._graph_x = x
        return graph.replay


def bitnet_linear_noalloc(packed: torch.Tensor, gamma: torch.Tensor, x: torch.Tensor, y=None):
    """BitLinear using the library's fixed device scratch array instead of a
    workspace (for callers that cannot allocate).  Returns y bf16 [M,N]."""
    _dev(packed, "packed")
    _dev(gamma, "gamma")
    _bits16(x, "x")
    N, Kb = packed.shape
    M, K = x.shape
    if K != 4 * Kb:
        raise ValueError("x and packed disagree on K")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    st = lib().bitnet_linear_noalloc(_ptr(packed), _ptr(gamma), N, K, _ptr(x), M, _ptr(y),
                                     _stream())
    _check("bitnet_linear_noalloc", st)
    return y


def bitnet_linear_w1_workspace_size(M: int, N: int, K: int) -> int:
    return lib().bitnet_linear_w1_workspace_size(M, N, K)


def bitnet_pack_weights_w1(W: torch.Tensor, packed=None, alpha=None, workspace=None):
    """BitNet v1 sign weights: W fp32 [N,K] -> (packed uint8 [N,K/8], alpha fp32 [1])."""
    _dev(W, "W")
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 tensor")
    N, K = W.shape
    packed = torch.empty((N, K // 8), dtype=torch.uint8, device=W.device) if packed is None else packed
    alpha = torch.empty(1, dtype=torch.float32, device=W.device) if alpha is None else alpha
    nb = lib().bitnet_pack_w1_workspace_size(N, K)
    ws = _workspace(nb, W.device, workspace)
    st = lib().bitnet_pack_weights_w1(_ptr(W), N, K, _ptr(packed), _ptr(alpha), _ptr(ws), nb,
                                      _stream())
    _check("bitnet_pack_weights_w1", st)
    return packed, alpha


def bitnet_linear_w1(packed: torch.Tensor, alpha: torch.Tensor, x: torch.Tensor, y=None,
                     want_f32: bool = False, want_acc: bool = False, workspace=None,
                     y_f32=None, acc=None):
    """W1A8 BitLinear on sign-packed weights.  Returns (y bf16 [M,N], y_f32, acc)."""
    _dev(packed, "packed")
    _dev(alpha, "alpha")
    _bits16(x, "x")
    N, Kb = packed.shape
    M, K = x.shape
    if K != 8 * Kb:
        raise ValueError("x and packed disagree on K")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    y32 = y_f32 if y_f32 is not None else (
        torch.empty((M, N), dtype=torch.float32, device=x.device) if want_f32 else None)
    acc = acc if acc is not None else (
        torch.empty((M, N), dtype=torch.int32, device=x.device) if want_acc else None)
    nb = lib().bitnet_linear_w1_workspace_size(M, N, K)
    ws = _workspace(nb, x.device, workspace)
    st = lib().bitnet_linear_w1(_ptr(packed), _ptr(alpha), N, K, _ptr(x), M, _ptr(y), _ptr(y32),
                                _ptr(acc), _ptr(ws), nb, _stream())
    _check("bitnet_linear_w1", st)
    return y, y32, acc


def bitnet_linear_tl2(packed: torch.Tensor, gamma: torch.Tensor, x: torch.Tensor, y=None,
                      want_f32: bool = False, want_acc: bool = False, y_f32=None, acc=None):
    """One-token BitLinear through pair lookup tables (same result as bitnet_linear)."""
    _dev(packed, "packed")
    _dev(gamma, "gamma")
    _bits16(x, "x")
    N, Kb = packed.shape
    M, K = x.shape
    if M != 1 or K != 4 * Kb:
        raise ValueError("x must be [1, K] with K = 4 * packed.shape[1]")
    y = torch.empty((1, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    y32 = y_f32 if y_f32 is not None else (
        torch.empty((1, N), dtype=torch.float32, device=x.device) if want_f32 else None)
    acc = acc if acc is not None else (
        torch.empty((1, N), dtype=torch.int32, device=x.device) if want_acc else None)
    st = lib().bitnet_linear_tl2(_ptr(packed), _ptr(gamma), N, K, _ptr(x), _ptr(y), _ptr(y32),
                                 _ptr(acc), _stream())
    _check("bitnet_linear_tl2", st)
    return y, y32, acc


def bitnet_quant_act_a48(x: torch.Tensor, n_out: int):
    """a4.8 activations: x bf16 [M,K] -> (q4 int8 [M,K], s4 [M], q8 int8 [M,K], s8 [M])."""
    _bits16(x, "x")
    M, K = x.shape
    q4 = torch.empty((M, K), dtype=torch.int8, device=x.device)
    q8 = torch.empty((M, K), dtype=torch.int8, device=x.device)
    s4 = torch.empty(M, dtype=torch.float32, device=x.device)
    s8 = torch.empty(M, dtype=torch.float32, device=x.device)
    st = lib().bitnet_quant_act_a48(_ptr(x), M, K, int(n_out), _ptr(q4), _ptr(s4), _ptr(q8),
                                    _ptr(s8), _stream())
    _check("bitnet_quant_act_a48", st)
    return q4, s4, q8, s8


def bitnet_linear_a48_workspace_size(M: int, N: int, K: int) -> int:
    return lib().bitnet_linear_a48_workspace_size(M, N, K)


def bitnet_linear_a48(packed: torch.Tensor, gamma: torch.Tensor, x: torch.Tensor, n_out: int,
                      y=None, want_f32: bool = False, want_acc: bool = False, workspace=None,
                      y_f32=None, acc4=None, acc8=None):
    """a4.8 BitLinear.  Returns (y bf16 [M,N], y_f32, acc4, acc8)."""
    _dev(packed, "packed")
    _dev(gamma, "gamma")
    _bits16(x, "x")
    N, Kb = packed.shape
    M, K = x.shape
    if K != 4 * Kb:
        raise ValueError("x and packed disagree on K")
    dev = x.device
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    y32 = y_f32 if y_f32 is not None else (
        torch.empty((M, N), dtype=torch.float32, device=dev) if want_f32 else None)
    if want_acc:
        acc4 = torch.empty((M, N), dtype=torch.int32, device=dev) if acc4 is None else acc4
        acc8 = torch.empty((M, N), dtype=torch.int32, device=dev) if acc8 is None else acc8
    nb = lib().bitnet_linear_a48_workspace_size(M, N, K)
    ws = _workspace(nb, dev, workspace)
    st = lib().bitnet_linear_a48(_ptr(packed), _ptr(gamma), N, K, _ptr(x), M, int(n_out), _ptr(y),
                                 _ptr(y32), _ptr(acc4), _ptr(acc8), _ptr(ws), nb, _stream())
    _check("bitnet_linear_a48", st)
    return y, y32, acc4, acc8


def bitnet_ffn_tp_workspace_size(M: int, H: int, Ir: int) -> int:
    return lib().bitnet_ffn_tp_workspace_size(M, H, Ir)


def bitnet_ffn_tp_gate_up(x, gate, gamma_gate, up, gamma_up, norm1_w=None, norm2_w=None,
                          workspace=None):
    """Tensor-parallel FFN step 1 on this shard.  Returns (h [M,Ir] fp32,
    amax2 [M] fp32, sumsq_h [M] fp64, sumsq_x [M] fp64)."""
    _bits16(x, "x")
    M, H = x.shape
    Ir = gate.shape[0]
    dev = x.device
    h = torch.empty((M, Ir), dtype=torch.float32, device=dev)
    amax2 = torch.empty(M, dtype=torch.float32, device=dev)
    ssh = torch.empty(M, dtype=torch.float64, device=dev)
    ssx = torch.empty(M, dtype=torch.float64, device=dev)
    nb = lib().bitnet_ffn_tp_workspace_size(M, H, Ir)
    ws = _workspace(nb, dev, workspace)
    st = lib().bitnet_ffn_tp_gate_up(_ptr(x), M, H, Ir, _ptr(norm1_w), _ptr(gate), _ptr(gamma_gate),
                                     _ptr(up), _ptr(gamma_up), _ptr(norm2_w), _ptr(h), _ptr(amax2),
                                     _ptr(ssh), _ptr(ssx), _ptr(ws), nb, _stream())
    _check("bitnet_ffn_tp_gate_up", st)
    return h, amax2, ssh, ssx


def bitnet_ffn_tp_down(h, down, amax2, norm2_w=None, workspace=None):
    """Tensor-parallel FFN step 3 on this shard: partial int32 accumulators [M,H]."""
    _dev(h, "h")
    M, Ir = h.shape
    H = down.shape[0]
    acc = torch.empty((M, H), dtype=torch.int32, device=h.device)
    nb = lib().bitnet_ffn_tp_workspace_size(M, H, Ir)
    ws = _workspace(nb, h.device, workspace)
    st = lib().bitnet_ffn_tp_down(_ptr(h), M, H, Ir, _ptr(norm2_w), _ptr(down), _ptr(amax2),
                                  _ptr(acc), _ptr(ws), nb, _stream())
    _check("bitnet_ffn_tp_down", st)
    return acc


def bitnet_ffn_tp_finish(acc, I, gamma_down, amax2, sumsq_x, sumsq_h, eps=1e-5, y=None,
                         want_f32=False):
    """Tensor-parallel FFN step 5: y bf16 [M,H] (and y_f32) from the all-reduced values."""
    _dev(acc, "acc")
    M, H = acc.shape
    y = torch.empty((M, H), dtype=torch.bfloat16, device=acc.device) if y is None else y
    y32 = torch.empty((M, H), dtype=torch.float32, device=acc.device) if want_f32 else None
    st = lib().bitnet_ffn_tp_finish(_ptr(acc), M, H, int(I), _ptr(gamma_down), _ptr(amax2),
                                    _ptr(sumsq_x), _ptr(sumsq_h), float(eps), _ptr(y), _ptr(y32),
                                    _stream())
    _check("bitnet_ffn_tp_finish", st)
    return y, y32


# ------------------------------------------------- attention and its cache
# These calls take a few microseconds on the device, so their marshalling is
# kept short: device ordinals instead of device objects, the raw stream handle
# instead of a stream object.
_BITS16 = (torch.bfloat16, torch.int16, torch.uint16)
# (Both are private names that only CUDA builds of torch have: the public calls
# stand in for them, so that importing this file needs neither.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _run(name, dev, *args):
    """Call the entry point `name` on device ordinal `dev` and its current stream."""
    if dev < 0:
        raise ValueError(f"{name}: all tensors must be on a CUDA device")
    fn = getattr(_lib or lib(), name)
    if _current_device() == dev:
        st = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    if st != 0:
        raise BitnetError(name, st)


def _heads(t, name, dev):
    """A [tokens, heads, D] bf16 tensor on device ordinal `dev`, heads contiguous, any token
    stride.  Returns that stride."""
    if dev < 0 or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on the same device as the others")
    if t.dim() != 3 or t.dtype not in _BITS16:
        raise ValueError(f"{name} must be [tokens, heads, D] with 16-bit (bf16) elements")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if n < 1 or (s2 != 1 and d > 1) or (s1 != d and h > 1):
        raise ValueError(f"{name} must have contiguous heads and at least one token")
    return s0 if n > 1 else h * d


def _pages(t, name, pool, dev):
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the pool's device")
    s = t.shape
    if len(s) != 4 or t.dtype not in _BITS16 or s[0] != pool.n_pages or s[2] != pool.page_size:
        raise ValueError(f"{name} must be [n_pages, heads, page_size, D] with 16-bit elements")
    return s


def _index(t, name, dev, n=None):
    """The address of an int32 vector on device ordinal `dev` (None: a null pointer)."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.get_device() != dev or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 vector on the same device")
    if n is not None and t.numel() != n:
        raise ValueError(f"{name} must have {n} elements")
    return t.data_ptr()


def _like(t, name, shape, dtypes, dev):
    """Checks an output given by the caller (contiguous unless checked further)."""
    if t.get_device() != dev or tuple(t.shape) != shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must have shape {list(shape)} and the right type, on the same device")
    return t


def _lse_out(lse, want, shape, dev, device):
    if lse is None:
        return torch.empty(shape, dtype=torch.float32, device=device) if want else None
    return _dev(_like(lse, "lse", shape, (torch.float32,), dev), "lse")


def bitnet_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                       cu_k=None, scale=None, y=None, want_lse: bool = False, lse=None):
    """Causal attention over packed prompts: q [Tq,Hq,D], k and v [Tk,Hkv,D] bf16, sequence i in
    rows cu_q[i] .. cu_q[i+1] and keys cu_k[i] .. (None: cu_q).  scale defaults to D ** -0.5.
    Rows outside all sequences are left as they are.  Returns (y [Tq,Hq,D], lse [Tq,Hq] or None)."""
    dev = q.get_device()
    qs, ks, vs = _heads(q, "q", dev), _heads(k, "k", dev), _heads(v, "v", dev)
    Tq, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if Dk != D or v.shape != k.shape:
        raise ValueError("k and v must be [Tk, Hkv, D] with q's D")
    cq = _index(cu_q, "cu_q", dev)
    n = cu_q.numel()
    ck = cq if cu_k is None else _index(cu_k, "cu_k", dev, n)
    if y is None:
        y = torch.empty((Tq, Hq, D), dtype=torch.bfloat16, device=q.device)
    ys = _heads(_like(y, "y", (Tq, Hq, D), _BITS16, dev), "y", dev)
    if want_lse or lse is not None:
        lse = _lse_out(lse, want_lse, (Tq, Hq), dev, q.device)
    _run("bitnet_attn_prompt", dev, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, cq, ck,
         n - 1, Tq, Tk, Hq, Hkv, D, D ** -0.5 if scale is None else scale, y.data_ptr(), ys,
         None if lse is None else lse.data_ptr())
    return y, lse


class KvPool:
    """Tables of a paged key-value cache (see bitnet_kv_tables): table
    [n_slots, max_pages], lens [n_slots] and refs [n_pages], int32, in one
    allocation.  Built empty by bitnet_kv_pool."""

    def __init__(self, buf, n_slots, max_pages, n_pages, page_size, ws=None):
        if buf.get_device() < 0 or buf.dtype != torch.int32 or buf.dim() != 1 or not buf.is_contiguous() or \
                buf.numel() != n_slots * max_pages + n_slots + n_pages:
            raise ValueError("buf must be a contiguous int32 CUDA vector that holds table, lens and refs")
        self.buf, self.page_size, self.ws = buf, page_size, ws
        self.n_slots, self.max_pages, self.n_pages = n_slots, max_pages, n_pages
        self.dev = buf.get_device()
        a, p = n_slots * max_pages, buf.data_ptr()
        self.c = KvTables(p, p + 4 * a, p + 4 * (a + n_slots), n_slots, max_pages, n_pages, page_size)
        self.ref = ctypes.addressof(self.c)

    @property
    def table(self):
        return self.buf.as_strided((self.n_slots, self.max_pages), (self.max_pages, 1), 0)

    @property
    def lens(self):
        return self.buf.as_strided((self.n_slots,), (1,), self.n_slots * self.max_pages)

    @property
    def refs(self):
        return self.buf.as_strided((self.n_pages,), (1,), self.n_slots * (self.max_pages + 1))

    def clone(self):
        """A copy of the tables (the pages are not part of a pool).  The copy shares the
        scratch: use both on one stream."""
        return KvPool(self.buf.clone(), self.n_slots, self.max_pages, self.n_pages,
                      self.page_size, self.ws)


def bitnet_kv_workspace_size(n_slots: int, n_pages: int) -> int:
    return lib().bitnet_kv_workspace_size(n_slots, n_pages)


def bitnet_kv_pool(n_slots: int, max_pages: int, n_pages: int, page_size: int,
                   device="cuda") -> KvPool:
    """An empty pool with its scratch.  Each layer's pages are [n_pages, Hkv, page_size, D]
    tensors of the caller."""
    nb = lib().bitnet_kv_workspace_size(n_slots, n_pages)
    if nb == 0 or max_pages < 1:
        raise ValueError("n_slots, max_pages or n_pages out of range")
    if torch.device(device).type != "cuda":
        raise ValueError("device must be a CUDA device")
    buf = torch.zeros(n_slots * max_pages + n_slots + n_pages, dtype=torch.int32, device=device)
    pool = KvPool(buf, n_slots, max_pages, n_pages, page_size,
                  torch.empty(nb, dtype=torch.uint8, device=device))
    pool.table.fill_(-1)
    return pool


def bitnet_kv_extend(pool: KvPool, add: torch.Tensor, slots=None, short_pages=None):
    """Sequences (slots, or 0, 1, ...) grow by add[i] tokens.  short_pages (optional int32 [1])
    receives 0, the lacking pages or -1."""
    dev, ws = pool.dev, pool.ws
    n = add.numel()
    ap = _index(add, "add", dev)
    _run("bitnet_kv_extend", dev, pool.ref, _index(slots, "slots", dev, n), ap, n,
         _index(short_pages, "short_pages", dev, 1), ws.data_ptr(), ws.numel())


def bitnet_kv_append(k: torch.Tensor, v: torch.Tensor, cu: torch.Tensor, pool: KvPool,
                     k_pages: torch.Tensor, v_pages: torch.Tensor, slots=None):
    """Rows cu[b] .. cu[b+1] of k and v [T,Hkv,D] become the last tokens of slot b (slots[b])."""
    dev = pool.dev
    ks, vs = _heads(k, "k", dev), _heads(v, "v", dev)
    shape = k.shape
    T, Hkv, D = shape
    if v.shape != shape:
        raise ValueError("k and v must have one shape")
    s = _pages(k_pages, "k_pages", pool, dev)
    if _pages(v_pages, "v_pages", pool, dev) != s or s[1] != Hkv or s[3] != D:
        raise ValueError("k_pages and v_pages must have k's heads and D")
    n = cu.numel() - 1
    _run("bitnet_kv_append", dev, k.data_ptr(), ks, v.data_ptr(), vs, _index(cu, "cu", dev),
         _index(slots, "slots", dev, n), n, T, Hkv, D, pool.ref, k_pages.data_ptr(),
         v_pages.data_ptr())


def bitnet_attn_decode_workspace_size(B: int, Hq: int, Hkv: int, D: int) -> int:
    return lib().bitnet_attn_decode_workspace_size(B, Hq, Hkv, D)


def bitnet_attn_decode(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, pool: KvPool,
                       slots=None, scale=None, y=None, want_lse: bool = False, lse=None,
                       workspace=None):
    """One new token per sequence over the paged cache: q [B,Hq,D], row b reads slot b (slots[b]).
    Returns (y [B,Hq,D], lse [B,Hq] or None)."""
    dev = pool.dev
    qs = _heads(q, "q", dev)
    shape = q.shape
    B, Hq, D = shape
    s = _pages(k_pages, "k_pages", pool, dev)
    if _pages(v_pages, "v_pages", pool, dev) != s or s[3] != D:
        raise ValueError("k_pages and v_pages must have one shape with q's D")
    Hkv = s[1]
    sp = _index(slots, "slots", dev, B)
    if y is None:
        y = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    ys = _heads(_like(y, "y", (B, Hq, D), _BITS16, dev), "y", dev)
    if want_lse or lse is not None:
        lse = _lse_out(lse, want_lse, (B, Hq), dev, q.device)
    if workspace is None:
        nb = lib().bitnet_attn_decode_workspace_size(B, Hq, Hkv, D)
        workspace = torch.empty(max(nb, 1), dtype=torch.uint8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same device")
    _run("bitnet_attn_decode", dev, q.data_ptr(), qs, k_pages.data_ptr(), v_pages.data_ptr(),
         pool.ref, sp, B, Hq, Hkv, D, D ** -0.5 if scale is None else scale, y.data_ptr(), ys,
         None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes)
    return y, lse


def _pair_list(pairs, n_pairs, n, dev, device):
    if pairs is None:
        pairs = torch.empty((n, 2), dtype=torch.int32, device=device)
    else:
        _dev(_like(pairs, "pairs", (n, 2), (torch.int32,), dev), "pairs")
    if n_pairs is None:
        n_pairs = torch.empty(1, dtype=torch.int32, device=device)
    else:
        _like(n_pairs, "n_pairs", (1,), (torch.int32,), dev)
    return pairs, n_pairs


def bitnet_kv_fork(pool: KvPool, parents: torch.Tensor, children: torch.Tensor, short_pages=None,
                   pairs=None, n_pairs=None):
    """Slots children[i] become copies of parents[i].  Returns (pairs [n,2], n_pairs [1]): the page
    copies that bitnet_kv_copy_pages has to make in every layer."""
    dev, ws = pool.dev, pool.ws
    n = parents.numel()
    pp, cp = _index(parents, "parents", dev), _index(children, "children", dev, n)
    pairs, n_pairs = _pair_list(pairs, n_pairs, n, dev, pool.buf.device)
    _run("bitnet_kv_fork", dev, pool.ref, pp, cp, n, pairs.data_ptr(), n_pairs.data_ptr(),
         _index(short_pages, "short_pages", dev, 1), ws.data_ptr(), ws.numel())
    return pairs, n_pairs


def bitnet_kv_free(pool: KvPool, slots: torch.Tensor):
    """Free slots: their pages' counts drop, their rows become empty."""
    sp = _index(slots, "slots", pool.dev)
    _run("bitnet_kv_free", pool.dev, pool.ref, sp, slots.numel())


def bitnet_kv_compact(pool: KvPool, live=None, pairs=None, n_pairs=None):
    """Move the pages in use to the front of the pool.  Returns (pairs, n_pairs) for
    bitnet_kv_copy_pages; live (optional int32 [1]) receives the number of pages in use."""
    dev, ws = pool.dev, pool.ws
    pairs, n_pairs = _pair_list(pairs, n_pairs, max(1, pool.n_pages // 2), dev, pool.buf.device)
    _run("bitnet_kv_compact", dev, pool.ref, pairs.data_ptr(), n_pairs.data_ptr(),
         _index(live, "live", dev, 1), ws.data_ptr(), ws.numel())
    return pairs, n_pairs


def bitnet_kv_copy_pages(k_pages, v_pages, pairs: torch.Tensor, n_pairs: torch.Tensor):
    """Make the listed page copies in every layer: k_pages, v_pages are lists of the layers'
    [n_pages, Hkv, page_size, D] tensors, all of one shape."""
    L = len(k_pages)
    if len(v_pages) != L or not L:
        raise ValueError("k_pages and v_pages must be non-empty lists of equal length")
    first, dev = k_pages[0], n_pairs.get_device()
    if first.dim() != 4 or first.dtype not in _BITS16:
        raise ValueError("pages must be [n_pages, heads, page_size, D] with 16-bit elements")
    n, nbytes, ptrs = first.shape[0], first.nbytes, []
    for ts in (k_pages, v_pages):
        for t in ts:
            if t.nbytes != nbytes or t.get_device() != dev or not t.is_contiguous():
                raise ValueError("all pages must be contiguous CUDA tensors of one size")
            ptrs.append(t.data_ptr())
    np_ = _index(n_pairs, "n_pairs", dev, 1)
    if pairs.dtype != torch.int32 or pairs.dim() != 2 or pairs.shape[1] != 2 or \
            pairs.get_device() != dev or not pairs.is_contiguous():
        raise ValueError("pairs must be a contiguous [n, 2] int32 tensor")
    both = (ctypes.c_void_p * (2 * L))(*ptrs)
    at = ctypes.addressof(both)
    _run("bitnet_kv_copy_pages", dev, L, at, at + 8 * L, n, nbytes // n, pairs.data_ptr(), np_,
         min(pairs.shape[0], n))


def bitnet_last_device_status() -> int:
    """Synchronise the current stream and return (and clear) the device status word."""
    return lib().bitnet_last_device_status(_stream())
