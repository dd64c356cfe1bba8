"""Thin ctypes binding of libmoe.so.

Argument marshalling only: each function takes torch device tensors, allocates
outputs and the workspace with torch on the same device, passes raw pointers
and the current HIP stream to the C ABI, and turns a non-zero status into an
exception.  Every step of the layer runs in the library's HIP kernels; there is
no fallback of any kind, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_HIP"}
EXPORTS = ("moe_route", "moe_permute", "moe_grouped_ffn", "moe_combine", "moe_layer_forward", "moe_newton_schulz",
           "moe_grouped_ffn_backward", "moe_combine_backward", "moe_route_backward", "moe_layer_backward",
           "moe_layer_forward_noalloc", "moe_block_norm", "moe_block_norm_backward", "moe_w4_quantize", "moe_w4_pack",
           "moe_w4_dequantize", "moe_w4_matvec", "moe_w4_grouped_ffn")


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


_lib: Optional[ctypes.CDLL] = None

_i64, _int, _vp, _szp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)
_f32 = ctypes.c_float
_SIGS = {
    "moe_route": [_i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_permute": [_i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_grouped_ffn": [_i64, _i64, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_combine": [_i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp],
    "moe_layer_forward": [_i64, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                          _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_layer_forward_noalloc": [_i64, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _vp, _vp, _vp],
    "moe_newton_schulz": [_i64, _i64, _i64, _int, _i64, _f32, _f32, _f32, _f32, _vp, _vp, _vp, _szp, _vp],
    "moe_grouped_ffn_backward": [_i64, _i64, _i64, _i64, _int, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_combine_backward": [_i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
    "moe_route_backward": [_i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           _szp, _vp],
    "moe_layer_backward": [_i64, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_block_norm": [_i64, _i64, _i64, _int, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _int, _f32, _f32, _f32,
                       _vp, _vp, _vp, _vp, _vp],
    "moe_block_norm_backward": [_i64, _i64, _int, _vp, _vp, _vp, _i64, _int, _f32, _f32, _f32, _vp, _vp, _vp, _vp,
                                _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_w4_quantize": [_i64, _i64, _i64, _int, _i64, _vp, _vp, _vp, _vp],
    "moe_w4_pack": [_i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp],
    "moe_w4_dequantize": [_i64, _i64, _i64, _int, _i64, _vp, _vp, _vp, _vp],
    "moe_w4_matvec": [_i64, _i64, _i64, _int, _i64, _vp, _vp, _vp, _vp, _vp, _szp, _vp],
    "moe_w4_grouped_ffn": [_i64, _i64, _i64, _i64, _int, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                           _vp, _vp, _szp, _vp],
}

GATE_ACTS = {"none": 0, "sigmoid": 1, "tanh": 2}

MUON_COEFFS = (3.4445, -4.7750, 2.0315)


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        _lib = L
    return _lib


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return MOE_F32
    if dt == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported dtype {dt}")


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _raw_stream(dev: torch.device):
    """_stream without building torch's stream object: 0.1 us instead of 2, which counts next to a 3 us launch."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _check(fn: str, st: int):
    if st != 0:
        raise MoEError(fn, st)


def _query(fn: str, *args) -> int:
    """Workspace size for a call (the same arguments with ws = NULL)."""
    n = ctypes.c_size_t(0)
    _check(fn, getattr(lib(), fn)(*args, None, ctypes.byref(n), None))
    return n.value


def _ws(nbytes: int, dev) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)


def moe_route(x, w_router, k: int, bias=None, want_logits: bool = True):
    """Router GEMM + softmax + top-k.  Returns (topk_ids, topk_w, logits|None)."""
    T, d = x.shape
    E = w_router.shape[0]
    dev = x.device
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    w = torch.empty(T, k, dtype=torch.float32, device=dev)
    logits = torch.empty(T, E, dtype=torch.float32, device=dev) if want_logits else None
    head = (T, d, E, k, dtype_code(x.dtype), _p(x), _p(w_router), _p(bias), _p(logits), _p(ids), _p(w))
    need = _query("moe_route", *head)
    ws = _ws(need, dev)
    n = ctypes.c_size_t(ws.numel())
    _check("moe_route", lib().moe_route(*head, _p(ws), ctypes.byref(n), _stream(dev)))
    return ids, w, logits


def moe_permute(x, topk_ids, num_experts: int, copy_rows: bool = True):
    """Returns (offsets [E+1], row_token [T*k], slot_row [T,k], x_perm [T*k, d] | None).
    copy_rows=False produces only the indices (x_perm is None)."""
    T, d = x.shape
    k = topk_ids.shape[1]
    dev = x.device
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    row_token = torch.empty(T * k, dtype=torch.int32, device=dev)
    slot_row = torch.empty(T, k, dtype=torch.int32, device=dev)
    x_perm = torch.empty(T * k, d, dtype=x.dtype, device=dev) if copy_rows else None
    head = (T, d, num_experts, k, dtype_code(x.dtype), _p(x), _p(topk_ids), _p(offsets), _p(row_token),
            _p(slot_row), _p(x_perm))
    ws = _ws(_query("moe_permute", *head), dev)
    n = ctypes.c_size_t(ws.numel())
    _check("moe_permute", lib().moe_permute(*head, _p(ws), ctypes.byref(n), _stream(dev)))
    return offsets, row_token, slot_row, x_perm


def moe_grouped_ffn(x_in, offsets, w_gate, w_up, w_down, y_perm=None, a_rows=None, n_max=None, gu_out=None):
    """y_perm [n_max, d]: the SwiGLU FFN of each expert over its rows.  Without
    a_rows, x_in is x_perm (rows grouped by expert); with a_rows (row_token from
    moe_permute), x_in is the token matrix x read in place.  gu_out [n_max, 2F]
    (optional) receives the gate and up pre-activations for the backward."""
    d = x_in.shape[1]
    if a_rows is None:
        n_max, n_in = x_in.shape[0], 0
    else:
        n_max, n_in = (a_rows.numel() if n_max is None else n_max), x_in.shape[0]
    E, F, _ = w_gate.shape
    dev = x_in.device
    if y_perm is None:
        y_perm = torch.empty(n_max, d, dtype=x_in.dtype, device=dev)
    head = (n_max, d, E, F, dtype_code(x_in.dtype), _p(x_in), n_in, _p(a_rows), _p(offsets), _p(w_gate), _p(w_up),
            _p(w_down), _p(y_perm), _p(gu_out))
    ws = _ws(_query("moe_grouped_ffn", *head), dev)
    n = ctypes.c_size_t(ws.numel())
    _check("moe_grouped_ffn", lib().moe_grouped_ffn(*head, _p(ws), ctypes.byref(n), _stream(dev)))
    return y_perm


def moe_combine(y_perm, slot_row, topk_w, out=None):
    """y [T, d] = sum_j topk_w[t, j] * y_perm[slot_row[t, j]]."""
    T, k = slot_row.shape
    d = y_perm.shape[1]
    y = torch.empty(T, d, dtype=y_perm.dtype, device=y_perm.device) if out is None else out
    _check("moe_combine", lib().moe_combine(T, d, k, dtype_code(y_perm.dtype), _p(y_perm), _p(slot_row),
                                            _p(topk_w), _p(y), _stream(y_perm.device)))
    return y


class GroupedFfnBackward:
    """moe_grouped_ffn_backward with its outputs and workspace allocated once.
    x_in is x_perm, or (a_rows given) the token matrix read through a_rows; gu
    the forward's gate/up pre-activations (moe_grouped_ffn's gu_out), or None to
    recompute them."""

    def __init__(self, x_in, offsets, w_gate, w_up, w_down, dy_perm, a_rows=None, gu=None):
        E, F, d = w_gate.shape
        n_max = dy_perm.shape[0]
        dev = dy_perm.device
        n_in = x_in.shape[0] if a_rows is not None else 0
        self.t = (x_in, offsets, w_gate, w_up, w_down, dy_perm, a_rows, gu)
        self.dx = torch.empty(n_max, d, dtype=dy_perm.dtype, device=dev)
        self.dwg = torch.empty(E, F, d, dtype=torch.float32, device=dev)
        self.dwu = torch.empty(E, F, d, dtype=torch.float32, device=dev)
        self.dwd = torch.empty(E, d, F, dtype=torch.float32, device=dev)
        self.head = (n_max, d, E, F, dtype_code(dy_perm.dtype))
        self.mid = (_p(x_in), n_in, _p(a_rows), _p(offsets), _p(w_gate), _p(w_up), _p(w_down), _p(dy_perm),
                    _p(gu), _p(self.dx), _p(self.dwg), _p(self.dwu), _p(self.dwd))
        self.ws = _ws(_query("moe_grouped_ffn_backward", *self.head, *self.mid), dev)

    def __call__(self):
        n = ctypes.c_size_t(self.ws.numel())
        _check("moe_grouped_ffn_backward",
               lib().moe_grouped_ffn_backward(*self.head, *self.mid, _p(self.ws), ctypes.byref(n),
                                              _stream(self.dx.device)))
        return self.dx, self.dwg, self.dwu, self.dwd


def moe_grouped_ffn_backward(x_in, offsets, w_gate, w_up, w_down, dy_perm, a_rows=None, gu=None):
    """(dx_perm, dW_gate, dW_up, dW_down) of the grouped SwiGLU FFN."""
    return GroupedFfnBackward(x_in, offsets, w_gate, w_up, w_down, dy_perm, a_rows, gu)()


def moe_combine_backward(dy, y_perm, slot_row, topk_w, dy_perm=None):
    """Backward of moe_combine: returns (dy_perm, d_topk_w).  dy_perm rows that no
    slot refers to are left as allocated (zero when allocated here)."""
    T, k = slot_row.shape
    d = dy.shape[1]
    dev = dy.device
    if dy_perm is None:
        dy_perm = torch.zeros(y_perm.shape[0], d, dtype=dy.dtype, device=dev)
    g = torch.empty(T, k, dtype=torch.float32, device=dev)
    _check("moe_combine_backward",
           lib().moe_combine_backward(T, d, k, dtype_code(dy.dtype), _p(dy), _p(y_perm), _p(slot_row), _p(topk_w),
                                      _p(dy_perm), _p(g), _stream(dev)))
    return dy_perm, g


def moe_route_backward(x, w_router, topk_ids, topk_w, d_topk_w, dx_perm=None, slot_row=None, want_bias=True,
                       want_dlogits=False):
    """Backward of moe_route (plus the permutation's when dx_perm and slot_row are
    given).  Returns (dx, dW_router, dbias | None, dlogits | None)."""
    T, d = x.shape
    E = w_router.shape[0]
    k = topk_ids.shape[1]
    dev = x.device
    dx = torch.empty(T, d, dtype=x.dtype, device=dev)
    dwr = torch.empty(E, d, dtype=torch.float32, device=dev)
    db = torch.empty(E, dtype=torch.float32, device=dev) if want_bias else None
    dl = torch.empty(T, E, dtype=torch.float32, device=dev) if want_dlogits else None
    head = (T, d, E, k, dtype_code(x.dtype), _p(x), _p(w_router), _p(topk_ids), _p(topk_w), _p(d_topk_w),
            _p(dx_perm), _p(slot_row), _p(dx), _p(dwr), _p(db), _p(dl))
    ws = _ws(_query("moe_route_backward", *head), dev)
    n = ctypes.c_size_t(ws.numel())
    _check("moe_route_backward", lib().moe_route_backward(*head, _p(ws), ctypes.byref(n), _stream(dev)))
    return dx, dwr, db, dl


class LayerBackward:
    """moe_layer_backward with its outputs and workspace allocated once.  The
    forward's routing (topk_ids, topk_w) and expert outputs y_perm (rows in the
    permutation's order) are inputs; w_router None means pre-routed slots; gu the
    forward's gate/up pre-activations (moe_layer_forward's want_gu), or None to
    recompute them."""

    def __init__(self, x, w_router, w_gate, w_up, w_down, topk_ids, topk_w, y_perm, dy, want_bias: bool = True,
                 want_d_topk_w: bool = False, gu=None):
        T, d = x.shape
        E, F, _ = w_gate.shape
        k = topk_ids.shape[1]
        dev = x.device
        routed = w_router is not None
        self.t = (x, w_router, w_gate, w_up, w_down, topk_ids, topk_w, y_perm, gu, dy)
        self.dx = torch.empty(T, d, dtype=x.dtype, device=dev)
        self.dw_router = torch.empty(E, d, dtype=torch.float32, device=dev) if routed else None
        self.dbias = torch.empty(E, dtype=torch.float32, device=dev) if (routed and want_bias) else None
        self.dw_gate = torch.empty(E, F, d, dtype=torch.float32, device=dev)
        self.dw_up = torch.empty(E, F, d, dtype=torch.float32, device=dev)
        self.dw_down = torch.empty(E, d, F, dtype=torch.float32, device=dev)
        self.d_topk_w = torch.empty(T, k, dtype=torch.float32, device=dev) if want_d_topk_w else None
        self._head = (T, d, E, k, F, dtype_code(x.dtype), _p(x), _p(w_router), _p(w_gate), _p(w_up), _p(w_down),
                      _p(topk_ids), _p(topk_w), _p(y_perm), _p(gu), _p(dy), _p(self.dx), _p(self.dw_router),
                      _p(self.dbias), _p(self.dw_gate), _p(self.dw_up), _p(self.dw_down), _p(self.d_topk_w))
        self.ws = _ws(_query("moe_layer_backward", *self._head), dev)
        self._n = ctypes.c_size_t(self.ws.numel())
        self._ws_p = _p(self.ws)

    def __call__(self):
        _check("moe_layer_backward", lib().moe_layer_backward(*self._head, self._ws_p, ctypes.byref(self._n),
                                                              _stream(self.dx.device)))
        return self


def moe_layer_backward(x, w_router, w_gate, w_up, w_down, topk_ids, topk_w, y_perm, dy, want_bias=True,
                       want_d_topk_w=False, gu=None):
    """One call of the whole layer backward; returns the LayerBackward object
    holding dx, dw_router, dbias, dw_gate, dw_up, dw_down and d_topk_w."""
    return LayerBackward(x, w_router, w_gate, w_up, w_down, topk_ids, topk_w, y_perm, dy, want_bias,
                         want_d_topk_w, gu)()


class NewtonSchulz:
    """moe_newton_schulz on a fixed batch [n, R, C] (bf16) with its output and
    workspace allocated once."""

    def __init__(self, g, steps: int = 5, coeffs=MUON_COEFFS, eps: float = 1e-7):
        if g.dim() == 2:
            g = g.unsqueeze(0)
        self.g, self.steps, self.coeffs, self.eps = g, steps, coeffs, eps
        n, R, C = g.shape
        self.args = (n, R, C, dtype_code(g.dtype), steps, *coeffs, eps)
        self.x = torch.empty_like(g)
        self.ws = _ws(_query("moe_newton_schulz", *self.args, _p(g), _p(self.x)), g.device)

    def __call__(self):
        n = ctypes.c_size_t(self.ws.numel())
        _check("moe_newton_schulz", lib().moe_newton_schulz(*self.args, _p(self.g), _p(self.x), _p(self.ws),
                                                            ctypes.byref(n), _stream(self.g.device)))
        return self.x


def moe_newton_schulz(g, steps: int = 5, coeffs=MUON_COEFFS, eps: float = 1e-7):
    """Muon's Newton-Schulz orthogonalisation of g [R, C] or [n, R, C] (bf16)."""
    out = NewtonSchulz(g, steps, coeffs, eps)()
    return out if g.dim() == 3 else out[0]


class LayerForward:
    """moe_layer_forward with its outputs and workspace allocated once, so that
    repeated calls (benchmarks, graph capture) allocate nothing."""

    def __init__(self, x, w_router, bias, w_gate, w_up, w_down, k: int, topk_ids=None, topk_w=None,
                 want_logits: bool = False, want_routing: bool = False, want_offsets: bool = False,
                 want_y_perm: bool = False, want_gu: bool = False):
        self.x, self.w_router, self.bias = x, w_router, bias
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        T, d = x.shape
        E, F, _ = w_gate.shape
        self.T, self.d, self.E, self.k, self.F = T, d, E, k, F
        dev = x.device
        self.y = torch.empty(T, d, dtype=x.dtype, device=dev)
        routed = w_router is not None
        self.logits = torch.empty(T, E, dtype=torch.float32, device=dev) if (routed and want_logits) else None
        if routed:
            self.topk_ids = torch.empty(T, k, dtype=torch.int32, device=dev) if want_routing else None
            self.topk_w = torch.empty(T, k, dtype=torch.float32, device=dev) if want_routing else None
        else:
            self.topk_ids, self.topk_w = topk_ids, topk_w
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if want_offsets else None
        # training: the expert outputs and gate/up pre-activations the backward takes
        self.y_perm = torch.empty(T * k, d, dtype=x.dtype, device=dev) if want_y_perm else None
        self.gu = torch.empty(T * k, 2 * F, dtype=x.dtype, device=dev) if want_gu else None
        self._head = (T, d, E, k, F, dtype_code(x.dtype), _p(x), _p(w_router), _p(bias), _p(w_gate), _p(w_up),
                      _p(w_down), _p(self.y), _p(self.logits), _p(self.topk_ids), _p(self.topk_w),
                      _p(self.offsets), _p(self.y_perm), _p(self.gu))
        self.ws = _ws(_query("moe_layer_forward", *self._head), dev)
        self._n = ctypes.c_size_t(self.ws.numel())
        self._ws_p = _p(self.ws)

    def __call__(self):
        _check("moe_layer_forward", lib().moe_layer_forward(*self._head, self._ws_p, ctypes.byref(self._n),
                                                            _stream(self.x.device)))
        return self.y


def moe_layer_forward(x, w_router, bias, w_gate, w_up, w_down, k: int, topk_ids=None, topk_w=None,
                      want_logits=False, want_routing=False, want_offsets=False, want_y_perm=False, want_gu=False):
    """One call of the whole layer; returns the LayerForward object holding y
    and the optional outputs."""
    L = LayerForward(x, w_router, bias, w_gate, w_up, w_down, k, topk_ids, topk_w, want_logits, want_routing,
                     want_offsets, want_y_perm, want_gu)
    L()
    return L


def _typed(name: str, *args):
    """Arguments as objects of the call's own types, which ctypes otherwise makes again at every
    call (1.5 us instead of 1.8 for the twenty of moe_block_norm)."""
    return tuple(a if a is None or isinstance(a, t) else t(a) for a, t in zip(args, _SIGS[name]))


def _with_ws(name: str, head, dev: torch.device):
    """A workspace of the size that the call asks for, and the call's arguments up to the stream."""
    ws = _ws(_query(name, *head), dev)
    return ws, (*head, _p(ws), ctypes.byref(ctypes.c_size_t(ws.numel())))


def _launch(name: str, dev: torch.device, args):
    """One call on dev's current stream, with dev as the current device."""
    fn = getattr(lib(), name)
    if dev.index == torch.cuda.current_device():
        st = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    _check(name, st)


def _same(name: str, t: Optional[torch.Tensor], dev, dtype, shape):
    """Checks one operand: where it is given, it has this device, type and shape and is dense."""
    if t is None:
        return
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _gate_args(gate, gate_rows: int, gate_act: str, T: int, d: int, dev, dtype):
    if gate_act not in GATE_ACTS:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACTS)}")
    if gate is None:
        return 0, 0, GATE_ACTS[gate_act]
    if gate_rows < 1:
        raise ValueError("gate_rows must be at least 1")
    groups = -(-T // gate_rows)
    _same("gate", gate, dev, dtype, (groups, d))
    return groups, gate_rows, GATE_ACTS[gate_act]


class BlockNorm:
    """moe_block_norm with its outputs allocated once.  The block's output is y, or
    (y_perm, slot_row, topk_w) as moe_combine takes it, or nothing (the norm before a
    first block).  Calling it fills and returns the object: out, h and y_out are None
    where they are not computed.  out=x writes the new residual stream over x."""

    def __init__(self, x, y=None, y_perm=None, slot_row=None, topk_w=None, post_gain=None, gate=None,
                 gate_rows: int = 0, gate_act: str = "none", next_gain=None, res_scale: float = 1.0,
                 branch_scale: float = 1.0, eps: float = 1e-6, out=None, want_y: bool = False):
        T, d = x.shape
        dev, dt = x.device, x.dtype
        k = n_rows = 0
        _same("x", x, dev, dt, (T, d))
        _same("y", y, dev, dt, (T, d))
        if y_perm is not None:
            if slot_row is None or topk_w is None or slot_row.dim() != 2:
                raise ValueError("y_perm needs slot_row [T, k] and topk_w [T, k]")
            k, n_rows = slot_row.shape[1], y_perm.shape[0]
            _same("y_perm", y_perm, dev, dt, (n_rows, d))
            _same("slot_row", slot_row, dev, torch.int32, (T, k))
            _same("topk_w", topk_w, dev, torch.float32, (T, k))
        _same("post_gain", post_gain, dev, torch.float32, (d,))
        _same("next_gain", next_gain, dev, torch.float32, (d,))
        _, rows, act = _gate_args(gate, gate_rows, gate_act, T, d, dev, dt)
        branch = y is not None or y_perm is not None
        _same("out", out, dev, dt, (T, d))
        self.out = (torch.empty_like(x) if out is None else out) if branch else out
        self.h = torch.empty_like(x) if next_gain is not None else None
        self.y_out = torch.empty_like(x) if want_y else None
        self.t = (x, y, y_perm, slot_row, topk_w, post_gain, gate, next_gain)
        self.dev = dev
        self.args = _typed("moe_block_norm", T, d, k, dtype_code(dt), _p(x), _p(y), _p(y_perm), n_rows, _p(slot_row),
                           _p(topk_w), _p(post_gain), _p(gate), rows, act, res_scale, branch_scale, eps,
                           _p(next_gain), _p(self.out), _p(self.h), _p(self.y_out))

    def __call__(self):
        _launch("moe_block_norm", self.dev, self.args)
        return self


def moe_block_norm(x, y=None, **kw):
    """One call of the norms around a block (arguments as BlockNorm); returns the
    BlockNorm object holding out, h and y_out."""
    return BlockNorm(x, y, **kw)()


class BlockNormBackward:
    """moe_block_norm_backward with its outputs and workspace allocated once.  out is the
    forward's out (its x where there was no branch), y its y or y_out.  dx, dy,
    d_post_gain, dgate and d_next_gain are None where there is nothing to differentiate;
    dgate is float32 [groups, d], or [T, d] in the gate's type for gate_rows 1.
    dx=d_out writes over the incoming gradient."""

    def __init__(self, d_out=None, dh=None, out=None, y=None, post_gain=None, gate=None, gate_rows: int = 0,
                 gate_act: str = "none", next_gain=None, res_scale: float = 1.0, branch_scale: float = 1.0,
                 eps: float = 1e-6, dx=None):
        if next_gain is None:      # out is not read without the norm that follows it
            out = None
        if d_out is None and dh is None:
            raise ValueError("d_out or dh must be given")
        like = dh if d_out is None else d_out
        T, d = like.shape
        dev, dt = like.device, like.dtype
        for name, t in (("d_out", d_out), ("dh", dh), ("out", out), ("y", y), ("dx", dx)):
            _same(name, t, dev, dt, (T, d))
        _same("post_gain", post_gain, dev, torch.float32, (d,))
        _same("next_gain", next_gain, dev, torch.float32, (d,))
        groups, rows, act = _gate_args(gate, gate_rows, gate_act, T, d, dev, dt)
        f32 = dict(dtype=torch.float32, device=dev)
        self.dx = torch.empty_like(like) if dx is None else dx
        self.dy = torch.empty_like(like) if y is not None else None
        self.d_post_gain = torch.empty(d, **f32) if post_gain is not None else None
        self.dgate = None if gate is None else torch.empty_like(gate) if rows == 1 else torch.empty(groups, d, **f32)
        self.d_next_gain = torch.empty(d, **f32) if next_gain is not None else None
        self.t = (d_out, dh, out, y, post_gain, gate, next_gain)
        self.dev = dev
        head = _typed("moe_block_norm_backward", T, d, dtype_code(dt), _p(y), _p(post_gain), _p(gate), rows, act,
                      res_scale, branch_scale, eps, _p(out), _p(next_gain), _p(d_out), _p(dh), _p(self.dx),
                      _p(self.dy), _p(self.d_post_gain), _p(self.dgate), _p(self.d_next_gain))
        self.ws, self.args = _with_ws("moe_block_norm_backward", head, dev)

    def __call__(self):
        _launch("moe_block_norm_backward", self.dev, self.args)
        return self


def moe_block_norm_backward(d_out=None, dh=None, **kw):
    """One call of the block norm's backward (arguments as BlockNormBackward); returns the
    object holding dx, dy, d_post_gain, dgate and d_next_gain."""
    return BlockNormBackward(d_out, dh, **kw)()


class W4Weights:
    """n matrices [R, C] of 4-bit weights with one scale for `group` columns of a row, in
    the library's layout (made by moe_w4_quantize or moe_w4_pack)."""

    def __init__(self, n: int, R: int, C: int, group: int, dev):
        if group not in (32, 64, 128):
            raise MoEError("4-bit weights", 2)
        self.n, self.R, self.C, self.group = n, R, C, group
        row_tiles, col_tiles = n * -(-R // 16), -(-C // 128)
        self._codes = torch.empty(row_tiles * col_tiles * 1024, dtype=torch.uint8, device=dev)
        row_scales = -(-col_tiles * (128 // group) // 4) * 4
        self._scales = torch.empty(row_tiles * 16 * row_scales, dtype=torch.bfloat16, device=dev)
        self.device = self._codes.device
        self._sizes = (_i64(n), _i64(R), _i64(C))
        self._layout = (_i64(group), _p(self._codes), _p(self._scales))

    @property
    def codes(self):
        return self._codes

    @property
    def scales(self):
        return self._scales

    def dequantize(self, dtype=torch.bfloat16, out=None):
        """The values [n, R, C] that the codes and scales stand for, rounded once to dtype."""
        dev = self.device
        if out is None:
            out = torch.empty(self.n, self.R, self.C, dtype=dtype, device=dev)
        _same("out", out, dev, out.dtype, (self.n, self.R, self.C))
        _launch("moe_w4_dequantize", dev, (*self._sizes, dtype_code(out.dtype), *self._layout, out.data_ptr()))
        return out


class W4Quantize:
    """moe_w4_quantize of w [R, C] or [n, R, C] with its W4Weights allocated once."""

    def __init__(self, w, group: int = 128):
        self.w = w if w.dim() == 3 else w.unsqueeze(0)
        n, R, C = self.w.shape
        self.out = W4Weights(n, R, C, group, w.device)
        self.args = _typed("moe_w4_quantize", n, R, C, dtype_code(w.dtype), group, _p(self.w), _p(self.out.codes),
                           _p(self.out.scales))

    def __call__(self) -> W4Weights:
        _launch("moe_w4_quantize", self.w.device, self.args)
        return self.out


def moe_w4_quantize(w, group: int = 128) -> W4Weights:
    """4-bit codes and scales of w [R, C] or [n, R, C]."""
    return W4Quantize(w, group)()


def moe_w4_pack(q, s, group: int = 128) -> W4Weights:
    """W4Weights from codes q [n, R, C/2] (uint8, the even column in the low half) and
    scales s [n, R, ceil(C/group)] (bf16)."""
    n, R, half = q.shape
    dev = q.device
    out = W4Weights(n, R, 2 * half, group, dev)
    _same("q", q, dev, torch.uint8, (n, R, half))
    _same("s", s, dev, torch.bfloat16, (n, R, -(-2 * half // group)))
    _launch("moe_w4_pack", dev, (n, R, 2 * half, group, _p(q), _p(s), _p(out.codes), _p(out.scales)))
    return out


class W4Matvec:
    """moe_w4_matvec: y [T, R] = x [T, C] W^T with its output and workspace allocated once."""

    def __init__(self, x, w: W4Weights, out=None):
        T = x.shape[0]
        if w.n != 1:
            raise ValueError("moe_w4_matvec takes one matrix")
        dev = x.device
        _same("x", x, dev, x.dtype, (T, w.C))
        _same("weights", w.codes, dev, torch.uint8, w.codes.shape)
        _same("out", out, dev, x.dtype, (T, w.R))
        self.y = torch.empty(T, w.R, dtype=x.dtype, device=dev) if out is None else out
        self.t = (x, w)
        self.dev = dev
        head = _typed("moe_w4_matvec", T, w.C, w.R, dtype_code(x.dtype), w.group, _p(x), _p(w.codes), _p(w.scales),
                      _p(self.y))
        self.ws, self.args = _with_ws("moe_w4_matvec", head, dev)

    def __call__(self):
        _launch("moe_w4_matvec", self.dev, self.args)
        return self.y


def moe_w4_matvec(x, w: W4Weights, out=None):
    """y [T, R] = x [T, C] W^T over one 4-bit matrix."""
    return W4Matvec(x, w, out)()


class W4GroupedFfn:
    """moe_w4_grouped_ffn with its output and workspace allocated once: the SwiGLU FFN of
    each expert over its rows, on 4-bit weights gate and up (E matrices [F, d]) and down
    (E matrices [d, F]).  x_in, offsets, a_rows, n_max and y_perm as moe_grouped_ffn."""

    def __init__(self, x_in, offsets, gate: W4Weights, up: W4Weights, down: W4Weights, a_rows=None, n_max=None,
                 y_perm=None):
        E, F, d, group = gate.n, gate.R, gate.C, gate.group
        dev, dt = x_in.device, x_in.dtype
        for name, w, shape in (("up", up, (E, F, d, group)), ("down", down, (E, d, F, group))):
            if (w.n, w.R, w.C, w.group) != shape:
                raise ValueError(f"{name} is {(w.n, w.R, w.C)} in groups of {w.group}, expected {shape}")
        for name, w in (("gate", gate), ("up", up), ("down", down)):
            _same(name, w.codes, dev, torch.uint8, w.codes.shape)
        _same("x_in", x_in, dev, dt, (x_in.shape[0], d))
        _same("offsets", offsets, dev, torch.int32, (E + 1,))
        if a_rows is None:
            if n_max is not None and n_max > x_in.shape[0]:
                raise ValueError("n_max is larger than x_in")
            n_max, n_in = x_in.shape[0] if n_max is None else n_max, 0
        else:
            n_max, n_in = (a_rows.numel() if n_max is None else n_max), x_in.shape[0]
            _same("a_rows", a_rows, dev, torch.int32, a_rows.shape)
            if a_rows.numel() < n_max:
                raise ValueError("a_rows has fewer than n_max entries")
        _same("y_perm", y_perm, dev, dt, (n_max, d))
        self.y_perm = torch.empty(n_max, d, dtype=dt, device=dev) if y_perm is None else y_perm
        self.t = (x_in, offsets, gate, up, down, a_rows)
        self.dev = dev
        head = _typed("moe_w4_grouped_ffn", n_max, d, E, F, dtype_code(dt), group, _p(x_in), n_in, _p(a_rows),
                      _p(offsets), _p(gate.codes), _p(gate.scales), _p(up.codes), _p(up.scales), _p(down.codes),
                      _p(down.scales), _p(self.y_perm))
        self.ws, self.args = _with_ws("moe_w4_grouped_ffn", head, dev)

    def __call__(self):
        _launch("moe_w4_grouped_ffn", self.dev, self.args)
        return self.y_perm


def moe_w4_grouped_ffn(x_in, offsets, gate: W4Weights, up: W4Weights, down: W4Weights, a_rows=None, n_max=None,
                       y_perm=None):
    """y_perm [n_max, d]: the SwiGLU FFN of each 4-bit expert over its rows."""
    return W4GroupedFfn(x_in, offsets, gate, up, down, a_rows, n_max, y_perm)()
