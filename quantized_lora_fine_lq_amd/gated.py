"""A gated pair of quantized projections with adapters (include/lq_gated.h):
h = act(g) * u, g and u two projections of the same X, in the manner of
``adapters.py``.

* ``GatedPair``                          the weights, their adapters, the activation
* ``gated_forward``, ``gated_backward``
* ``GatedSaved``, ``GatedGrads``         what the forward keeps, what the backward gives
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import LQ_BF16, LQ_F32, QWeight, QW_P, _check, _torch, c_i32, c_i64, c_sz, c_vp, lib
from .adapters import SET_P, AdapterSet, _at, _drop_args, _stream, _tokens, _tokens_args, on_device
from .dropouts import DROP_P

LQ_SILU, LQ_GELU, LQ_GELU_TANH = 0, 1, 2
ACTS = {"silu": LQ_SILU, "gelu": LQ_GELU, "gelu_tanh": LQ_GELU_TANH}


class lq_gated(ctypes.Structure):
    _fields_ = [("gate", QW_P), ("up", QW_P), ("gate_set", SET_P), ("up_set", SET_P), ("act", c_i32)]


PAIR_P = ctypes.POINTER(lq_gated)

# name -> (restype, argtypes); the full export list of include/lq_gated.h
SIGNATURES = {
    "lq_check_gated": (ctypes.c_int, [PAIR_P]),
    "lq_gated_forward_workspace": (c_sz, [PAIR_P, c_i64, c_i32]),
    "lq_gated_forward": (ctypes.c_int, [PAIR_P, c_vp, c_i64, c_vp, c_vp, DROP_P, DROP_P, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                                        c_vp, c_sz, c_vp]),
    "lq_gated_backward_workspace": (c_sz, [PAIR_P, c_i64]),
    "lq_gated_backward": (ctypes.c_int, [PAIR_P, c_vp, c_vp, c_i64, c_vp, c_vp, DROP_P, DROP_P, c_vp, c_vp, c_vp, c_vp, c_vp,
                                         c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]),
}


def declare(handle: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the signatures on a loaded library (release or debug build)."""
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


declare(lib)


class GatedSaved(NamedTuple):
    """What a forward keeps for its backward: g, u bf16 [M, N]; t_gate, t_up f32
    [M, r_max] of each set (None without sets, or to be formed again)."""
    g: object
    u: object
    t_gate: object = None
    t_up: object = None


class GatedGrads(NamedTuple):
    """grad_X bf16 [M, K]; the adapters' gradients flat, as adapters_backward's
    (AdapterSet.split gives them by adapter)."""
    grad_X: object
    dA_gate: object
    dB_gate: object
    dA_up: object
    dB_up: object


class GatedPair:
    """Two [N, K] quantized weights and, for each or for neither, its adapters
    (sets with as many adapters: a token's id names its adapter in both)."""

    def __init__(self, gate: QWeight, up: QWeight, gate_adapters: Optional[AdapterSet] = None,
                 up_adapters: Optional[AdapterSet] = None, act: str = "silu"):
        if act not in ACTS:
            raise ValueError(f"act must be one of {', '.join(ACTS)}")
        if (gate.N, gate.K) != (up.N, up.K) or gate.device != up.device:
            raise ValueError("gate and up must be of one size, on one device")
        if (gate_adapters is None) != (up_adapters is None):
            raise ValueError("adapters belong to both projections or to neither")
        self.gate, self.up, self.act = gate, up, act
        self.gate_adapters, self.up_adapters = gate_adapters, up_adapters
        self.N, self.K, self.device = gate.N, gate.K, gate.device
        self.n = 0
        if gate_adapters is not None:
            self.n = gate_adapters.n
            if up_adapters.n != self.n:
                raise ValueError("the sets must have as many adapters")
            for s in (gate_adapters, up_adapters):
                if (s.N, s.K) != (self.N, self.K) or s.device != self.device:
                    raise ValueError(f"the adapters belong to a [{s.N}, {s.K}] weight on {s.device}")
        ref = ctypes.pointer
        self.desc = lq_gated(ref(gate.desc), ref(up.desc), None if gate_adapters is None else ref(gate_adapters.desc),
                             None if up_adapters is None else ref(up_adapters.desc), ACTS[act])
        _check(lib.lq_check_gated(self.ref()), "lq_check_gated")

    def ref(self):
        return ctypes.byref(self.desc)


def _pair_args(torch, pair, M, ids, route, dropout):
    """ids and route checked; the two dropouts."""
    if pair.n:
        if ids is None:
            raise ValueError("a pair with adapters takes each token's id")
        _tokens_args(torch, M, pair.gate, pair.gate_adapters, ids, route, pair.device)
    elif ids is not None or route is not None or dropout is not None:
        raise ValueError("a pair without adapters takes no ids, route or dropout")
    if dropout is None:
        return None, None
    gate, up = dropout
    for d in (gate, up):
        if d is not None:
            _drop_args(d, pair.device)
    return gate, up


def _ref(d):
    return None if d is None else d.ref()


def gated_forward(pair: GatedPair, X, ids=None, out_dtype=None, save: bool = True, route=None, dropout=None):
    """h = act(g) u with g[m] = W'_gate X[m] + s_a B_a A_a X[m] and u[m] likewise,
    a = ids[m] (outside [0, n): the base weights alone). Returns (H [M, N],
    GatedSaved or None). dropout: (gate's Dropout, up's), either None, of the
    adapters' input; two sites, or they drop alike."""
    torch = _torch()
    if out_dtype is None:
        out_dtype = torch.bfloat16
    f32 = out_dtype is torch.float32
    if not f32 and out_dtype is not torch.bfloat16:
        raise ValueError("out_dtype must be bfloat16 or float32")
    dev = pair.device
    _tokens(torch, X, "X", pair.K, dev)
    M = X.size(0)
    d0, d1 = _pair_args(torch, pair, M, ids, route, dropout)
    N, p, empty = pair.N, pair.ref(), torch.empty_strided
    H = empty((M, N), (N, 1), dtype=out_dtype, device=dev)
    saved = None
    if save:
        g = empty((M, N), (N, 1), dtype=torch.bfloat16, device=dev)
        u = empty((M, N), (N, 1), dtype=torch.bfloat16, device=dev)
        saved = GatedSaved(g, u)
        if pair.n:
            r0, r1 = pair.gate_adapters.r_max, pair.up_adapters.r_max
            saved = GatedSaved(g, u, empty((M, r0), (r0, 1), dtype=torch.float32, device=dev),
                               empty((M, r1), (r1, 1), dtype=torch.float32, device=dev))
    ws_bytes = lib.lq_gated_forward_workspace(p, M, d0 is not None or d1 is not None)
    ws = empty((max(ws_bytes, 1),), (1,), dtype=torch.uint8, device=dev)
    g, u, t0, t1 = (_at(t) for t in saved) if save else (None,) * 4
    with on_device(torch, dev):
        _check(lib.lq_gated_forward(p, X.data_ptr(), M, _at(ids), _at(route), _ref(d0), _ref(d1), H.data_ptr(),
                                    LQ_F32 if f32 else LQ_BF16, g, u, t0, t1, ws.data_ptr(), ws_bytes, _stream(dev)),
               "lq_gated_forward")
    return H, saved


def _kept(torch, t, name, shape, dtype, device):
    if not (t.is_cuda and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device):
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on the weights' device")


def gated_backward(pair: GatedPair, X, G, ids, saved: GatedSaved, need_grad_x: bool = True, need_dA: bool = True,
                   need_dB: bool = True, route=None, dropout=None):
    """Gradients for G = dL/dH (bf16 [M, N]; N % 8 == 0) as GatedGrads, each None
    if not needed (without adapters: grad_X alone). saved: the forward's; its t
    may be None, to be formed again from X. dropout: the forward's, on the key as
    it stood there. dg and du are float32 in the adapters' gradients and bfloat16 in
    grad_X's product with the weights."""
    torch = _torch()
    dev = pair.device
    N, K = pair.N, pair.K
    _tokens(torch, G, "G", N, dev)
    M = G.size(0)
    if X is not None:
        _tokens(torch, X, "X", K, dev)
        if X.size(0) != M:
            raise ValueError("X and G differ in their tokens")
    d0, d1 = _pair_args(torch, pair, M, ids, route, dropout)
    f32, empty = torch.float32, torch.empty_strided
    _kept(torch, saved.g, "g", (M, N), torch.bfloat16, dev)
    _kept(torch, saved.u, "u", (M, N), torch.bfloat16, dev)
    sets = (pair.gate_adapters, pair.up_adapters) if pair.n else ()
    for t, s, name in zip((saved.t_gate, saved.t_up), sets, ("t_gate", "t_up")):
        if t is not None:
            _kept(torch, t, name, (M, s.r_max), f32, dev)
    gx = empty((M, K), (K, 1), dtype=torch.bfloat16, device=dev) if need_grad_x else None
    grads = [None] * 4
    for i, s in enumerate(sets):
        if need_dA:
            grads[2 * i] = empty((s.r_sum, K), (K, 1), dtype=f32, device=dev)
        if need_dB:
            grads[2 * i + 1] = empty((N * s.r_sum,), (1,), dtype=f32, device=dev)
    p = pair.ref()
    ws_bytes = lib.lq_gated_backward_workspace(p, M)
    ws = empty((max(ws_bytes, 1),), (1,), dtype=torch.uint8, device=dev)
    with on_device(torch, dev):
        _check(lib.lq_gated_backward(p, _at(X), G.data_ptr(), M, _at(ids), _at(route), _ref(d0), _ref(d1),
                                     saved.g.data_ptr(), saved.u.data_ptr(), _at(saved.t_gate) if sets else None,
                                     _at(saved.t_up) if sets else None, _at(gx), *(_at(t) for t in grads), ws.data_ptr(),
                                     ws_bytes, _stream(dev)), "lq_gated_backward")
    return GatedGrads(gx, *grads)
