"""Many adapters over one quantized projection (include/lq_adapters.h):
tensor helpers in the manner of the package's others -- PyTorch gives device
memory and the current stream, the library's HIP kernels do the arithmetic.

* ``AdapterSet``          the adapters of one projection
* ``adapter_route``       tokens sorted by adapter, for every projection of a step
* ``adapters_forward``, ``adapters_backward``
* ``GradList``, ``grad_norm``, ``clip_grad_norm``
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

from . import (LQ_BF16, LQ_F32, QWeight, _check, _contig_cuda, _dtype_code, _ptr, _stream, _torch, c_f32, c_i32, c_i64,
               c_sz, c_vp, lib, QW_P)

LQ_ADAPTERS_MAX = 1000


class lq_adapter(ctypes.Structure):
    _fields_ = [("A", c_vp), ("B", c_vp), ("r", c_i32), ("scale", c_f32), ("row", c_i32), ("row8", c_i32)]


class lq_adapter_set(ctypes.Structure):
    _fields_ = [("host", c_vp), ("dev", c_vp), ("n", c_i32), ("r_max", c_i32)]


class lq_grad_tensor(ctypes.Structure):
    _fields_ = [("data", c_vp), ("numel", c_i64), ("dtype", c_i32), ("group", c_i32)]


class lq_grad_list(ctypes.Structure):
    _fields_ = [("dev", c_vp), ("n_pieces", c_i64), ("n_slots", c_i32), ("n_groups", c_i32),
                ("digest", ctypes.c_uint64)]


SET_P, LIST_P = ctypes.POINTER(lq_adapter_set), ctypes.POINTER(lq_grad_list)

# name -> (restype, argtypes); the full export list of include/lq_adapters.h
SIGNATURES = {
    "lq_check_adapters": (ctypes.c_int, [SET_P, c_i64, c_i64]),
    "lq_adapter_route_bytes": (c_sz, [c_i64, c_i32]),
    "lq_adapter_route": (ctypes.c_int, [c_vp, c_i64, c_i32, c_vp, c_sz, c_vp]),
    "lq_adapters_forward_workspace": (c_sz, [QW_P, c_i64, SET_P]),
    "lq_adapters_forward": (ctypes.c_int, [QW_P, c_vp, c_i64, SET_P, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_sz, c_vp]),
    "lq_adapters_backward_workspace": (c_sz, [QW_P, c_i64, SET_P]),
    "lq_adapters_backward": (ctypes.c_int, [QW_P, c_vp, c_vp, c_i64, SET_P, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                            c_sz, c_vp]),
    "lq_grad_list_bytes": (c_sz, [c_vp, c_i64, c_i32]),
    "lq_grad_list_build": (ctypes.c_int, [c_vp, c_i64, c_i32, c_vp, c_sz, LIST_P]),
    "lq_grad_norm_workspace": (c_sz, [LIST_P]),
    "lq_grad_norm": (ctypes.c_int, [LIST_P, c_vp, c_vp, c_sz, c_vp]),
    "lq_clip_grad_norm": (ctypes.c_int, [LIST_P, LIST_P, c_f32, c_f32, c_vp, c_vp, c_sz, c_vp]),
}


def declare(handle: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the signatures on a loaded library (release or debug build)."""
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


declare(lib)


class AdapterSet:
    """The adapters of many requests or fine-tuning jobs over one [N, K]
    projection: a sequence of (A bf16 [r, K], B bf16 [N, r], alpha). Keeps the
    tensors; their values may change between calls (training), their addresses
    may not. Ranks may differ (1..128)."""

    def __init__(self, adapters: Sequence[Tuple]):
        torch = _torch()
        self.adapters = [(A, B, float(alpha)) for A, B, alpha in adapters]
        if not 1 <= len(self.adapters) <= LQ_ADAPTERS_MAX:
            raise ValueError(f"a set has 1 to {LQ_ADAPTERS_MAX} adapters")
        self.n = len(self.adapters)
        self.K, self.N = self.adapters[0][0].shape[1], self.adapters[0][1].shape[0]
        self.device = self.adapters[0][0].device
        self._host = (lq_adapter * self.n)()
        row = row8 = 0
        for a, (A, B, alpha) in enumerate(self.adapters):
            for name, t in (("A", A), ("B", B)):
                _contig_cuda(t, f"{name} of adapter {a}")
                if t.dtype != torch.bfloat16 or t.device != self.device:
                    raise ValueError(f"{name} of adapter {a} must be bfloat16 on the set's device")
            r = A.shape[0]
            if A.shape != (r, self.K) or B.shape != (self.N, r):
                raise ValueError(f"adapter {a}: A must be [r, {self.K}] and B [{self.N}, r]")
            self._host[a] = lq_adapter(A.data_ptr(), B.data_ptr(), r, alpha / r, row, row8)
            row, row8 = row + r, row8 + (r + 7) // 8 * 8
        self.ranks = [A.shape[0] for A, _, _ in self.adapters]
        self.r_max, self.r_sum = max(self.ranks), row
        self._dev = torch.frombuffer(bytearray(self._host), dtype=torch.uint8).to(self.device)
        self.desc = lq_adapter_set(ctypes.addressof(self._host), self._dev.data_ptr(), self.n, self.r_max)
        _check(lib.lq_check_adapters(self.ref(), self.N, self.K), "lq_check_adapters")

    def ref(self):
        return ctypes.byref(self.desc)

    def split(self, dA, dB):
        """The flat gradients of adapters_backward as a list of (dA [r, K], dB [N, r]) views."""
        out, row = [], 0
        for r in self.ranks:
            out.append((dA[row:row + r], dB[self.N * row:self.N * (row + r)].view(self.N, r)))
            row += r
        return out


def _check_ids(ids, M, device):
    torch = _torch()
    _contig_cuda(ids, "ids")
    if ids.dtype != torch.int32 or tuple(ids.shape) != (M,) or ids.device != device:
        raise ValueError(f"ids must be int32 [{M}] on the tokens' device")


def _check_tokens(x, name, cols, device):
    torch = _torch()
    _contig_cuda(x, name)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != cols or x.device != device:
        raise ValueError(f"{name} must be bfloat16 [tokens, {cols}] on the weight's device")


def _check_set(qw, adapters):
    if (adapters.N, adapters.K) != (qw.N, qw.K) or adapters.device != qw.device:
        raise ValueError(f"the adapters belong to a [{adapters.N}, {adapters.K}] weight on {adapters.device}")


def _check_route(route, ids, n):
    torch = _torch()
    if route is not None:
        _contig_cuda(route, "route")
        if route.dtype != torch.int32 or route.device != ids.device or \
                4 * route.numel() < lib.lq_adapter_route_bytes(ids.numel(), n):
            raise ValueError("route is not one of these ids and this many adapters")


def adapter_route(ids, n: int):
    """Tokens sorted by adapter (int32 buffer) for ids int32 [M] and sets of n
    adapters; pass it to the calls of every projection of the step."""
    torch = _torch()
    _contig_cuda(ids, "ids")
    if ids.dtype != torch.int32 or ids.dim() != 1:
        raise ValueError("ids must be int32 [tokens]")
    M = ids.shape[0]
    size = lib.lq_adapter_route_bytes(M, n)
    route = torch.empty(max(size // 4, 1), dtype=torch.int32, device=ids.device)
    _check(lib.lq_adapter_route(_ptr(ids), M, n, _ptr(route), size, _stream(ids.device)), "lq_adapter_route")
    return route


def adapters_forward(qw: QWeight, X, adapters: AdapterSet, ids, out_dtype=None, save_t: bool = True, route=None):
    """H[m] = W' X[m] + (alpha_a / r_a) B_a A_a X[m] with a = ids[m] (outside
    [0, n): the base weight alone). Returns (H [M, N], t [M, r_max] f32 or None)."""
    torch = _torch()
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be bfloat16 or float32")
    _check_tokens(X, "X", qw.K, qw.device)
    M = X.shape[0]
    _check_set(qw, adapters)
    _check_ids(ids, M, X.device)
    _check_route(route, ids, adapters.n)
    H = torch.empty(M, qw.N, dtype=out_dtype, device=X.device)
    t = torch.empty(M, adapters.r_max, dtype=torch.float32, device=X.device) if save_t else None
    ws_bytes = lib.lq_adapters_forward_workspace(qw.ref(), M, adapters.ref())
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=X.device)
    h_code = LQ_F32 if out_dtype == torch.float32 else LQ_BF16
    _check(lib.lq_adapters_forward(qw.ref(), _ptr(X), M, adapters.ref(), _ptr(ids), _ptr(route), _ptr(H), h_code,
                                   _ptr(t), _ptr(ws), ws_bytes, _stream(X.device)), "lq_adapters_forward")
    return H, t


def adapters_backward(qw: QWeight, X, G, adapters: AdapterSet, ids, t=None, need_grad_x: bool = True,
                      need_dA: bool = True, need_dB: bool = True, route=None):
    """Returns (grad_X bf16 [M, K], dA f32 [sum of ranks, K], dB f32 [N * sum of
    ranks]), each None if not needed; adapters.split(dA, dB) gives them by
    adapter. t: the forward's, or None to form it again from X."""
    torch = _torch()
    _check_tokens(G, "G", qw.N, qw.device)
    M, dev = G.shape[0], G.device
    _check_set(qw, adapters)
    if X is not None:
        _check_tokens(X, "X", qw.K, dev)
        if X.shape[0] != M:
            raise ValueError("X and G differ in their tokens")
    _check_ids(ids, M, dev)
    _check_route(route, ids, adapters.n)
    if t is not None:
        _contig_cuda(t, "t")
        if t.dtype != torch.float32 or tuple(t.shape) != (M, adapters.r_max) or t.device != dev:
            raise ValueError(f"t must be float32 [{M}, {adapters.r_max}] on the tokens' device")
    gx = torch.empty(M, qw.K, dtype=torch.bfloat16, device=dev) if need_grad_x else None
    dA = torch.empty(adapters.r_sum, qw.K, dtype=torch.float32, device=dev) if need_dA else None
    dB = torch.empty(qw.N * adapters.r_sum, dtype=torch.float32, device=dev) if need_dB else None
    ws_bytes = lib.lq_adapters_backward_workspace(qw.ref(), M, adapters.ref())
    ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _check(lib.lq_adapters_backward(qw.ref(), _ptr(X), _ptr(G), M, adapters.ref(), _ptr(ids), _ptr(route), _ptr(t),
                                    _ptr(gx), _ptr(dA), _ptr(dB), _ptr(ws), ws_bytes, _stream(dev)),
           "lq_adapters_backward")
    return gx, dA, dB


class GradList:
    """Gradient tensors (contiguous, f32 / bf16 / f16, any element alignment)
    prepared for grad_norm and clip_grad_norm; groups[i] is the group whose
    norm tensor i counts in (default: one group for all). Keeps the tensors;
    their values may change between calls, their addresses may not."""

    def __init__(self, tensors: Sequence, groups: Optional[Sequence[int]] = None, n_groups: Optional[int] = None,
                 device=None):
        torch = _torch()
        self.tensors = list(tensors)
        groups = [0] * len(self.tensors) if groups is None else [int(g) for g in groups]
        if len(groups) != len(self.tensors):
            raise ValueError("groups must have one entry per tensor")
        self.n_groups = max(groups, default=0) + 1 if n_groups is None else int(n_groups)
        self.device = self.tensors[0].device if self.tensors else torch.device("cuda" if device is None else device)
        arr = (lq_grad_tensor * max(len(self.tensors), 1))()
        for i, (t, g) in enumerate(zip(self.tensors, groups)):
            _contig_cuda(t, f"gradient {i}")
            if t.dtype not in (torch.float32, torch.bfloat16, torch.float16) or t.device != self.device:
                raise ValueError(f"gradient {i} must be float32, bfloat16 or float16 on the list's device")
            arr[i] = lq_grad_tensor(t.data_ptr() if t.numel() else None, t.numel(), _dtype_code(t), g)
        size = lib.lq_grad_list_bytes(arr, len(self.tensors), self.n_groups)
        host = torch.zeros(max(size, 16), dtype=torch.uint8)
        self.desc = lq_grad_list()
        _check(lib.lq_grad_list_build(arr, len(self.tensors), self.n_groups, c_vp(host.data_ptr()), size,
                                      ctypes.byref(self.desc)), "lq_grad_list_build")
        self._dev = host.to(self.device)
        self.desc.dev = self._dev.data_ptr()

    def ref(self):
        return ctypes.byref(self.desc)


def _norm_buffers(grads: GradList):
    torch = _torch()
    norms = torch.empty(grads.n_groups, dtype=torch.float32, device=grads.device)
    ws_bytes = lib.lq_grad_norm_workspace(grads.ref())
    return norms, torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=grads.device), ws_bytes


def grad_norm(grads: GradList):
    """The L2 norm of each group's gradients (f32 [n_groups])."""
    norms, ws, ws_bytes = _norm_buffers(grads)
    _check(lib.lq_grad_norm(grads.ref(), _ptr(norms), _ptr(ws), ws_bytes, _stream(grads.device)), "lq_grad_norm")
    return norms


def clip_grad_norm(grads: GradList, max_norm: float, out: Optional[GradList] = None, eps: float = 1e-6):
    """Scales each group's gradients by min(1, max_norm / (norm + eps)), in place
    or into `out` (a list of the same sizes, types and groups). Returns the
    norms before clipping (f32 [n_groups]); a group whose norm is not finite
    shows there."""
    out = grads if out is None else out
    if out.device != grads.device:
        raise ValueError("the lists are on different devices")
    norms, ws, ws_bytes = _norm_buffers(grads)
    _check(lib.lq_clip_grad_norm(grads.ref(), out.ref(), float(max_norm), float(eps), _ptr(norms), _ptr(ws), ws_bytes,
                                 _stream(grads.device)), "lq_clip_grad_norm")
    return norms
