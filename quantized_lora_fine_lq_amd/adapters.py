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

from . import (LQ_BF16, LQ_F32, QWeight, _check, _contig_cuda, _dtype_code, _ptr, _torch, c_f32, c_i32, c_i64,
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
        for a, (A, B, _) in enumerate(self.adapters):
            if A.dim() != 2 or B.dim() != 2 or A.shape[0] < 1:
                raise ValueError(f"adapter {a}: A and B must be matrices of a rank of at least 1")
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


# The smallest calls run for ten microseconds, so these helpers cost as little
# as they can: one condition each, the words only on failure; and the stream's
# handle by device index instead of a Stream object (2 us); and outputs by
# empty_strided, a third of a microsecond less than empty.
def _stream(dev):
    return _torch()._C._cuda_getCurrentRawStream(dev.index)


def _tokens(torch, x, name, cols, device):
    if not (x.is_cuda and x.dtype is torch.bfloat16 and x.dim() == 2 and x.size(1) == cols and x.is_contiguous()
            and x.device == device):
        raise ValueError(f"{name} must be contiguous bfloat16 [tokens, {cols}] on the weight's device")


def _tokens_args(torch, M, qw, adapters, ids, route, device):
    if adapters.N != qw.N or adapters.K != qw.K or adapters.device != device:
        raise ValueError(f"the adapters belong to a [{adapters.N}, {adapters.K}] weight on {adapters.device}")
    if not (ids.is_cuda and ids.dtype is torch.int32 and ids.dim() == 1 and ids.size(0) == M and ids.is_contiguous()
            and ids.device == device):
        raise ValueError(f"ids must be contiguous int32 [{M}] on the tokens' device")
    # a route of other sizes has its arrays elsewhere, and positions past this call's tokens
    if route is not None and not (
            getattr(route, "lq_route_of", None) == (M, adapters.n) and route.device == device
            and route.dtype is torch.int32 and route.is_contiguous()
            and 4 * route.numel() >= lib.lq_adapter_route_bytes(M, adapters.n)):
        raise ValueError(f"route must be adapter_route's, of {M} ids and {adapters.n} adapters")


def adapter_route(ids, n: int):
    """Tokens sorted by adapter (int32 buffer) for ids int32 [M] and sets of n
    adapters; pass it to the calls of every projection of the step. The buffer
    carries (M, n) as lq_route_of: the calls take it for these sizes alone, and
    no copy of it."""
    torch = _torch()
    _contig_cuda(ids, "ids")
    if ids.dtype != torch.int32 or ids.dim() != 1:
        raise ValueError("ids must be int32 [tokens]")
    M = ids.shape[0]
    size = lib.lq_adapter_route_bytes(M, n)
    route = torch.empty(max(size // 4, 1), dtype=torch.int32, device=ids.device)
    _check(lib.lq_adapter_route(_ptr(ids), M, n, _ptr(route), size, _stream(ids.device)), "lq_adapter_route")
    route.lq_route_of = (M, n)
    return route


def adapters_forward(qw: QWeight, X, adapters: AdapterSet, ids, out_dtype=None, save_t: bool = True, route=None):
    """H[m] = W' X[m] + (alpha_a / r_a) B_a A_a X[m] with a = ids[m] (outside
    [0, n): the base weight alone). Returns (H [M, N], t [M, r_max] f32 or None)."""
    torch = _torch()
    if out_dtype is None:
        out_dtype = torch.bfloat16
    f32 = out_dtype is torch.float32
    if not f32 and out_dtype is not torch.bfloat16:
        raise ValueError("out_dtype must be bfloat16 or float32")
    dev = qw.device
    _tokens(torch, X, "X", qw.K, dev)
    M = X.size(0)
    _tokens_args(torch, M, qw, adapters, ids, route, dev)
    N, r, w, s, empty = qw.N, adapters.r_max, qw.ref(), adapters.ref(), torch.empty_strided
    H = empty((M, N), (N, 1), dtype=out_dtype, device=dev)
    t = empty((M, r), (r, 1), dtype=torch.float32, device=dev) if save_t else None
    ws_bytes = lib.lq_adapters_forward_workspace(w, M, s)
    ws = empty((max(ws_bytes, 1),), (1,), dtype=torch.uint8, device=dev)
    _check(lib.lq_adapters_forward(w, X.data_ptr(), M, s, ids.data_ptr(), None if route is None else route.data_ptr(),
                                   H.data_ptr(), LQ_F32 if f32 else LQ_BF16, t.data_ptr() if save_t else None,
                                   ws.data_ptr(), ws_bytes, _stream(dev)), "lq_adapters_forward")
    return H, t


def adapters_backward(qw: QWeight, X, G, adapters: AdapterSet, ids, t=None, need_grad_x: bool = True,
                      need_dA: bool = True, need_dB: bool = True, route=None):
    """Returns (grad_X bf16 [M, K], dA f32 [sum of ranks, K], dB f32 [N * sum of
    ranks]), each None if not needed; adapters.split(dA, dB) gives them by
    adapter. t: the forward's, or None to form it again from X."""
    torch = _torch()
    dev = qw.device
    _tokens(torch, G, "G", qw.N, dev)
    M = G.size(0)
    if X is not None:
        _tokens(torch, X, "X", qw.K, dev)
        if X.size(0) != M:
            raise ValueError("X and G differ in their tokens")
    _tokens_args(torch, M, qw, adapters, ids, route, dev)
    if t is not None and not (t.is_cuda and t.dtype is torch.float32 and t.shape == (M, adapters.r_max)
                              and t.is_contiguous() and t.device == dev):
        raise ValueError(f"t must be contiguous float32 [{M}, {adapters.r_max}] on the tokens' device")
    K, w, s, empty, f32 = qw.K, qw.ref(), adapters.ref(), torch.empty_strided, torch.float32
    gx = empty((M, K), (K, 1), dtype=torch.bfloat16, device=dev) if need_grad_x else None
    dA = empty((adapters.r_sum, K), (K, 1), dtype=f32, device=dev) if need_dA else None
    dB = empty((qw.N * adapters.r_sum,), (1,), dtype=f32, device=dev) if need_dB else None
    ws_bytes = lib.lq_adapters_backward_workspace(w, M, s)
    ws = empty((max(ws_bytes, 1),), (1,), dtype=torch.uint8, device=dev)
    _check(lib.lq_adapters_backward(w, _at(X), G.data_ptr(), M, s, ids.data_ptr(), _at(route), _at(t), _at(gx), _at(dA),
                                    _at(dB), ws.data_ptr(), ws_bytes, _stream(dev)), "lq_adapters_backward")
    return gx, dA, dB


def _at(t):
    return None if t is None else t.data_ptr()


class GradList:
    """Gradient tensors (contiguous, f32 / bf16 / f16, any element alignment)
    prepared for grad_norm and clip_grad_norm; groups[i] is the group whose
    norm tensor i counts in (default: one group for all). Keeps the tensors;
    their values may change between calls, their addresses may not. Building a
    list walks its tensors on the host and copies a table to the device, for
    which the host waits (44 us for 14 tensors, 2.3 ms for 1792): keep it where
    the gradients stay in place. adapters_backward returns new tensors every
    time; lq_adapters_backward itself writes where its caller says."""

    def __init__(self, tensors: Sequence, groups: Optional[Sequence[int]] = None, n_groups: Optional[int] = None,
                 device=None):
        torch = _torch()
        self.tensors = list(tensors)
        groups = [0] * len(self.tensors) if groups is None else [int(g) for g in groups]
        if len(groups) != len(self.tensors):
            raise ValueError("groups must have one entry per tensor")
        self.n_groups = max(groups, default=0) + 1 if n_groups is None else int(n_groups)
        if self.tensors:
            self.device = self.tensors[0].device
        else:   # as tensors name it, with its index
            self.device = torch.empty(0, device="cuda" if device is None else device).device
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
        self._ws_bytes = lib.lq_grad_norm_workspace(self.ref())

    def ref(self):
        return ctypes.byref(self.desc)

    def _buffers(self):
        torch = _torch()
        empty, dev = torch.empty_strided, self.device
        return (empty((self.n_groups,), (1,), dtype=torch.float32, device=dev),
                empty((max(self._ws_bytes, 1),), (1,), dtype=torch.uint8, device=dev))


def grad_norm(grads: GradList):
    """The L2 norm of each group's gradients (f32 [n_groups])."""
    norms, ws = grads._buffers()
    _check(lib.lq_grad_norm(grads.ref(), norms.data_ptr(), ws.data_ptr(), grads._ws_bytes, _stream(grads.device)),
           "lq_grad_norm")
    return norms


def clip_grad_norm(grads: GradList, max_norm: float, out: Optional[GradList] = None, eps: float = 1e-6):
    """Scales each group's gradients by min(1, max_norm / (norm + eps)), in place
    or into `out` (a list of the same sizes, types and groups). Returns the
    norms before clipping (f32 [n_groups]); a group whose norm is not finite
    shows there."""
    if out is None:
        out = grads
    elif out.device != grads.device:
        raise ValueError("the lists are on different devices")
    norms, ws = grads._buffers()
    _check(lib.lq_clip_grad_norm(grads.ref(), out.ref(), float(max_norm), float(eps), norms.data_ptr(), ws.data_ptr(),
                                 grads._ws_bytes, _stream(grads.device)), "lq_clip_grad_norm")
    return norms
