"""Dropout from a counter-based generator (include/lq_dropout.h): the mask is a
function of (seed, step, site, element) and is stored nowhere, so a gradient's
mask is formed again from the same key.

* ``dropout_key``   the generator's key in device memory
* ``Dropout``       a rate and a place of the model on a key
* ``dropout``       of a tensor; its gradient is the same call on the gradient

``adapters_forward``, ``adapters_backward``, ``gated_forward`` and
``gated_backward`` take a ``Dropout`` for the adapters' input.
"""
from __future__ import annotations

import ctypes

from . import _check, _dtype_code, _torch, c_i32, c_i64, c_sz, c_vp, lib, QW_P
from .adapters import SET_P, on_device

LQ_DROPOUT_SITES = 1 << 20


class lq_dropout(ctypes.Structure):
    _fields_ = [("key", c_vp), ("p", ctypes.c_double), ("site", ctypes.c_uint32)]


DROP_P = ctypes.POINTER(lq_dropout)

# name -> (restype, argtypes); the full export list of include/lq_dropout.h
SIGNATURES = {
    "lq_dropout_apply": (ctypes.c_int, [DROP_P, c_vp, c_i64, c_i32, c_vp, c_vp]),
    "lq_adapters_forward_dropout_workspace": (c_sz, [QW_P, c_i64, SET_P]),
    "lq_adapters_forward_dropout": (ctypes.c_int, [QW_P, c_vp, c_i64, SET_P, c_vp, c_vp, DROP_P, c_vp, c_i32, c_vp, c_vp,
                                                   c_sz, c_vp]),
    "lq_adapters_backward_dropout_workspace": (c_sz, [QW_P, c_i64, SET_P]),
    "lq_adapters_backward_dropout": (ctypes.c_int, [QW_P, c_vp, c_vp, c_i64, SET_P, c_vp, c_vp, DROP_P, c_vp, c_vp, c_vp,
                                                    c_vp, c_vp, c_sz, c_vp]),
}


def declare(handle: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the signatures on a loaded library (release or debug build)."""
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


declare(lib)


def dropout_key(seed: int, step: int = 0, device="cuda"):
    """The generator's key, int64 [2] in device memory: seed and step (bit
    patterns of two unsigned 64-bit words). Advance the step (``key[1] += 1``,
    also inside a captured graph) after the backward that belongs to a forward."""
    torch = _torch()
    words = [(int(v) + (1 << 63)) % (1 << 64) - (1 << 63) for v in (seed, step)]
    return torch.tensor(words, dtype=torch.int64).to(device)


class Dropout:
    """Dropout at rate p (in steps of 2^-16) at one place (site) of a model, on a
    key that several places may share. Keeps the key, which the kernels read when
    they run."""

    def __init__(self, p: float, key, site: int = 0):
        torch = _torch()
        if not 0.0 <= p < 1.0:
            raise ValueError("p must be in [0, 1)")
        if not 0 <= site < LQ_DROPOUT_SITES:
            raise ValueError(f"site must be in [0, {LQ_DROPOUT_SITES})")
        if not key.is_cuda or key.dtype != torch.int64 or key.shape != (2,) or not key.is_contiguous():
            raise ValueError("key must be a contiguous int64 [2] device tensor (dropout_key)")
        self.p, self.key, self.site = float(p), key, int(site)
        self.desc = lq_dropout(key.data_ptr(), self.p, self.site)

    @property
    def device(self):
        return self.key.device

    def ref(self):
        return ctypes.byref(self.desc)


def dropout(x, drop: Dropout, out=None):
    """Dropped elements of x (f32 / bf16 / f16, contiguous) are 0, the others
    multiplied by 65536 / (65536 - round(65536 p)). out: x itself (in place), or a
    tensor that does not overlap it; default: a new one."""
    torch = _torch()
    dev = x.device
    if not (x.is_cuda and x.is_contiguous() and x.dtype in (torch.float32, torch.bfloat16, torch.float16)):
        raise ValueError("x must be a contiguous float32, bfloat16 or float16 device tensor")
    if drop.device != dev:
        raise ValueError("the key is on another device")
    if out is None:
        out = torch.empty_like(x)
    elif not (out.is_contiguous() and out.dtype is x.dtype and out.shape == x.shape and out.device == dev):
        raise ValueError("out must be contiguous, of x's shape and type, on its device")
    else:
        a, b, size = x.data_ptr(), out.data_ptr(), x.numel() * x.element_size()
        if a != b and a < b + size and b < a + size:
            raise ValueError("out overlaps x")
    with on_device(torch, dev):
        _check(lib.lq_dropout_apply(drop.ref(), x.data_ptr(), x.numel(), _dtype_code(x), out.data_ptr(),
                                    torch._C._cuda_getCurrentRawStream(dev.index)), "lq_dropout_apply")
    return out
