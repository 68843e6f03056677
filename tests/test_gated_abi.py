"""CPU tests of the gated pair: exports, refusals before any launch, size
queries, and the oracle's activations against differences."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import gated as og
from test_adapters_abi import A, make_set, nf4, vp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lq_gated.h")


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def ad(lq):
    from quantized_lora_fine_lq_amd import adapters
    return adapters


@pytest.fixture(scope="module")
def ga(lq):
    from quantized_lora_fine_lq_amd import gated
    return gated


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_oracle_slopes(kind):
    g = np.linspace(-8, 8, 401)
    h = 1e-6
    value, slope = og.act(g, kind)
    # central differences: h^2 / 6 of the third derivative (below 2), and rounding over 2 h
    assert np.allclose(slope, (og.act(g + h, kind)[0] - og.act(g - h, kind)[0]) / (2 * h), atol=h * h + 8 * 2e-16 / h)
    assert og.act(0.0, kind)[0] == 0 and og.act(0.0, kind)[1] == 0.5
    # known values at 1: 1 / (1 + 1/e); the normal distribution function at 1; its tanh form
    want = {"silu": 0.7310585786300049, "gelu": 0.8413447460685429, "gelu_tanh": 0.8411919906082768}[kind]
    assert abs(og.act(1.0, kind)[0] - want) < 1e-15


def test_every_declared_symbol_is_exported(lq, ga):
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(lq_\w+)\s*\(", text, re.M)))
    assert names == sorted(ga.SIGNATURES)
    dbg = ga.declare(lq.load_debug_library())
    for name in names:
        assert hasattr(lq.lib, name) and hasattr(dbg, name)
    for name, value in re.findall(r"(LQ_(?:SILU|GELU|GELU_TANH)) = (\d)", text):
        assert getattr(ga, name) == int(value)


def pair(lq, ad, ga, gate=None, up=None, sets=True, ranks=([8, 16, 5], [4, 8, 64]), act=0, **kw):
    ptr = ctypes.pointer
    gate, up = gate or nf4(lq), up or nf4(lq)
    s0, s1 = (make_set(ad, r) for r in ranks)
    p = ga.lq_gated(ptr(gate), ptr(up), ptr(s0) if sets else None, ptr(s1) if sets else None, act)
    p.keep = (gate, up, s0, s1)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def test_check(lq, ad, ga):
    check = lambda **kw: lq.lib.lq_check_gated(ctypes.byref(pair(lq, ad, ga, **kw)))
    assert check() == lq.LQ_OK and check(sets=False) == lq.LQ_OK and check(act=2) == lq.LQ_OK
    assert lq.lib.lq_check_gated(None) == lq.LQ_ERR_ARG
    for kw in (dict(act=-1), dict(act=3), dict(gate_set=None), dict(up_set=None)):
        assert check(**kw) == lq.LQ_ERR_ARG, kw
    assert lq.lib.lq_check_gated(ctypes.byref(pair(lq, ad, ga, gate_set=None, up_set=None))) == lq.LQ_OK
    p = pair(lq, ad, ga)
    p.up = None
    assert lq.lib.lq_check_gated(ctypes.byref(p)) == lq.LQ_ERR_ARG
    assert check(up=nf4(lq, N=192)) == lq.LQ_ERR_SHAPE and check(up=nf4(lq, K=128)) == lq.LQ_ERR_SHAPE
    assert check(ranks=([8, 16], [8])) == lq.LQ_ERR_SHAPE and check(ranks=([8, 16], [8, 129])) == lq.LQ_ERR_SHAPE
    assert check(gate=nf4(lq, blocksize=32)) == lq.LQ_ERR_UNSUPPORTED
    assert check(up=nf4(lq, codes=A + 8)) == lq.LQ_ERR_ARG


def drop(lq, key=A, p=0.1, site=3):
    from quantized_lora_fine_lq_amd import dropouts
    return ctypes.byref(dropouts.lq_dropout(key, p, site))


def test_forward_refusals(lq, ad, ga):
    L = lq.lib
    p, bare = pair(lq, ad, ga), pair(lq, ad, ga, sets=False)
    P, B = ctypes.byref(p), ctypes.byref(bare)
    size = L.lq_gated_forward_workspace(P, 300, 1)
    assert size > 4 * 128 * 256 and L.lq_gated_forward_workspace(P, 300, 0) == size
    assert 0 < L.lq_gated_forward_workspace(B, 300, 0) < size
    for M in (0, -1, 1 << 31):
        assert L.lq_gated_forward_workspace(P, M, 0) == 0
    assert L.lq_gated_forward_workspace(None, 300, 0) == 0

    def fwd(p=P, X=A, M=300, ids=A, route=None, d0=None, d1=None, H=A, dt=lq.LQ_BF16, g=None, u=None, t0=None, t1=None,
            ws=A, size=size):
        return L.lq_gated_forward(p, vp(X), M, vp(ids), vp(route), d0, d1, vp(H), dt, vp(g), vp(u), vp(t0), vp(t1), vp(ws),
                                  size, vp(None))
    for kw in (dict(p=None), dict(X=None), dict(H=None), dict(ids=None), dict(X=A + 8), dict(ids=A + 2), dict(H=A + 8),
               dict(g=A + 8), dict(u=A + 2), dict(t0=A + 2), dict(t1=A + 1), dict(route=A + 4), dict(ws=A + 8),
               dict(d0=drop(lq, p=1.0)), dict(d1=drop(lq, key=None)), dict(d1=drop(lq, site=1 << 20)),
               dict(p=B), dict(p=B, ids=None, t0=A), dict(p=B, ids=None, t1=A), dict(p=B, ids=None, route=A),
               dict(p=B, ids=None, d0=drop(lq))):
        assert fwd(**kw) == lq.LQ_ERR_ARG, kw
    assert fwd(M=0) == lq.LQ_ERR_SHAPE and fwd(M=1 << 31) == lq.LQ_ERR_SHAPE
    assert fwd(dt=lq.LQ_F16) == lq.LQ_ERR_UNSUPPORTED
    assert fwd(size=size - 1) == lq.LQ_ERR_WORKSPACE and fwd(ws=None) == lq.LQ_ERR_WORKSPACE
    assert fwd(H=A + 4, dt=lq.LQ_F32, ws=None) == lq.LQ_ERR_WORKSPACE      # 4 bytes are enough for a float32 H
    wide = pair(lq, ad, ga, gate=nf4(lq, K=1 << 18), up=nf4(lq, K=1 << 18))
    assert fwd(p=ctypes.byref(wide), M=1 << 29, d0=drop(lq)) == lq.LQ_ERR_SHAPE
    assert L.lq_gated_forward_workspace(ctypes.byref(wide), 1 << 29, 1) == 0


def test_backward_refusals(lq, ad, ga):
    L = lq.lib
    p, bare = pair(lq, ad, ga), pair(lq, ad, ga, sets=False)
    P, B = ctypes.byref(p), ctypes.byref(bare)
    size = L.lq_gated_backward_workspace(P, 300)
    assert size > 4 * 128 * 256 + 4 * 300 * 128 and 0 < L.lq_gated_backward_workspace(B, 300) < size
    odd = pair(lq, ad, ga, gate=nf4(lq, N=100), up=nf4(lq, N=100))
    assert L.lq_gated_backward_workspace(ctypes.byref(odd), 300) == 0 and L.lq_gated_backward_workspace(P, 0) == 0

    def bwd(p=P, X=A, G=A, M=300, ids=A, route=None, d0=None, d1=None, g=A, u=A, t0=None, t1=None, gx=A, dA0=A, dB0=A,
            dA1=A, dB1=A, ws=A, size=size):
        return L.lq_gated_backward(p, vp(X), vp(G), M, vp(ids), vp(route), d0, d1, vp(g), vp(u), vp(t0), vp(t1), vp(gx),
                                   vp(dA0), vp(dB0), vp(dA1), vp(dB1), vp(ws), size, vp(None))
    none = dict(dA0=None, dB0=None, dA1=None, dB1=None)
    for kw in (dict(p=None), dict(G=None), dict(g=None), dict(u=None), dict(ids=None), dict(X=None), dict(X=None, t0=A, t1=A),
               dict(X=None, dA0=None, dA1=None, t0=A), dict(G=A + 8), dict(g=A + 8), dict(u=A + 8), dict(X=A + 8),
               dict(gx=A + 8), dict(dA0=A + 2), dict(dB0=A + 2), dict(dA1=A + 2), dict(dB1=A + 1), dict(t0=A + 2), dict(t1=A + 2),
               dict(ws=A + 8), dict(route=A + 8), dict(ids=A + 1), dict(d0=drop(lq, p=-1.0)),
               dict(p=B, ids=None), dict(p=B, **none), dict(p=B, ids=None, t0=A, **none), dict(p=B, ids=None, d1=drop(lq), **none)):
        assert bwd(**kw) == lq.LQ_ERR_ARG, kw
    assert bwd(p=ctypes.byref(odd)) == lq.LQ_ERR_SHAPE and bwd(M=0) == lq.LQ_ERR_SHAPE
    assert bwd(size=size - 1) == lq.LQ_ERR_WORKSPACE and bwd(ws=None) == lq.LQ_ERR_WORKSPACE
    assert bwd(gx=None, X=None, **none) == lq.LQ_OK      # nothing wanted: nothing launched


def test_where_a_forward_keeps_the_packed_weights(lq, ad, ga):
    """The sizes that the header promises a small workspace for, and those just past them."""
    size = lambda M, drops=0, **kw: lq.lib.lq_gated_forward_workspace(ctypes.byref(pair(lq, ad, ga, **kw)), M, drops)
    N = 4096

    def both(K, r, **kw):
        return dict(gate=nf4(lq, N, K), up=nf4(lq, N, K, **kw), ranks=([r, 3], [8, r]))
    for T, M in ((16, 16), (32, 17), (64, 33), (64, 64)):
        for r in (8, 33, 64, 128):
            r8 = (r + 7) // 8 * 8
            last = min((130560 - 6 * T * 2 * r8) // 2 // 64 * 64, 49152)
            small = 2 * (8 * M * 2 * r8 * 4) + 2 * T * (last + 64) + (1 << 17)      # up to eight parts of t, X, the steps' list
            assert size(M, **both(last, r)) <= small < 4 * N * last
            past = min(last + 1024, 49152 + 64)      # (what fits is a little more than what is promised)
            assert size(M, **both(past, r)) >= 4 * N * past
        assert size(M, sets=False, **both(49152, 8)) < 4 * N * 49152 / 64
        dq = dict(absmax=None, absmax_q=A, dq_scale=A, dq_mean=A)
        assert size(M, **both(256, 16, **dq)) >= 4 * N * 256 and size(M, drops=1, **both(256, 16)) >= 4 * N * 256
    assert size(65, **both(256, 16)) >= 4 * N * 256
