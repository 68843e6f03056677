"""CPU tests of dropout: exports, refusals before any launch, size queries, and
the oracle's generator against published answers and its own definition."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import dropout as odr
from test_adapters_abi import A, make_set, nf4, vp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lq_dropout.h")


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def ad(lq):
    from quantized_lora_fine_lq_amd import adapters
    return adapters


@pytest.fixture(scope="module")
def dr(lq):
    from quantized_lora_fine_lq_amd import dropouts
    return dropouts


# Answers that the generator's authors publish with it.
@pytest.mark.parametrize("counter, key, words", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_known_answers(counter, key, words):
    assert tuple(int(w) for w in odr.philox(counter, key)) == words


def test_fields_and_rate():
    f = odr.fields(5, 7, 3, 0, 1 << 16)
    assert np.array_equal(odr.fields(5, 7, 3, 1001, 300), f[1001:1301])
    w = odr.philox((3, 3 * 4096, 7, 0), (5, 0))
    assert [int(v) for v in f[24:32]] == [int(w[j // 2]) >> 16 * (j % 2) & 0xFFFF for j in range(8)]
    far = odr.fields(5, 7, 3, 8 << 33, 8)      # a block past 2^32
    w = odr.philox((0, 3 * 4096 + 2, 7, 0), (5, 0))
    assert [int(v) for v in far] == [int(w[j // 2]) >> 16 * (j % 2) & 0xFFFF for j in range(8)]
    mask, factor = odr.kept(5, 7, 3, 0.3, (256, 256))
    # a binomial share: five standard deviations
    assert abs(mask.mean() - 0.7) < 5 * (0.21 / 65536) ** 0.5 and factor == 65536 / (65536 - 19661)
    assert odr.threshold(0.0) == 0 and odr.threshold(1.0 - 1e-9) == 65535


def test_every_declared_symbol_is_exported(lq, dr):
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(lq_\w+)\s*\(", text, re.M)))
    assert names == sorted(dr.SIGNATURES)
    dbg = dr.declare(lq.load_debug_library())
    for name in names:
        assert hasattr(lq.lib, name) and hasattr(dbg, name)
    assert "#define LQ_DROPOUT_SITES (1 << 20)" in text and dr.LQ_DROPOUT_SITES == 1 << 20


BAD = [dict(key=None), dict(key=A + 4), dict(p=-0.1), dict(p=1.0), dict(p=float("nan")), dict(site=1 << 20)]


def drop(dr, key=A, p=0.1, site=3):
    return ctypes.byref(dr.lq_dropout(key, p, site))


def test_apply_refusals(lq, dr):
    call = lambda d=drop(dr), x=A, n=100, dt=lq.LQ_F32, out=A: lq.lib.lq_dropout_apply(d, vp(x), n, dt, vp(out), vp(None))
    for kw in BAD:
        assert call(d=drop(dr, **kw)) == lq.LQ_ERR_ARG, kw
    for kw in (dict(d=None), dict(x=None), dict(out=None), dict(x=A + 2), dict(out=A + 1), dict(x=A + 1, dt=lq.LQ_BF16),
               dict(dt=3), dict(dt=-1)):
        assert call(**kw) == lq.LQ_ERR_ARG, kw
    assert call(n=-1) == lq.LQ_ERR_SHAPE and call(n=1 << 47) == lq.LQ_ERR_SHAPE
    assert call(n=0) == lq.LQ_OK and call(n=0, x=None, out=None) == lq.LQ_OK


def test_adapter_refusals(lq, ad, dr):
    L = lq.lib
    w, s = nf4(lq), make_set(ad, [8, 16, 5])
    W, S = ctypes.byref(w), ctypes.byref(s)
    ws, wb = L.lq_adapters_forward_dropout_workspace(W, 300, S), L.lq_adapters_backward_dropout_workspace(W, 300, S)
    assert ws == L.lq_adapters_forward_workspace(W, 300, S) and wb == L.lq_adapters_backward_workspace(W, 300, S)
    # few tokens run as many do
    assert L.lq_adapters_forward_dropout_workspace(W, 16, S) > 2 * 128 * 256
    assert L.lq_adapters_forward_dropout_workspace(W, 0, S) == 0 and L.lq_adapters_forward_dropout_workspace(W, 5, None) == 0

    def fwd(w=W, X=A, M=300, d=drop(dr), H=A, wsp=A, size=ws):
        return L.lq_adapters_forward_dropout(w, vp(X), M, S, vp(A), vp(None), d, vp(H), lq.LQ_BF16, vp(None), vp(wsp),
                                             size, vp(None))

    def bwd(w=W, X=A, M=300, d=drop(dr), wsp=A, size=wb):
        return L.lq_adapters_backward_dropout(w, vp(X), vp(A), M, S, vp(A), vp(None), d, vp(None), vp(A), vp(A), vp(A),
                                              vp(wsp), size, vp(None))
    for kw in BAD:
        assert fwd(d=drop(dr, **kw)) == lq.LQ_ERR_ARG and bwd(d=drop(dr, **kw)) == lq.LQ_ERR_ARG, kw
    assert fwd(d=None) == lq.LQ_ERR_ARG and bwd(d=None) == lq.LQ_ERR_ARG
    assert fwd(size=ws - 1) == lq.LQ_ERR_WORKSPACE and bwd(size=wb - 1) == lq.LQ_ERR_WORKSPACE
    assert fwd(X=None) == lq.LQ_ERR_ARG and bwd(X=None) == lq.LQ_ERR_ARG and fwd(H=A + 8) == lq.LQ_ERR_ARG
    assert fwd(M=0) == lq.LQ_ERR_SHAPE and bwd(M=1 << 31) == lq.LQ_ERR_SHAPE
    wide = ctypes.byref(nf4(lq, K=1 << 18))      # M K = 2^47: past the generator's count
    assert fwd(w=wide, M=1 << 29) == lq.LQ_ERR_SHAPE and bwd(w=wide, M=1 << 29) == lq.LQ_ERR_SHAPE
    assert L.lq_adapters_forward_dropout_workspace(wide, 1 << 29, S) == 0
    assert L.lq_adapters_backward_dropout_workspace(wide, 1 << 29, S) == 0


@pytest.mark.parametrize("M,rank,shares", [(1024, 64, 8), (4096, 64, 8), (16384, 64, 2), (65536, 128, 1)])
def test_partial_sums_of_t_take_what_their_call_can_use(lq, ad, M, rank, shares):
    """Workspaces of large calls: route, three terms, the weight, and as many partial sums of t as the tokens' 64-row
    tiles leave CUs for; dropout may split the columns further, up to 4096 tiles of sums in all."""
    N = K = 4096
    w, s = ctypes.byref(nf4(lq, N, K)), ctypes.byref(make_set(ad, [rank] * 4))
    plain, drops = lq.lib.lq_adapters_forward_workspace(w, M, s), lq.lib.lq_adapters_forward_dropout_workspace(w, M, s)
    sums = 4 * M * rank
    known = lq.lib.lq_adapter_route_bytes(M, 4) + 2 * 3 * M * rank + 2 * N * K
    pieces = 8 * 256      # each begins at a multiple of 256 bytes
    assert known + sums <= plain <= known + shares * sums + pieces
    assert plain <= drops <= known + max(shares, min(16, 4096 * 64 // M)) * sums + pieces
    known += 2 * (3 * M * rank) + 2 * 4 * rank * (N + K) + 2 * (2 * -(-M // 256) * rank * K * 4)
    plain, drops = lq.lib.lq_adapters_backward_workspace(w, M, s), lq.lib.lq_adapters_backward_dropout_workspace(w, M, s)
    assert known + 2 * sums <= plain <= known + 2 * shares * sums + 2 * pieces
    assert plain <= drops <= known + 2 * max(shares, min(16, 4096 * 64 // M)) * sums + 2 * pieces
