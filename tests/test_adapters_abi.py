"""CPU tests of the many-adapter entry points: exports, refusals before any
launch, size queries, the host-built gradient table, and the oracle against a
loop over single adapters."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import adapters as oad
from oracle import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lq_adapters.h")
A = 0x10000            # 16-byte aligned fake device address, never dereferenced
vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def ad(lq):
    from quantized_lora_fine_lq_amd import adapters
    return adapters


def make_set(ad, ranks, **kw):
    arr = (ad.lq_adapter * len(ranks))()
    row = row8 = 0
    for i, r in enumerate(ranks):
        arr[i] = ad.lq_adapter(A, A, r, 2.0, row, row8)
        row, row8 = row + r, row8 + (r + 7) // 8 * 8
    d = dict(host=ctypes.addressof(arr), dev=A, n=len(ranks), r_max=max(ranks))
    d.update(kw)
    s = ad.lq_adapter_set(**d)
    s.keep = arr
    return s


def nf4(lq, N=128, K=256, **kw):
    d = dict(format=0, blocksize=64, N=N, K=K, codes=A, absmax=A, absmax_q=None, dq_scale=None, dq_mean=None,
             dq_blocksize=256, reserved0=0, row_bits=None, row_offset=None, levels=None)
    d.update(kw)
    return lq.lq_qweight(**d)


def test_every_declared_symbol_is_exported(lq, ad):
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(lq_\w+)\s*\(", text, re.M)))
    assert names == sorted(ad.SIGNATURES)
    dbg = ad.declare(lq.load_debug_library())
    for name in names:
        assert hasattr(lq.lib, name) and hasattr(dbg, name)
    assert int(re.search(r"#define LQ_ADAPTERS_MAX (\d+)", text).group(1)) == ad.LQ_ADAPTERS_MAX


def test_check_adapters(lq, ad):
    ref = ctypes.byref
    check = lambda s, N=128, K=256: lq.lib.lq_check_adapters(ref(s), N, K)
    assert check(make_set(ad, [8, 16, 5])) == lq.LQ_OK
    assert lq.lib.lq_check_adapters(None, 128, 256) == lq.LQ_ERR_ARG
    for kw in (dict(host=None), dict(dev=None), dict(dev=A + 4), dict(r_max=15), dict(r_max=17)):
        assert check(make_set(ad, [8, 16, 5], **kw)) == lq.LQ_ERR_ARG, kw
    for kw in (dict(n=0), dict(n=-1), dict(n=ad.LQ_ADAPTERS_MAX + 1)):
        assert check(make_set(ad, [8, 16, 5], **kw)) == lq.LQ_ERR_SHAPE, kw
    assert check(make_set(ad, [8]), 0, 256) == lq.LQ_ERR_SHAPE
    for bad in ([0, 8], [8, 129]):
        assert check(make_set(ad, bad)) == lq.LQ_ERR_SHAPE
    for field, value in (("A", None), ("B", None), ("A", A + 8), ("B", A + 2), ("row", 9), ("row8", 7)):
        s = make_set(ad, [8, 16])
        setattr(s.keep[1], field, value)
        assert check(s) == lq.LQ_ERR_ARG, field


def test_route_refusals(lq, ad):
    L = lq.lib
    size = L.lq_adapter_route_bytes(100, 7)
    assert size >= 4 * (9 + 200)
    assert L.lq_adapter_route_bytes(0, 7) == 0 and L.lq_adapter_route_bytes(1 << 31, 7) == 0
    assert L.lq_adapter_route_bytes(100, 0) == 0 and L.lq_adapter_route_bytes(100, ad.LQ_ADAPTERS_MAX + 1) == 0
    call = lambda ids=A, M=100, n=7, route=A, b=size: L.lq_adapter_route(vp(ids), M, n, vp(route), b, vp(None))
    assert call(ids=None) == lq.LQ_ERR_ARG and call(route=None) == lq.LQ_ERR_ARG
    assert call(ids=A + 2) == lq.LQ_ERR_ARG and call(route=A + 4) == lq.LQ_ERR_ARG
    assert call(M=0) == lq.LQ_ERR_SHAPE and call(n=0) == lq.LQ_ERR_SHAPE
    assert call(b=size - 1) == lq.LQ_ERR_WORKSPACE


def test_forward_and_backward_refusals(lq, ad):
    L = lq.lib
    w, s = nf4(lq), make_set(ad, [8, 16, 5])
    W, S = ctypes.byref(w), ctypes.byref(s)
    ws = L.lq_adapters_forward_workspace(W, 300, S)
    assert ws > 0
    assert L.lq_adapters_forward_workspace(W, 0, S) == 0 and L.lq_adapters_forward_workspace(W, 300, None) == 0

    def fwd(w=W, X=A, M=300, set_=S, ids=A, route=None, H=A, dt=lq.LQ_BF16, t=None, wsp=A, size=ws):
        return L.lq_adapters_forward(w, vp(X), M, set_, vp(ids), vp(route), vp(H), dt, vp(t), vp(wsp), size, vp(None))
    assert fwd(size=ws - 1) == lq.LQ_ERR_WORKSPACE and fwd(wsp=None) == lq.LQ_ERR_WORKSPACE
    for kw in (dict(X=None), dict(ids=None), dict(H=None), dict(X=A + 8), dict(ids=A + 2), dict(H=A + 8),
               dict(t=A + 2), dict(route=A + 4), dict(wsp=A + 8), dict(w=None), dict(set_=None)):
        assert fwd(**kw) == lq.LQ_ERR_ARG, kw
    assert fwd(M=0) == lq.LQ_ERR_SHAPE and fwd(M=1 << 31) == lq.LQ_ERR_SHAPE
    assert fwd(dt=lq.LQ_F16) == lq.LQ_ERR_UNSUPPORTED
    assert fwd(set_=ctypes.byref(make_set(ad, [8], r_max=9))) == lq.LQ_ERR_ARG
    assert fwd(w=ctypes.byref(nf4(lq, K=100))) == lq.LQ_ERR_SHAPE

    wb = L.lq_adapters_backward_workspace(W, 300, S)
    assert wb > 0

    def bwd(w=W, X=A, G=A, M=300, set_=S, ids=A, route=None, t=None, gx=A, dA=A, dB=A, wsp=A, size=wb):
        return L.lq_adapters_backward(w, vp(X), vp(G), M, set_, vp(ids), vp(route), vp(t), vp(gx), vp(dA), vp(dB),
                                      vp(wsp), size, vp(None))
    assert bwd(size=wb - 1) == lq.LQ_ERR_WORKSPACE and bwd(wsp=None) == lq.LQ_ERR_WORKSPACE
    for kw in (dict(X=None), dict(X=None, t=A), dict(G=None), dict(ids=None), dict(G=A + 8), dict(X=A + 8),
               dict(gx=A + 8), dict(dA=A + 2), dict(dB=A + 2), dict(t=A + 2), dict(route=A + 8), dict(wsp=A + 4)):
        assert bwd(**kw) == lq.LQ_ERR_ARG, kw
    odd = nf4(lq, N=100)
    assert bwd(w=ctypes.byref(odd)) == lq.LQ_ERR_SHAPE and bwd(M=0) == lq.LQ_ERR_SHAPE
    assert L.lq_adapters_backward_workspace(ctypes.byref(odd), 300, S) == 0


def grad_table(lq, ad, specs, n_groups):
    arr = (ad.lq_grad_tensor * max(len(specs), 1))(*[ad.lq_grad_tensor(*s) for s in specs])
    size = lq.lib.lq_grad_list_bytes(arr, len(specs), n_groups)
    lst = ad.lq_grad_list()
    buf = np.zeros(max(size, 16) // 8 + 2, dtype=np.uint64)
    st = lq.lib.lq_grad_list_build(arr, len(specs), n_groups, vp(buf.ctypes.data), size, ctypes.byref(lst))
    return st, lst, buf.view(np.uint8), size


@pytest.mark.parametrize("seed", range(6))
def test_grad_table_covers_every_element_once(lq, ad, seed):
    """Decodes the table: every element of every tensor lies in one piece, pieces of one slot are of its group, and
    the slots of a group follow each other."""
    rng = np.random.default_rng(seed)
    n_groups = int(rng.integers(1, 5))
    sizes = [int(v) for v in rng.choice([0, 1, 63, 4096, 4097, 100000, 3000001][:4 + seed // 2], rng.integers(0, 40))]
    specs, at = [], A
    for n in sizes:
        dt = int(rng.integers(0, 3))
        specs.append((at if n else None, n, dt, int(rng.integers(0, n_groups))))
        at += n * (4 if dt == 0 else 2) + 64
        at = (at + 3) // 4 * 4
    st, lst, buf, size = grad_table(lq, ad, specs, n_groups)
    assert st == lq.LQ_OK and lst.n_groups == n_groups
    slots = np.frombuffer(buf[:32 * lst.n_slots].tobytes(), dtype=np.int32).reshape(-1, 8)
    po = (32 * lst.n_slots + 255) // 256 * 256
    assert po + 16 * lst.n_pieces <= size
    pieces = np.frombuffer(buf[po:po + 16 * lst.n_pieces].tobytes(),
                           dtype=[("p", np.uint64), ("n", np.int32), ("dt", np.int32)])
    covered = np.zeros(lst.n_pieces, dtype=int)
    owner = {}
    for i, (first, count, group, gfirst, gcount, *_) in enumerate(slots):
        covered[first:first + count] += 1
        assert gfirst <= i < gfirst + gcount and (slots[gfirst:gfirst + gcount, 2] == group).all()
        for k in range(first, first + count):
            owner[k] = group
    assert (covered == 1).all() and set(slots[:, 2]) == set(range(n_groups))
    left = {i: (p, n) for i, (p, n, _, _) in enumerate(specs) if n}
    for k, (p, n, dt) in enumerate(pieces):
        hit = [i for i, (q, m) in left.items() if q == int(p) and specs[i][2] == dt and specs[i][3] == owner[k]]
        assert len(hit) == 1 and 0 < n <= left[hit[0]][1]
        q, m = left.pop(hit[0])
        if m > n:
            left[hit[0]] = (q + int(n) * (4 if dt == 0 else 2), m - int(n))
    assert not left


def test_grad_list_refusals(lq, ad):
    ok = (A, 10, 0, 0)
    assert grad_table(lq, ad, [ok], 1)[0] == lq.LQ_OK
    assert grad_table(lq, ad, [(None, 0, 0, 0)], 1)[0] == lq.LQ_OK
    for bad in ((None, 10, 0, 0), (A + 2, 10, 0, 0), (A + 1, 10, 1, 0), (A, 10, 3, 0), (A, 10, 0, 1), (A, 10, 0, -1)):
        assert grad_table(lq, ad, [bad], 1)[0] == lq.LQ_ERR_ARG, bad
    assert grad_table(lq, ad, [(A, -1, 0, 0)], 1)[0] == lq.LQ_ERR_SHAPE
    assert grad_table(lq, ad, [(A, 1 << 50, 0, 0)], 1)[0] == lq.LQ_ERR_SHAPE
    assert grad_table(lq, ad, [ok], 0)[0] == lq.LQ_ERR_SHAPE and grad_table(lq, ad, [ok], 65536)[0] == lq.LQ_ERR_SHAPE
    arr = (ad.lq_grad_tensor * 1)(ad.lq_grad_tensor(*ok))
    size = lq.lib.lq_grad_list_bytes(arr, 1, 1)
    lst, buf = ad.lq_grad_list(), np.zeros(size, dtype=np.uint8)
    build = lambda t, b: lq.lib.lq_grad_list_build(arr, 1, 1, t, b, ctypes.byref(lst))
    assert build(vp(buf.ctypes.data), size - 1) == lq.LQ_ERR_WORKSPACE and build(None, size) == lq.LQ_ERR_ARG

    _, a, _, _ = grad_table(lq, ad, [ok], 1)
    _, b, _, _ = grad_table(lq, ad, [(A, 11, 0, 0)], 1)
    a.dev = b.dev = A
    ws = lq.lib.lq_grad_norm_workspace(ctypes.byref(a))
    assert ws >= 8

    def clip(x=a, y=a, m=1.0, eps=1e-6, norms=A, wsp=A, size=ws):
        return lq.lib.lq_clip_grad_norm(ctypes.byref(x), ctypes.byref(y), m, eps, vp(norms), vp(wsp), size, vp(None))
    assert clip(y=b) == lq.LQ_ERR_ARG          # other sizes
    for kw in (dict(m=-1.0), dict(m=float("nan")), dict(m=float("inf")), dict(eps=0.0), dict(eps=float("nan")),
               dict(norms=None), dict(norms=A + 2), dict(wsp=A + 4)):
        assert clip(**kw) == lq.LQ_ERR_ARG, kw
    assert clip(size=ws - 1) == lq.LQ_ERR_WORKSPACE and clip(wsp=None) == lq.LQ_ERR_WORKSPACE
    unset = ad.lq_grad_list()
    assert clip(x=unset, y=unset) == lq.LQ_ERR_ARG
    norm = lambda l, n=A, size=ws: lq.lib.lq_grad_norm(ctypes.byref(l), vp(n), vp(A), size, vp(None))
    assert norm(unset) == lq.LQ_ERR_ARG and norm(a, None) == lq.LQ_ERR_ARG and norm(a, A, 0) == lq.LQ_ERR_WORKSPACE


def test_oracle_equals_single_adapter_layers():
    """The oracle's rows of each adapter are the single-adapter oracle's on those tokens."""
    rng = np.random.default_rng(2)
    N, K, M = 24, 64, 19
    Wd, X, G = rng.standard_normal((N, K)), rng.standard_normal((M, K)), rng.standard_normal((M, N))
    ads = [(rng.standard_normal((r, K)), rng.standard_normal((N, r)), s) for r, s in ((3, 2.0), (8, 0.5), (1, 1.0))]
    ids = rng.integers(-1, 3, M)
    ids[ids == 2] = 0                           # adapter 2 has no tokens
    H, t, *_ = oad.forward(Wd, X, ads, ids)
    (dX, dA, dB), _ = oad.backward(Wd, X, G, ads, ids)
    for a, (A_, B_, s) in enumerate(ads):
        m, r = ids == a, A_.shape[0]
        h, tt = layer.forward(Wd, X[m], A_, B_, s * r)
        x, da, db = layer.backward(Wd, X[m], G[m], A_, B_, s * r)
        for got, want in ((H[m], h), (t[m, :r], tt), (dX[m], x), (dA[a], da), (dB[a], db)):
            assert np.allclose(got, want, rtol=1e-12, atol=1e-12)
    base = ids < 0
    assert np.allclose(H[base], X[base] @ Wd.T) and np.allclose(dX[base], G[base] @ Wd)
    assert not dA[2].any() and not dB[2].any()
    off, perm, sid = oad.route(ids, 3)
    assert sorted(perm) == list(range(M)) and (ids[perm][:off[3]] == sid[:off[3]]).all() and off[4] == M


def test_oracle_gradients_against_differences():
    """sum(G * H) is linear in each of X, A and B, so difference quotients are exact up to rounding."""
    rng = np.random.default_rng(4)
    N, K, M = 6, 10, 9
    Wd, X, G = rng.standard_normal((N, K)), rng.standard_normal((M, K)), rng.standard_normal((M, N))
    ads = [(rng.standard_normal((2, K)), rng.standard_normal((N, 2)), 1.5), (rng.standard_normal((3, K)), rng.standard_normal((N, 3)), 0.7)]
    ids = rng.integers(-1, 2, M)
    (dX, dA, dB), _ = oad.backward(Wd, X, G, ads, ids)
    loss = lambda X, ads: (G * oad.forward(Wd, X, ads, ids)[0]).sum()
    base = loss(X, ads)
    d = rng.standard_normal(X.shape)
    assert np.isclose(loss(X + d, ads) - base, (dX * d).sum())
    for a in range(2):
        for which, grad in ((0, dA), (1, dB)):
            d = rng.standard_normal(ads[a][which].shape)
            moved = [list(x) for x in ads]
            moved[a][which] = moved[a][which] + d
            assert np.isclose(loss(X, moved) - base, (grad[a] * d).sum())


def test_oracle_clip():
    x = [np.array([3.0, 0.0]), np.array([[4.0]]), np.array([1e3])]
    norms, out = oad.clip(x, [0, 0, 1], 3, 1.0, 1e-6)
    assert np.allclose(norms, [5.0, 1e3, 0.0])
    assert np.allclose(out[0], [3.0 / (5 + 1e-6), 0]) and np.allclose(out[1], 4.0 / (5 + 1e-6))
    norms, out = oad.clip(x, [0, 0, 0], 1, 1e4, 1e-6)
    assert all(np.array_equal(a, b) for a, b in zip(x, out))


# ---- routes that are not the call's: refused by the helpers before any launch ----
class FakeTensor:
    """As much of a device tensor as the helpers look at; never dereferenced."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, dtype):
        self.shape, self.dtype = tuple(shape), dtype

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def numel(self):
        return int(np.prod(self.shape))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return A


class Launched(Exception):
    pass


@pytest.fixture
def host_only(lq, ad, monkeypatch):
    """The helpers over fake tensors; the entry points that would launch raise Launched (adapter_route's returns)."""
    import types

    import torch

    def launch(*args):
        raise Launched
    stub = types.SimpleNamespace(int32=torch.int32, float32=torch.float32, bfloat16=torch.bfloat16, uint8=torch.uint8,
                                 empty=lambda n, dtype, device: FakeTensor((n,), dtype),
                                 empty_strided=lambda shape, stride, dtype, device: FakeTensor(shape, dtype))
    library = types.SimpleNamespace(**{name: getattr(lq.lib, name) for name in ad.SIGNATURES})
    library.lq_adapter_route = lambda *args: lq.LQ_OK
    library.lq_adapters_forward = library.lq_adapters_backward = launch
    monkeypatch.setattr(ad, "_torch", lambda: stub)
    monkeypatch.setattr(ad, "lib", library)
    monkeypatch.setattr(ad, "_stream", lambda dev: None)
    N, K, ranks = 128, 256, [8, 16, 5, 4]
    desc, c_set = nf4(lq, N, K), make_set(ad, ranks)
    qw = types.SimpleNamespace(N=N, K=K, device="cuda:0", ref=lambda: ctypes.byref(desc))
    adapters = types.SimpleNamespace(N=N, K=K, device="cuda:0", n=len(ranks), r_max=16, r_sum=33,
                                     ref=lambda: ctypes.byref(c_set))

    def call(which, M, route):
        ids, X = FakeTensor((M,), torch.int32), FakeTensor((M, K), torch.bfloat16)
        if which == "forward":
            ad.adapters_forward(qw, X, adapters, ids, route=route)
        else:
            ad.adapters_backward(qw, X, FakeTensor((M, N), torch.bfloat16), adapters, ids, route=route)
    return types.SimpleNamespace(call=call, ids=lambda M: FakeTensor((M,), torch.int32), ad=ad, lib=lq.lib,
                                 buffer=lambda words: FakeTensor((words,), torch.int32))


@pytest.mark.parametrize("which", ["forward", "backward"])
def test_a_route_of_other_tokens_or_adapters_is_refused(host_only, which):
    """Such a route's positions lie elsewhere in the buffer, and its tokens past the call's: read as this call's it
    would send the kernels out of range."""
    h = host_only
    for M in (1, 70, 128):                        # its own
        with pytest.raises(Launched):
            h.call(which, M, h.ad.adapter_route(h.ids(M), 4))
        with pytest.raises(Launched):
            h.call(which, M, None)
    for M, tokens, n in [(70, 128, 4),            # the last, shorter batch with the route of a full one
                         (70, 72, 4), (70, 71, 4), (70, 69, 4), (128, 70, 4),
                         (70, 70, 6), (70, 70, 3), (70, 70, 1000)]:
        if (tokens, n) in ((72, 4), (71, 4), (70, 6)):     # padded to the same size
            assert h.lib.lq_adapter_route_bytes(tokens, n) == h.lib.lq_adapter_route_bytes(M, 4)
        with pytest.raises(ValueError):
            h.call(which, M, h.ad.adapter_route(h.ids(tokens), n))
    # a buffer that no adapter_route call wrote
    with pytest.raises(ValueError):
        h.call(which, 70, h.buffer(h.lib.lq_adapter_route_bytes(70, 4) // 4))


def test_adapters_that_are_no_matrices_are_refused_in_words(ad):
    import torch
    m = lambda *shape: FakeTensor(shape, torch.bfloat16)
    ok = (m(8, 256), m(128, 8), 1.0)
    for bad in [(m(0, 256), m(128, 0), 1.0), (m(256), m(128, 8), 1.0), (m(8, 256), m(128), 1.0),
                (m(1, 8, 256), m(128, 8), 1.0), (m(), m(128, 8), 1.0)]:
        for adapters in ([bad], [ok, bad]):
            with pytest.raises(ValueError):
                ad.AdapterSet(adapters)
