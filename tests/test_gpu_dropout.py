"""GPU parity of dropout: of a tensor (exactly), and inside the many-adapter
forward and backward against the formulas in float64.

Tolerances of the products as in test_gpu_adapters.py, element by element from
the sums of the absolute values of the terms; the factor of the kept elements
adds its own rounding and one product's to t and u (2 U of each).
"""
import numpy as np
import pytest

from oracle import dropout as odr
from test_gpu_adapters import U, Layer, assert_within, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


SEED, STEP = 0x9876543210ABCDEF, 0xFEDCBA9876543211


def expected(torch, x, p, site, seed=SEED, step=STEP):
    mask, factor = odr.kept(seed, step, site, p, tuple(x.shape))
    mask = torch.from_numpy(mask).cuda()
    return torch.where(mask, (x.float() * torch.tensor(factor, dtype=torch.float32, device="cuda")).to(x.dtype),
                       torch.zeros_like(x))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("numel", [1, 7, 8, 9, 4096, 300 * 1021, (1 << 20) + 5])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.99999999])
def test_dropout(lq, torch, dtype, numel, p):
    dt = getattr(torch, dtype)
    x = torch.randn(numel + 1, generator=torch.Generator(device="cuda").manual_seed(numel), device="cuda").to(dt)
    x[::5] = float("nan")
    x[3::7] = -float("inf")
    for off in (0, 1):      # the second at an address that is aligned to the element alone
        v = x[off:off + numel]
        drop = lq.Dropout(p, lq.dropout_key(SEED, STEP), site=77)
        y = lq.dropout(v, drop)
        want = expected(torch, v, p, 77)
        same = (y == want) | (torch.isnan(y) & torch.isnan(want))
        assert same.all() and not torch.signbit(y[(want == 0) & (v != 0)]).any()
        z = v.clone()
        assert lq.dropout(z, drop, out=z) is z
        assert torch.equal(z.view(torch.uint8), y.view(torch.uint8))
        w = torch.full((numel + 2,), 7.0, dtype=dt, device="cuda")      # what lies around the output stays
        lq.dropout(v, drop, out=w[1:-1])
        assert torch.equal(w[1:-1].view(torch.uint8), y.view(torch.uint8)) and w[0] == 7 and w[-1] == 7


def test_empty_and_sites(lq, torch):
    key = lq.dropout_key(1, 2)
    assert lq.dropout(torch.empty(0, 5, device="cuda"), lq.Dropout(0.5, key)).shape == (0, 5)
    x = torch.ones(64, 64, device="cuda")
    a, b = lq.dropout(x, lq.Dropout(0.5, key, 0)), lq.dropout(x, lq.Dropout(0.5, key, (1 << 20) - 1))
    assert not torch.equal(a, b)
    assert torch.equal(b, expected(torch, x, 0.5, (1 << 20) - 1, 1, 2))
    assert torch.equal(lq.dropout(x, lq.Dropout(0.5, lq.dropout_key(1, 3))), expected(torch, x, 0.5, 0, 1, 3))


def test_refusals(lq, torch):
    key = lq.dropout_key(0)
    for kw in (dict(p=1.0), dict(p=-0.5), dict(p=float("nan")), dict(site=-1), dict(site=1 << 20), dict(key=key.cpu()),
               dict(key=key.int()), dict(key=torch.zeros(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            lq.Dropout(**{**dict(p=0.1, key=key, site=0), **kw})
    d = lq.Dropout(0.1, key)
    x = torch.ones(8, 8, device="cuda")
    for bad in (x.t()[1:], x.double(), x.cpu(), x[:, 1:]):
        with pytest.raises(ValueError):
            lq.dropout(bad, d)
    flat = torch.ones(100, device="cuda")
    for out in (x.bfloat16(), torch.ones(8, 9, device="cuda"), x.cpu()):
        with pytest.raises(ValueError):
            lq.dropout(x, d, out=out)
    with pytest.raises(ValueError):
        lq.dropout(flat[:64], d, out=flat[1:65])


def test_a_captured_step_draws_anew(lq, torch):
    """A graph that advances the key gives the eager result of every step."""
    key = lq.dropout_key(11, 100)
    drop = lq.Dropout(0.3, key, 4)
    x = torch.randn(333, 77, device="cuda").to(torch.bfloat16)
    y = torch.empty_like(x)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lq.dropout(x, drop, out=y)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lq.dropout(x, drop, out=y)
        key[1] += 1
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, expected(torch, x, 0.3, 4, 11, 100 + k))
        x.normal_()


# ---- inside the adapters ---------------------------------------------------------
def reference(torch, L, mask, factor, t=None):
    """The formulas in float64: outputs and sums of absolute values."""
    W, X, G = torch.from_numpy(L.Wd).cuda(), L.X.double(), L.G.double()
    keep = torch.from_numpy(mask).cuda().double() * factor
    D = torch.where(keep > 0, X, 0.0) * keep
    n, r_max = len(L.adapters), L.set.r_max
    H, mH, gx, mX = X @ W.T, X.abs() @ W.abs().T, G @ W, G.abs() @ W.abs()
    lH, lX = torch.zeros_like(H), torch.zeros_like(gx)
    T, mT = torch.zeros(L.M, r_max, dtype=torch.float64, device="cuda"), torch.zeros(L.M, r_max, dtype=torch.float64, device="cuda")
    dA, dB = [], []
    for a, (A, B, _) in enumerate(L.adapters):
        m = (L.ids_dev == a).nonzero()[:, 0]
        A, B, s, r = A.double(), B.double(), L.host[a][2], A.shape[0]
        ta, tm = D[m] @ A.T, D[m].abs() @ A.abs().T
        T[m, :r], mT[m, :r] = ta, tm
        H[m] += s * ta @ B.T
        lH[m] = s * tm @ B.abs().T
        u, um = G[m] @ B, G[m].abs() @ B.abs()
        gx[m] += s * (u @ A) * keep[m]
        lX[m] = s * (um @ A.abs()) * keep[m]
        if t is not None:
            ta, tm = t[m, :r].double(), t[m, :r].double().abs()
        dA.append((s * u.T @ D[m], s * um.T @ D[m].abs()))
        dB.append((s * G[m].T @ ta, s * G[m].abs().T @ tm))
    return (H, mH, lH), (T, mT), (gx, mX, lX), dA, dB


def inside(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


def check(lq, torch, L, p, out="bf16", saved=True, site=9):
    dt = torch.float32 if out == "f32" else torch.bfloat16
    drop = lq.Dropout(p, lq.dropout_key(SEED, STEP), site)
    mask, factor = odr.kept(SEED, STEP, site, p, (L.M, L.K))
    H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=dt, dropout=drop)
    (rH, mH, lH), (T, mT), (rX, mX, lX), rA, rB = reference(torch, L, mask, factor, t if saved else None)
    r, N, K = L.set.r_max, L.N, L.K
    tiny = 2.0 ** -130
    inside(t, T, (K + 10) * U * mT, "t")
    hb = (K + 3 * r + 8) * U * (mH + lH) + (K + 2) * U * lH
    if out == "bf16":
        hb += 2.0 ** -16 * lH + 2.0 ** -8 * rH.abs() + tiny
    inside(H, rH, hb, "H")
    if N % 8:
        return
    gx, dA, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t if saved else None, dropout=drop)
    xb = (N + 3 * r + 8) * U * (mX + lX) + (N + 2) * U * lX + 2.0 ** -16 * lX + 2.0 ** -8 * rX.abs() + tiny
    inside(gx, rX, xb, "grad_X")
    for a, (da, db) in enumerate(L.set.split(dA, dB)):
        tokens = int((L.ids == a).sum())
        inside(da, rA[a][0], (3 * tokens + N + 18) * U * rA[a][1], f"dA {a}")
        inside(db, rB[a][0], (3 * tokens + (0 if saved else K + 2) + 16) * U * rB[a][1], f"dB {a}")
    return H, t, gx, dA, dB


CASES = [
    # N, K, M, ranks, ids, weight, p, out, saved t
    (64, 64, 1, [8], "mixed", "nf4_dq", 0.5, "bf16", True),
    (72, 128, 16, [16, 4, 1], "mixed", "nf4_f32", 0.1, "f32", False),
    (264, 320, 33, [4, 7, 16, 33, 64], "mixed", "nf4_dq", 0.05, "bf16", False),
    (77, 192, 64, [5, 24], "runs", "codebook", 0.2, "f32", True),
    (512, 256, 300, [16, 8, 64, 1, 7], "runs", "nf4_dq", 0.1, "f32", True),
    (200, 448, 517, [12, 40], "mixed", "codebook", 0.9, "bf16", False),
    (128, 64, 1025, [128, 3], "runs", "nf4_f32", 0.05, "bf16", False),
    (256, 256, 129, [16] * 40, "mixed", "nf4_dq", 0.1, "bf16", True),
    (264, 192, 2100, [16], "runs", "nf4_dq", 0.3, "f32", False),
    (136, 192, 4500, [16, 32], "runs", "nf4_dq", 0.1, "bf16", False),      # t in tiles, ranks up to 32
    (1000, 320, 1100, [64, 64, 64], "runs", "nf4_dq", 0.05, "bf16", True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_adapters(lq, torch, case):
    N, K, M, ranks, ids, weight, p, out, saved = case
    check(lq, torch, Layer(lq, torch, N, K, M, ranks, ids, weight), p, out, saved)


# the result of the backward is [M, K]: tiles of 256 x 128 (first two), 256 x 256, and 64 x 64 above the CUs' count
@pytest.mark.parametrize("case", [(72, 4096, 2047, [16, 8, 64, 24], "runs", "nf4_dq"),
                                  (64, 4096, 1800, [16] * 9, "mixed", "codebook"),
                                  (136, 8192, 4001, [64, 16, 128], "runs", "nf4_dq"),
                                  (64, 8192, 4096, [32, 7, 16, 8], "mixed", "nf4_f32"),
                                  (200, 1088, 1999, [3, 64] * 20, "mixed", "nf4_dq")], ids=str)
def test_large(lq, torch, case):
    N, K, M, ranks, ids, weight = case
    check(lq, torch, Layer(lq, torch, N, K, M, ranks, ids, weight), 0.1, saved=False)


@pytest.mark.parametrize("case", [(64, 1024, 20480, [16, 40], "runs", "nf4_dq"), (64, 192, 70000, [7], "mixed", "nf4_dq")], ids=str)
def test_more_tokens_than_a_share_each(lq, torch, case):
    """t in tiles of so many tokens that the columns' shares are fewer than they could be."""
    test_large(lq, torch, case)


def test_no_token_has_an_adapter(lq, torch):
    for N, K, M in ((128, 128, 70), (64, 4096, 2048), (64, 8192, 4096)):
        check(lq, torch, Layer(lq, torch, N, K, M, [16, 8], ids=np.full(M, -1)), 0.5)


def test_rate_zero_is_no_dropout(lq, torch):
    for M in (65, 300, 2049):
        L = Layer(lq, torch, 264, 320, M, [16, 40, 7])
        drop = lq.Dropout(0.0, lq.dropout_key(3), 1)
        H0, t0 = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev)
        H1, t1 = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, dropout=drop)
        assert torch.equal(H0, H1) and torch.equal(t0, t1)
        for a, b in zip(lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev),
                        lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, dropout=drop)):
            assert torch.equal(a, b)


def test_the_adapters_see_the_dropped_tensor(lq, torch):
    """At rate 1/2 the factor is 2: t is that of dropout(X) itself, and the gradient of D passes dropout's own mask."""
    L = Layer(lq, torch, 256, 512, 300, [16, 8])
    drop = lq.Dropout(0.5, lq.dropout_key(5, 6), 2)
    _, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, dropout=drop)
    _, t2 = lq.adapters_forward(L.qw, lq.dropout(L.X, drop), L.set, L.ids_dev)
    assert torch.equal(t, t2)      # a power of two commutes with every rounding


@pytest.mark.parametrize("M", [50, 300, 2048])
def test_what_is_not_finite_and_dropped(lq, torch, M):
    """A dropped NaN of X reaches neither t nor dA; an adapter's infinity reaches the kept elements of grad_X alone."""
    K = 4096 if M == 2048 else 128
    L = Layer(lq, torch, 72, K, M, [16, 8], seed=5)
    drop = lq.Dropout(0.5, lq.dropout_key(SEED, STEP), 9)
    mask, _ = odr.kept(SEED, STEP, 9, 0.5, (M, K))
    dropped = torch.from_numpy(~mask).cuda()
    t0 = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, dropout=drop)[1]
    gx0, dA0, _ = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t0, dropout=drop)
    X = torch.where(dropped, float("nan"), L.X)
    assert torch.equal(lq.adapters_forward(L.qw, X, L.set, L.ids_dev, dropout=drop)[1], t0)
    assert torch.equal(lq.adapters_backward(L.qw, X, L.G, L.set, L.ids_dev, t=t0, dropout=drop)[1], dA0)
    L.adapters[0][0].fill_(float("inf"))
    gx1 = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t0, need_dA=False, need_dB=False, dropout=drop)[0]
    mine = (L.ids_dev == 0)[:, None]
    assert torch.equal(gx1[~mine[:, 0]], gx0[~mine[:, 0]])
    assert torch.equal(torch.isfinite(gx1), ~(mine & ~dropped))
    assert torch.equal(gx1[mine & dropped], gx0[mine & dropped])


def test_repeats_and_route(lq, torch):
    for M in (40, 333, 1500):
        L = Layer(lq, torch, 264, 320, M, [16, 8, 40])
        drop = lq.Dropout(0.1, lq.dropout_key(1), 1)
        route = lq.adapter_route(L.ids_dev, 3)
        runs = [(*lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, dropout=drop, route=r),
                 *lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, dropout=drop, route=r)) for r in (None, route)]
        assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_a_captured_training_step(lq, torch):
    """Forward and backward in one graph, the key advanced at its end: each replay is that step's eager result."""
    L = Layer(lq, torch, 264, 320, 300, [16, 40])
    key = lq.dropout_key(21, 500)
    drop = lq.Dropout(0.2, key, 3)

    def step():
        H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, dropout=drop)
        return (H, t, *lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t, dropout=drop))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
        key[1] += 1
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        eager = lq.Dropout(0.2, lq.dropout_key(21, 500 + k), 3)
        H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, dropout=eager)
        want = (H, t, *lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t, dropout=eager))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        L.X.copy_(torch.randn_like(L.X))
        torch.cuda.synchronize()


def test_gradients_against_differences(lq, torch):
    """d/d eps of sum(H * R) along a direction of A and of B, under one mask, by central differences in
    float64 of the oracle's forward at the masked X; the kernels' gradients give the same number."""
    L = Layer(lq, torch, 64, 128, 90, [8, 16], seed=2)
    drop = lq.Dropout(0.25, lq.dropout_key(SEED, STEP), 9)
    mask, factor = odr.kept(SEED, STEP, 9, 0.25, (90, 128))
    D = f64(L.X) * mask * factor
    _, dA, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, dropout=drop)
    G, rng = f64(L.G), np.random.default_rng(1)
    for a, (da, db) in enumerate(L.set.split(dA, dB)):
        A, B, s = L.host[a]
        m = np.nonzero(L.ids == a)[0]
        VA, VB = rng.standard_normal(A.shape), rng.standard_normal(B.shape)

        def loss(e, f):
            return float(((s * D[m] @ (A + e * VA).T @ (B + f * VB).T) * G[m]).sum())
        h = 1e-3      # the loss is linear in e and in f apart: differences are exact up to float64
        for got, v, d in ((f64(da), VA, (loss(h, 0) - loss(-h, 0)) / (2 * h)), (f64(db), VB, (loss(0, h) - loss(0, -h)) / (2 * h))):
            terms = np.abs(got * v).sum()
            assert abs((got * v).sum() - d) <= (3 * len(m) + 128 + 64 + 32) * U * 40 * terms + 1e-7 * abs(d)


def test_elements_past_32_bits(lq, torch):
    """A tensor of more than 2^35 elements: the block counter's upper word, and more than one share a workgroup."""
    numel = (1 << 35) + 1003
    if torch.cuda.mem_get_info()[0] < 3 * numel:
        pytest.skip("needs 96 GiB of device memory")
    x = torch.ones(numel, dtype=torch.bfloat16, device="cuda")
    drop = lq.Dropout(0.5, lq.dropout_key(SEED, STEP), site=(1 << 20) - 1)
    lq.dropout(x, drop, out=x)
    for first in (0, (1 << 31) - 500, (1 << 32) - 500, (1 << 34) + 77, (1 << 35) - 500, numel - 1000):
        kept = odr.fields(SEED, STEP, (1 << 20) - 1, first, 1000) >= 32768
        assert np.array_equal(x[first:first + 1000].float().cpu().numpy(), 2.0 * kept), first


def test_adapters_past_32_bits(lq, torch):
    """M K past 2^31 elements: the rows at the end against the formulas (t, grad_X), and every row's dropout in dA."""
    N, K, r, p, site = 64, 65536, 4, 0.25, 3
    M = (1 << 31) // K + 300
    L = Layer(lq, torch, N, K, 40, [r], ids=np.zeros(40, dtype=np.int64))
    X = torch.randn(M, K, dtype=torch.bfloat16, device="cuda")
    G = torch.randn(M, N, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    drop = lq.Dropout(p, lq.dropout_key(SEED, STEP), site)
    H, t = lq.adapters_forward(L.qw, X, L.set, ids, dropout=drop)
    gx, dA, dB = lq.adapters_backward(L.qw, X, G, L.set, ids, t=t, dropout=drop)
    (A, B, _), s = L.adapters[0], L.host[0][2]
    A, B, W = A.double(), B.double(), torch.from_numpy(L.Wd).cuda()
    cols = torch.arange(K - 64, K, device="cuda")          # of dA: 64 columns over all rows
    keepc = torch.empty(M, 64, dtype=torch.bool)
    rows = np.arange(M - 20, M)
    factor = 65536.0 / (65536.0 - odr.threshold(p))
    for m in range(M):
        keepc[m] = torch.from_numpy(odr.fields(SEED, STEP, site, m * K + K - 64, 64) >= odr.threshold(p))
    u = G.double() @ B
    D = X[:, cols].double() * keepc.cuda() * factor
    ref, mag = s * u.T @ D, s * (G.double().abs() @ B.abs()).T @ D.abs()
    got = L.set.split(dA, dB)[0][0]
    inside(got[:, cols], ref, (3 * M + N + 18) * U * mag, "dA")
    keep = torch.from_numpy(odr.fields(SEED, STEP, site, int(rows[0]) * K, 20 * K).reshape(20, K) >= odr.threshold(p)).cuda()
    D = X[M - 20:].double() * keep * factor
    ta, tm = D @ A.T, D.abs() @ A.abs().T
    inside(t[M - 20:], ta, (K + 10) * U * tm, "t")
    x, g = X[M - 20:].double(), G[M - 20:].double()
    h, mh, lh = x @ W.T + s * ta @ B.T, x.abs() @ W.abs().T, s * tm @ B.abs().T
    inside(H[M - 20:], h, (K + 3 * r + 8) * U * (mh + lh) + (K + 2) * U * lh + 2.0 ** -16 * lh + 2.0 ** -8 * h.abs(), "H")
    lx = s * (g.abs() @ B.abs()) @ A.abs() * keep * factor
    rx, mx = g @ W + s * (g @ B) @ A * keep * factor, g.abs() @ W.abs()
    inside(gx[M - 20:], rx, (N + 3 * r + 8) * U * (mx + lx) + (N + 2) * U * lx + 2.0 ** -16 * lx + 2.0 ** -8 * rx.abs() + 2.0 ** -130,
           "grad_X")
