"""GPU parity of the many-adapter path against the float64 oracle.

Tolerances are derived, element by element, from the sums of the absolute
values of the terms: float32 accumulation of n products in any order is off by
at most n * 2^-24 times that sum (the products of two bfloat16 values are exact
in float32); the adapter part of a bfloat16 result carries t and u as two
bfloat16 terms (2^-16 of each); a bfloat16 result adds half a unit in its last
place, 2^-8 of the value.
"""
import numpy as np
import pytest

from oracle import adapters as oad

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def make_weight(lq, torch, rng, N, K, weight):
    W = torch.from_numpy((rng.standard_normal((N, K)) * 0.02).astype(np.float32)).cuda()
    if weight == "codebook":
        bits = torch.from_numpy(rng.integers(1, 5, N).astype(np.uint8)).cuda()
        levels, thresholds, _ = lq.lloyd_codebooks(W[:, :8192].contiguous(), bits, max_iters=3)   # it fits shorter rows only
        return lq.QWeight.from_codebook(W, bits, thresholds, levels)
    return lq.QWeight.from_weight(W, double_quantize=weight == "nf4_dq")


class Layer:
    """Inputs of one case, on the device and as float64 values."""

    def __init__(self, lq, torch, N, K, M, ranks, ids="mixed", weight="nf4_dq", base=0.15, seed=0):
        rng = np.random.default_rng([seed, N, K, M, len(ranks)])
        bf = lambda shape, std=1.0: torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).cuda().to(
            torch.bfloat16)
        self.N, self.K, self.M, n = N, K, M, len(ranks)
        self.qw = make_weight(lq, torch, rng, N, K, weight)
        self.X, self.G = bf((M, K)), bf((M, N))
        self.adapters = [(bf((r, K), 0.05), bf((N, r), 0.05), float(rng.uniform(0.5, 3.0) * r)) for r in ranks]
        if isinstance(ids, str):
            if ids == "mixed":
                self.ids = rng.integers(0, n, M)
                self.ids[rng.random(M) < base] = -1
            else:      # runs: one request after the other
                cuts = np.sort(rng.integers(0, M + 1, n - 1))
                self.ids = np.repeat(rng.permutation(n), np.diff(np.concatenate([[0], cuts, [M]])))
        else:
            self.ids = np.asarray(ids)
        self.ids_dev = torch.from_numpy(self.ids.astype(np.int32)).cuda()
        self.set = lq.AdapterSet(self.adapters)
        self.Wd = f64(lq.dequant(self.qw))
        self.host = [(f64(A), f64(B), float(np.float32(alpha / A.shape[0]))) for A, B, alpha in self.adapters]


def assert_within(got, ref, bound, what):
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - ref) - bound)}"


def forward_bounds(L, ref, f32):
    H, t, mag, tmag, lora = ref
    r = max(A.shape[0] for A, _, _ in L.host)
    acc = (L.K + 3 * r + 8) * U * (mag + lora) + L.K * U * lora       # the sum; t's own error
    tb = (L.K + 8) * U * tmag
    if f32:
        return acc, tb
    return acc + 2.0 ** -16 * lora + 2.0 ** -8 * np.abs(H) + 2.0 ** -130, tb


def check_forward(lq, torch, L, out="bf16", route=None):
    dt = torch.float32 if out == "f32" else torch.bfloat16
    H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=dt, route=route)
    ref = oad.forward(L.Wd, f64(L.X), L.host, L.ids)
    hb, tb = forward_bounds(L, ref, out == "f32")
    assert_within(f64(t), ref[1], tb, "t")
    assert_within(f64(H), ref[0], hb, "H")
    return H, t


FORWARD = [
    # N, K, M, ranks, ids, weight, out
    (64, 64, 1, [8], "mixed", "nf4_dq", "bf16"),
    (80, 128, 1, [16, 4], "mixed", "nf4_f32", "f32"),
    (256, 512, 16, [16] * 16, "mixed", "nf4_dq", "bf16"),
    (256, 512, 16, [16] * 16, "mixed", "nf4_dq", "f32"),
    (264, 320, 33, [4, 7, 16, 33, 64], "mixed", "nf4_dq", "bf16"),
    (512, 1024, 64, [8, 16, 32], "mixed", "nf4_dq", "f32"),
    (100, 192, 64, [1, 128], "mixed", "nf4_f32", "bf16"),
    (77, 192, 65, [5, 24], "runs", "nf4_dq", "bf16"),
    (77, 192, 65, [5, 24], "runs", "codebook", "f32"),
    (512, 256, 300, [16, 8, 64, 1, 7], "runs", "nf4_dq", "bf16"),
    (300, 448, 517, [12, 40], "mixed", "nf4_f32", "f32"),
    (1000, 320, 700, [64, 64, 64], "runs", "nf4_dq", "bf16"),
    (256, 256, 129, [16] * 40, "mixed", "codebook", "bf16"),
    (128, 64, 1025, [128, 3], "runs", "nf4_dq", "f32"),
]


@pytest.mark.parametrize("case", FORWARD, ids=str)
def test_forward(lq, torch, case):
    N, K, M, ranks, ids, weight, out = case
    check_forward(lq, torch, Layer(lq, torch, N, K, M, ranks, ids, weight), out)


BACKWARD = [
    # N, K, M, ranks, ids, weight, saved t
    (64, 64, 1, [8], "mixed", "nf4_dq", False),
    (72, 128, 5, [16, 4, 1], "mixed", "nf4_f32", True),
    (264, 320, 33, [4, 7, 16, 33, 64], "mixed", "nf4_dq", False),
    (512, 256, 300, [16, 8, 64, 1, 7], "runs", "nf4_dq", True),
    (200, 448, 517, [12, 40], "mixed", "codebook", False),
    (1000, 320, 700, [64, 64, 64], "runs", "nf4_dq", True),
    (128, 64, 1025, [128, 3], "runs", "nf4_f32", False),
    (256, 256, 129, [16] * 40, "mixed", "nf4_dq", True),
    (264, 192, 2100, [16], "runs", "nf4_dq", False),
]


def check_backward(lq, torch, L, saved=False, route=None):
    t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev)[1] if saved else None
    gx, dA, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t, route=route)
    (rX, rA, rB), (mag, lora, mA, mB) = oad.backward(L.Wd, f64(L.X), f64(L.G), L.host, L.ids,
                                                     None if t is None else f64(t))
    r = L.set.r_max
    xb = (L.N + 3 * r + 8) * U * (mag + lora) + L.N * U * lora + 2.0 ** -16 * lora + 2.0 ** -8 * np.abs(rX) + 2.0 ** -130
    assert_within(f64(gx), rX, xb, "grad_X")
    for a, (da, db) in enumerate(L.set.split(dA, dB)):
        tokens = int((L.ids == a).sum())
        assert_within(f64(da), rA[a], (3 * tokens + L.N + 16) * U * mA[a], f"dA {a}")
        assert_within(f64(db), rB[a], (3 * tokens + (0 if saved else L.K) + 16) * U * mB[a], f"dB {a}")
    return gx, dA, dB


@pytest.mark.parametrize("case", BACKWARD, ids=str)
def test_backward(lq, torch, case):
    N, K, M, ranks, ids, weight, saved = case
    check_backward(lq, torch, Layer(lq, torch, N, K, M, ranks, ids, weight), saved)


def reference64(torch, L, t=None):
    """The oracle's formulas in float64 torch on the device, for the large shapes: outputs and absolute sums."""
    W, X, G = torch.from_numpy(L.Wd).cuda(), L.X.double(), L.G.double()
    H, mH, gx, mX = X @ W.T, X.abs() @ W.abs().T, G @ W, G.abs() @ W.abs()
    lH, lX = torch.zeros_like(H), torch.zeros_like(gx)
    dA, dB = [], []
    for a, (A, B, alpha) in enumerate(L.adapters):
        m = (L.ids_dev == a).nonzero()[:, 0]
        A, B, s = A.double(), B.double(), L.host[a][2]
        tm = X[m] @ A.T if t is None else t[m, :A.shape[0]].double()
        u = G[m] @ B
        ta, ua = X[m].abs() @ A.abs().T, G[m].abs() @ B.abs()
        H[m] += s * (X[m] @ A.T) @ B.T
        lH[m] = s * ta @ B.abs().T
        gx[m] += s * u @ A
        lX[m] = s * ua @ A.abs()
        dA.append((s * u.T @ X[m], s * ua.T @ X[m].abs()))
        dB.append((s * G[m].T @ tm, s * G[m].abs().T @ (ta if t is None else tm.abs())))
    return (H, mH, lH), (gx, mX, lX), dA, dB


LARGE = [
    # N, K, M, ranks, ids, weight: tiles of 256 x 128 (first three) and 256 x 256, uneven edges
    (4104, 192, 2047, [16, 8, 64, 24], "runs", "nf4_dq"),
    (4099, 64, 1800, [16] * 9, "mixed", "nf4_f32"),
    (4096, 320, 2048, [40], "runs", "codebook"),
    (8184, 128, 4001, [64, 16, 128], "runs", "nf4_dq"),
    (8192, 64, 4096, [32, 7, 16, 8], "mixed", "nf4_f32"),
]


@pytest.mark.parametrize("case", LARGE, ids=str)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_large_forward(lq, torch, case, out):
    N, K, M, ranks, ids, weight = case
    L = Layer(lq, torch, N, K, M, ranks, ids, weight)
    H, _ = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    (ref, mag, lora), _, _, _ = reference64(torch, L)
    bound = (K + 3 * max(ranks) + 8) * U * (mag + lora) + K * U * lora
    if out == "bf16":
        bound += 2.0 ** -16 * lora + 2.0 ** -8 * ref.abs() + 2.0 ** -130
    assert ((H.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("ranks,ids", [([16, 8, 7], "runs"), ([128] * 200, "mixed"), ([3, 64] * 20, "mixed")], ids=str)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_more_small_tiles_than_compute_units(lq, torch, ranks, ids, out):
    """Tiles of 64 x 64, one group of waves each; an adapter to nearly every token of a tile."""
    L = Layer(lq, torch, 1037, 192, 1999, ranks, ids)
    H, _ = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    (ref, mag, lora), _, _, _ = reference64(torch, L)
    bound = (192 + 3 * max(ranks) + 8) * U * (mag + lora) + 192 * U * lora
    if out == "bf16":
        bound += 2.0 ** -16 * lora + 2.0 ** -8 * ref.abs() + 2.0 ** -130
    assert ((H.double() - ref).abs() <= bound).all()
    if out == "bf16":
        B = Layer(lq, torch, 200, 1088, 1999, ranks, ids)
        gx = lq.adapters_backward(B.qw, B.X, B.G, B.set, B.ids_dev, need_dA=False, need_dB=False)[0]
        _, (ref, mag, lora), _, _ = reference64(torch, B)
        bound = (200 + 3 * max(ranks) + 8) * U * (mag + lora) + 200 * U * lora + 2.0 ** -16 * lora + 2.0 ** -8 * ref.abs()
        assert ((gx.double() - ref).abs() <= bound + 2.0 ** -130).all()


# the backward's result is [M, K], its contraction N: the same tiles with N and K exchanged
@pytest.mark.parametrize("case", [(200, 4096, 2047, [16, 8, 64, 24], "runs", "nf4_dq"),
                                  (64, 4096, 1800, [16] * 9, "mixed", "codebook"),
                                  (136, 8192, 4001, [64, 16, 128], "runs", "nf4_dq"),
                                  (328, 8192, 4096, [32, 7, 16, 8], "mixed", "nf4_f32")], ids=str)
def test_large_backward(lq, torch, case):
    N, K, M, ranks, ids, weight = case
    L = Layer(lq, torch, N, K, M, ranks, ids, weight)
    gx, dA, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev)
    _, (ref, mag, lora), rA, rB = reference64(torch, L)
    bound = (N + 3 * max(ranks) + 8) * U * (mag + lora) + N * U * lora + 2.0 ** -16 * lora + 2.0 ** -8 * ref.abs()
    assert ((gx.double() - ref).abs() <= bound + 2.0 ** -130).all()
    for a, (da, db) in enumerate(L.set.split(dA, dB)):
        tokens = int((L.ids == a).sum())
        assert ((da.double() - rA[a][0]).abs() <= (3 * tokens + N + 16) * U * rA[a][1]).all()
        assert ((db.double() - rB[a][0]).abs() <= (3 * tokens + K + 16) * U * rB[a][1]).all()


@pytest.mark.parametrize("M,n", [(1, 1), (2, 3), (63, 5), (64, 64), (65, 1), (1000, 40), (5000, 1000), (4096, 7)])
def test_route(lq, torch, M, n):
    rng = np.random.default_rng(M * 1001 + n)
    ids = rng.integers(-2, n + 2, M)         # ids outside [0, n) have no adapter
    ids[rng.random(M) < 0.1] = np.iinfo(np.int32).min
    ids[rng.random(M) < 0.1] = np.iinfo(np.int32).max
    got = lq.adapter_route(torch.from_numpy(ids.astype(np.int32)).cuda(), n).cpu().numpy()
    off, perm, sid = oad.route(ids, n)
    w = (n + 2 + 3) // 4 * 4
    m4 = (M + 3) // 4 * 4
    assert np.array_equal(got[:n + 2], off)
    assert np.array_equal(got[w:w + M], perm)
    assert np.array_equal(got[w + m4:w + m4 + M], sid)


def test_no_token_has_an_adapter(lq, torch):
    """Every id outside the set: the base projection alone, t = 0, zero gradients."""
    for M in (1, 16, 70, 300):
        L = Layer(lq, torch, 128, 128, M, [16, 8], ids=np.full(M, -1))
        _, t = check_forward(lq, torch, L)
        assert not t.any()
        _, dA, dB = check_backward(lq, torch, L)
        assert not dA.any() and not dB.any()


def test_all_tokens_share_one_adapter(lq, torch):
    """One adapter of several in use: the single-adapter entry points' results, up to float32 order."""
    for M in (1, 16, 64, 300):
        L = Layer(lq, torch, 256, 256, M, [8, 16, 32], ids=np.full(M, 1))
        check_forward(lq, torch, L, "f32")
        _, dA, dB = check_backward(lq, torch, L)
        parts = L.set.split(dA, dB)
        assert not parts[0][0].any() and not parts[2][1].any() and parts[1][0].any()


@pytest.mark.parametrize("M", [3, 16, 50, 64, 100, 300])
def test_an_adapters_infinities_stay_with_its_tokens(lq, torch, M):
    """NaN and infinities in one adapter's A and B, and in one token's X and G,
    reach that adapter's and that token's results alone."""
    L = Layer(lq, torch, 136, 128, M, [16, 8, 12], base=0.2, seed=3)
    H0, t0 = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=torch.float32)
    gx0, dA0, dB0 = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev)
    A, B, _ = L.adapters[1]
    A[3, 7] = float("nan")
    B[5, 2] = float("inf")
    B[100] = float("nan")
    bad_token = int(np.nonzero(L.ids != 0)[0][0]) if (L.ids != 0).any() else 0
    L.X[bad_token, 3] = float("nan")
    L.G[bad_token, 9] = float("inf")
    H1, t1 = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=torch.float32)
    gx1, dA1, dB1 = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev)
    clean = torch.from_numpy((L.ids != 1) & (np.arange(M) != bad_token)).cuda()
    assert clean.any()
    assert torch.equal(H0[clean], H1[clean]) and torch.equal(t0[clean], t1[clean])
    assert torch.equal(gx0[clean], gx1[clean])
    p0, p1 = L.set.split(dA0, dB0), L.set.split(dA1, dB1)
    for a in (0, 2):
        if a != L.ids[bad_token]:
            assert torch.equal(p0[a][0], p1[a][0]) and torch.equal(p0[a][1], p1[a][1])
    if ((L.ids == 1) & (np.arange(M) != bad_token)).any():
        mine = torch.from_numpy(L.ids == 1).cuda()
        assert torch.isnan(H1[mine][:, 100]).all()


def test_route_given_and_repeatable(lq, torch):
    """A route built once gives the results of a call that builds its own, and
    every call repeats bit for bit."""
    for M in (40, 333):
        L = Layer(lq, torch, 264, 320, M, [16, 8, 40])
        route = lq.adapter_route(L.ids_dev, 3)
        a, b = check_forward(lq, torch, L), check_forward(lq, torch, L, route=route)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        a, b = check_backward(lq, torch, L), check_backward(lq, torch, L, route=route)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_partial_outputs(lq, torch):
    """Each gradient alone equals the one of the full call."""
    L = Layer(lq, torch, 136, 192, 150, [16, 8])
    full = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev)
    for k in range(3):
        need = [i == k for i in range(3)]
        got = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, need_grad_x=need[0], need_dA=need[1],
                                   need_dB=need[2])
        assert torch.equal(got[k], full[k])
        assert all(got[i] is None for i in range(3) if i != k)
    # grad_X and dA with t given need no X for t; dB needs none at all
    t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev)[1]
    gx, _, dB = lq.adapters_backward(L.qw, None, L.G, L.set, L.ids_dev, t=t, need_dA=False)
    assert torch.equal(gx, full[0]) and dB is not None


def test_gradients_against_differences(lq, torch):
    """Directional differences of the float32 forward's loss sum(G * H) in A and
    B. H is linear in A and in B, so the difference quotient has no truncation
    error; what is left is the forward's float32 accumulation."""
    L = Layer(lq, torch, 128, 128, 90, [16, 8], ids="runs")
    _, dA, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev)
    G = f64(L.G)
    rng = np.random.default_rng(11)
    loss = lambda ads: (G * f64(lq.adapters_forward(L.qw, L.X, lq.AdapterSet(ads), L.ids_dev,
                                                   out_dtype=torch.float32)[0])).sum()
    for a in range(2):
        for which in (0, 1):
            P = L.adapters[a][which]
            step = torch.from_numpy(rng.choice([-0.25, 0.25], size=tuple(P.shape)).astype(np.float32)).cuda()
            # both points are bfloat16 values, so the direction is exact
            plus = (P.float() + step).to(torch.bfloat16)
            minus = (P.float() - step).to(torch.bfloat16)
            d = f64(plus) - f64(minus)
            vals, mags = [], []
            for Q in (plus, minus):
                ads = [list(x) for x in L.adapters]
                ads[a][which] = Q
                vals.append(loss([tuple(x) for x in ads]))
                host = [(f64(x), f64(y), float(np.float32(al / x.shape[0]))) for x, y, al in ads]
                _, _, mag, _, lora = oad.forward(L.Wd, f64(L.X), host, L.ids)
                mags.append((np.abs(G) * (mag + 2 * lora)).sum())
            g = f64(L.set.split(dA, dB)[a][which])
            tol = (L.K + 3 * 16 + 8) * U * sum(mags) + (3 * 90 + 128 + 16) * U * np.abs(g * d).sum()
            assert abs((vals[0] - vals[1]) - (g * d).sum()) <= tol


def test_on_a_side_stream(lq, torch):
    L = Layer(lq, torch, 136, 192, 150, [16, 8])
    want = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev)[0]
    s.synchronize()
    assert torch.equal(want, got)


# ---------------------------------------------------------------------------
# gradient norms and clipping
# ---------------------------------------------------------------------------
def grads_of(torch, rng, sizes, dtype, offset=0, scale=1.0):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    out = []
    for n in sizes:
        buf = torch.from_numpy((rng.standard_normal(n + offset) * scale).astype(np.float32)).cuda().to(dt)
        out.append(buf[offset:])
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("sizes", [[1], [0, 5, 0], [4096], [4097, 1, 63, 64, 65], [7] * 50, [100001, 33, 70000]], ids=str)
@pytest.mark.parametrize("limit", [0.25, 4.0])
def test_clip(lq, torch, dtype, offset, sizes, limit):
    rng = np.random.default_rng([len(sizes), sum(sizes), offset])
    xs = grads_of(torch, rng, sizes, dtype, offset)
    groups = [i % 3 for i in range(len(sizes))]
    host = [f64(x) for x in xs]
    scale = float(np.sqrt(sum(np.square(h).sum() for h in host)) / 2)
    lst = lq.GradList(xs, groups, n_groups=3)
    out = [torch.full_like(x, 7.0) for x in xs]
    max_norm = float(np.float32(max(scale, 1e-3) * limit))
    norms = lq.clip_grad_norm(lst, max_norm, out=lq.GradList(out, groups, n_groups=3))
    rn, rc = oad.clip(host, groups, 3, max_norm, 1e-6)
    # float64 sums of exact squares, one rounding to float32
    assert (np.abs(f64(norms) - rn) <= 2.0 ** -24 * rn * 1.001).all()
    assert torch.equal(lq.grad_norm(lst), norms)
    # the factor and the product in float32, rounded once to the type: bit for bit
    norms32 = norms.cpu().numpy()
    coef = np.minimum(np.float32(1), np.float32(max_norm) / (norms32 + np.float32(1e-6)))
    for x, h, o, g, ref in zip(xs, host, out, groups, rc):
        assert np.array_equal(f64(x), h)                     # the input stays
        want = torch.from_numpy(h.astype(np.float32) * coef[g]).to(o.dtype)
        assert torch.equal(o.cpu(), want)
        assert np.linalg.norm(f64(o) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    # in place, bit for bit the same
    again = lq.clip_grad_norm(lst, max_norm)
    assert torch.equal(again, norms)
    assert all(torch.equal(x, o) for x, o in zip(xs, out))


def test_clip_large_and_many_groups(lq, torch):
    rng = np.random.default_rng(5)
    sizes = [3_000_001, 12, 500_000] + [int(v) for v in rng.integers(1, 3000, 300)]
    xs = grads_of(torch, rng, sizes, "f32")
    groups = [int(v) for v in rng.integers(0, 70, len(sizes))]
    norms = lq.clip_grad_norm(lq.GradList(xs, groups, n_groups=80), 1.0, out=lq.GradList([torch.empty_like(x) for x in xs], groups, n_groups=80))
    rn, _ = oad.clip([f64(x) for x in xs], groups, 80, 1.0, 1e-6)
    assert (np.abs(f64(norms) - rn) <= 2.0 ** -24 * rn * 1.001).all()
    assert (f64(norms)[70:] == 0).all()                     # groups without tensors


def test_clip_extremes(lq, torch):
    """Squares past float32's range, subnormals, NaN and infinity by group."""
    big = torch.full((1000,), 3e38, device="cuda")
    tiny = torch.full((1000,), 1e-40, device="cuda")
    nan = torch.ones(300, device="cuda")
    nan[17] = float("nan")
    inf = torch.ones(300, device="cuda")
    inf[299] = float("inf")
    zero = torch.zeros(10, device="cuda")
    xs = [big, tiny, nan, inf, zero]
    norms = lq.clip_grad_norm(lq.GradList(xs, range(5)), 1.0)
    n = f64(norms)
    assert np.isinf(n[0])          # sqrt(1000) * 3e38 is past float32: the factor is 0
    assert abs(n[1] - np.sqrt(1000.0) * float(np.float32(1e-40))) <= 2.0 ** -149
    assert np.isnan(n[2]) and np.isinf(n[3]) and n[4] == 0
    assert not big.any() and torch.isnan(nan).all() and torch.isnan(inf[299]) and not inf[:299].any()
    assert not zero.any() and (tiny == 1e-40).all()
    assert lq.grad_norm(lq.GradList([torch.full((1000,), 1e30, device="cuda")])).item() == pytest.approx(
        float(np.sqrt(1000.0) * np.float32(1e30)), rel=2.0 ** -23)


def test_no_gradients(lq, torch):
    assert lq.grad_norm(lq.GradList([], n_groups=2)).tolist() == [0.0, 0.0]
    assert lq.clip_grad_norm(lq.GradList([], n_groups=1), 1.0).tolist() == [0.0]


DECODE = [
    # N, K, M, ranks, out: one, two and four row groups per workgroup by N; odd K / 64; N % 4; ranks % 8
    (4096, 192, 1, [16], "bf16"),
    (4090, 320, 20, [16, 3, 40], "f32"),
    (8200, 128, 1, [8, 5], "f32"),
    (8200, 192, 17, [16] * 5, "bf16"),
    (8191, 64, 64, [128, 1, 24], "bf16"),
    (16384, 192, 1, [64], "bf16"),
    (16386, 448, 30, [7, 16, 33, 64], "f32"),
    (16390, 1088, 64, [8, 16, 32] * 4, "bf16"),
    (20000, 64, 33, [100, 128], "f32"),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
@pytest.mark.parametrize("weight", ["nf4_dq", "nf4_f32"])
def test_decode_sizes(lq, torch, case, weight):
    N, K, M, ranks, out = case
    L = Layer(lq, torch, N, K, M, ranks, "mixed", weight)
    H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    (ref, mag, lora), _, _, _ = reference64(torch, L)
    bound = (K + 3 * max(ranks) + 8) * U * (mag + lora) + K * U * lora
    if out == "bf16":
        bound += 2.0 ** -16 * lora + 2.0 ** -8 * ref.abs() + 2.0 ** -130
    assert ((H.double() - ref).abs() <= bound).all()
    for m, a in enumerate(L.ids):      # t: zero past the adapter's rank and without one
        r = ranks[a] if a >= 0 else 0
        assert not t[m, r:].any() and bool(t[m, :r].any()) == (r > 0)
    again = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=H.dtype)
    assert torch.equal(again[0], H) and torch.equal(again[1], t)


@pytest.mark.parametrize("N", [48, 16400])
def test_decode_every_token_its_own_large_adapter(lq, torch, N):
    """64 adapters of rank 128 in float32: the most steps that the adapters' part can have."""
    check_forward(lq, torch, Layer(lq, torch, N, 64, 64, [128] * 64, ids=np.random.default_rng(0).permutation(64)), "f32")


@pytest.mark.parametrize("weight", ["nf4_dq", "codebook"])
@pytest.mark.parametrize("K", [12288, 49152, 49216])
def test_long_rows(lq, torch, K, weight):
    """Row constants that fill the LDS of the decode form, and rows past it."""
    check_forward(lq, torch, Layer(lq, torch, 24, K, 5, [16, 9], weight=weight))
    check_forward(lq, torch, Layer(lq, torch, 24, K, 64, [128, 9], weight=weight), "f32")


@pytest.mark.parametrize("M", [1, 16, 60, 200])
@pytest.mark.parametrize("weight", ["nf4_dq", "codebook"])
def test_in_a_graph(lq, torch, M, weight):
    """Captured forward and backward: every replay, with other work and
    other values between, equals the eager calls."""
    L = Layer(lq, torch, 264, 320, M, [16, 8, 40], weight=weight)

    def step():
        H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev)
        gx, dA, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t)
        return H, t, gx, dA, dB

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    rng = np.random.default_rng(M)
    for _ in range(4):
        L.X.copy_(torch.from_numpy(rng.standard_normal((M, 320)).astype(np.float32)).cuda())
        L.ids_dev.copy_(torch.from_numpy(rng.integers(-1, 3, M).astype(np.int32)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, step()):
            assert torch.equal(x, y)


def test_clip_in_a_graph(lq, torch):
    rng = np.random.default_rng(7)
    xs = grads_of(torch, rng, [4097, 63, 100001], "f32")
    out = [torch.zeros_like(x) for x in xs]
    src, dst = lq.GradList(xs, [0, 1, 0]), lq.GradList(out, [0, 1, 0])
    lq.clip_grad_norm(src, 1.0, out=dst)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norms = lq.clip_grad_norm(src, 1.0, out=dst)
    for k in range(4):
        for x in xs:
            x.mul_(1.5)
        graph.replay()
        got = [x.clone() for x in out]
        want = lq.clip_grad_norm(src, 1.0, out=dst)
        assert torch.equal(norms, want) and all(torch.equal(a, b) for a, b in zip(got, out))


def test_refusals(lq, torch):
    L = Layer(lq, torch, 64, 128, 5, [8, 4])
    X, ids, G = L.X, L.ids_dev, L.G
    wide = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    bad_forward = [
        dict(X=X.float()), dict(X=X.cpu()), dict(X=X[0]), dict(X=wide), dict(X=wide[:, ::2]), dict(X=X[:4]),
        dict(ids=ids.long()), dict(ids=ids[:3]), dict(ids=ids.cpu()), dict(ids=ids[:, None]),
        dict(ids=torch.zeros(10, dtype=torch.int32, device="cuda")[::2]),
        dict(out_dtype=torch.float16), dict(route=torch.zeros(3, dtype=torch.int32, device="cuda")),
        dict(route=torch.zeros(64, device="cuda")), dict(adapters=Layer(lq, torch, 64, 64, 1, [8]).set),
    ]
    for change in bad_forward:
        args = dict(qw=L.qw, X=X, adapters=L.set, ids=ids)
        args.update(change)
        with pytest.raises(ValueError):
            lq.adapters_forward(**args)
    for change in [dict(G=X), dict(X=X[:4]), dict(t=torch.zeros(5, 4, device="cuda")),
                   dict(t=torch.zeros(5, 8, device="cuda", dtype=torch.float64)), dict(ids=ids[:2])]:
        args = dict(qw=L.qw, X=X, G=G, adapters=L.set, ids=ids)
        args.update(change)
        with pytest.raises(ValueError):
            lq.adapters_backward(**args)
    with pytest.raises(lq.LqError):        # dA needs X
        lq.adapters_backward(L.qw, None, G, L.set, ids, t=torch.zeros(5, 8, device="cuda"))
    with pytest.raises(ValueError):
        lq.AdapterSet([])
    A, B, alpha = L.adapters[0]
    for bad in [(A.float(), B, 1.0), (A, B.cpu(), 1.0), (A, B[:, :4], 1.0), (A[:, ::2], B, 1.0)]:
        with pytest.raises(ValueError):
            lq.AdapterSet([(A, B, alpha), bad])
    with pytest.raises(lq.LqError):        # ranks end at 128
        lq.AdapterSet([(torch.zeros(129, 128, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(64, 129, dtype=torch.bfloat16, device="cuda"), 1.0)])
    g = torch.zeros(8, device="cuda")
    for bad in [dict(tensors=[g.long()]), dict(tensors=[g.cpu()]), dict(tensors=[g], groups=[0, 1]),
                dict(tensors=[torch.zeros(4, 4, device="cuda").T])]:
        with pytest.raises(ValueError):
            lq.GradList(**bad)
    lst = lq.GradList([g])
    for bad in [dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=0.0),
                dict(max_norm=1.0, out=lq.GradList([g[:4]]))]:
        with pytest.raises(lq.LqError):
            lq.clip_grad_norm(lst, **bad)


def test_example(torch):
    """examples/many_adapters.py: each job learns its own change (four fifths of
    the loss gone), and the trained adapters answer single tokens."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "many_adapters.py")
    spec = importlib.util.spec_from_file_location("many_adapters", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    first, last, h, want = mod.run()
    assert all(l < 0.2 * f for f, l in zip(first, last))
    assert torch.allclose(h[-1], want[-1], rtol=1e-4, atol=1e-4)     # no adapter: the frozen projection


def test_a_route_of_another_batch_is_refused(lq, torch):
    """The last, shorter batch with a full one's route, and a route of another number of adapters."""
    L = Layer(lq, torch, 72, 128, 70, [8, 4, 16, 5])
    full = torch.zeros(128, dtype=torch.int32, device="cuda")
    own = lq.adapter_route(L.ids_dev, 4)
    for route in (lq.adapter_route(full, 4), lq.adapter_route(L.ids_dev, 6), lq.adapter_route(full[:72], 4), own.clone()):
        with pytest.raises(ValueError):
            lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, route=route)
        with pytest.raises(ValueError):
            lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, route=route)
    check_forward(lq, torch, L, route=own)
    check_backward(lq, torch, L, route=own)


def with_alpha(lq, L, a, alpha):
    """L's adapters with another alpha for adapter a."""
    return lq.AdapterSet([(A, B, alpha if i == a else al) for i, (A, B, al) in enumerate(L.adapters)])


@pytest.mark.parametrize("M", [3, 16, 50, 64, 100, 300])
@pytest.mark.parametrize("alpha", [float("inf"), -float("inf"), float("nan")])
def test_a_scale_that_is_not_finite_stays_with_its_tokens(lq, torch, M, alpha):
    L = Layer(lq, torch, 136, 128, M, [16, 8, 12], ids=np.arange(M) % 4 - 1)
    bad = with_alpha(lq, L, 1, alpha)
    mine = torch.from_numpy(L.ids == 1).cuda()
    for dt in (torch.float32, torch.bfloat16):
        H0, t0 = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=dt)
        H1, t1 = lq.adapters_forward(L.qw, L.X, bad, L.ids_dev, out_dtype=dt)
        assert torch.equal(t0, t1)                       # t is not scaled
        assert torch.equal(H0[~mine], H1[~mine])
        assert not torch.isfinite(H1[mine]).any()
    gx0, dA0, dB0 = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev)
    gx1, dA1, dB1 = lq.adapters_backward(L.qw, L.X, L.G, bad, L.ids_dev)
    assert torch.equal(gx0[~mine], gx1[~mine]) and not torch.isfinite(gx1[mine]).any()
    p0, p1 = L.set.split(dA0, dB0), bad.split(dA1, dB1)
    for a in (0, 2):
        assert torch.equal(p0[a][0], p1[a][0]) and torch.equal(p0[a][1], p1[a][1])
    assert not torch.isfinite(p1[1][0]).any() and not torch.isfinite(p1[1][1]).any()


@pytest.mark.parametrize("M", [4, 16, 50, 64, 100, 300, 4100])
def test_an_infinite_t_or_u_stays_infinite(lq, torch, M):
    """An infinity in a row of A makes t infinite there, and an infinity in a row of B makes u infinite: the
    results are infinities of the definition's sign, not NaN. One token has the adapter, so that no sum mixes signs."""
    K, N = 128, 136
    ids = np.arange(M) % 3 - 1
    ids[ids == 1] = 2
    ids[M // 2] = 1
    for which in ("t", "u"):
        L = Layer(lq, torch, N, K, M, [16, 8, 12], ids=ids)
        assert bool((L.X != 0).all()) and bool((L.G != 0).all())
        A, B, _ = L.adapters[1]
        (A if which == "t" else B)[3, 5] = float("inf")
        L.host[1] = (f64(A), f64(B), L.host[1][2])
        if which == "t":
            ref = oad.forward(L.Wd, f64(L.X), L.host, ids)
            for dt in (torch.float32, torch.bfloat16):
                H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=dt)
                assert np.isinf(ref[1][M // 2, 3]) and np.isinf(ref[0][M // 2]).all()
                assert f64(t)[M // 2, 3] == ref[1][M // 2, 3] and np.array_equal(f64(H)[M // 2], ref[0][M // 2])
                assert torch.isfinite(H[L.ids_dev != 1]).all()
            for saved in (None, t):
                _, _, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=saved)
                got, want = f64(L.set.split(torch.empty(36, K), dB)[1][1]), oad.backward(L.Wd, f64(L.X), f64(L.G), L.host, ids)[0][2][1]
                assert np.isinf(want[:, 3]).all() and np.array_equal(got[:, 3], want[:, 3])
                assert np.isfinite(np.delete(got, 3, 1)).all()
        else:
            gx, dA, _ = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev)
            rX, rA, _ = oad.backward(L.Wd, f64(L.X), f64(L.G), L.host, ids)[0]
            assert np.isinf(rX[M // 2]).all() and np.array_equal(f64(gx)[M // 2], rX[M // 2])
            assert torch.isfinite(gx[L.ids_dev != 1]).all()
            got = f64(dA[16:24])
            assert np.isinf(rA[1][5]).all() and np.array_equal(got[5], rA[1][5])
            assert np.isfinite(np.delete(got, 5, 0)).all()


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_a_finite_t_past_the_largest_bfloat16(lq, torch, M, out):
    """t = 2^128 (1 - 2^-10): a float32 value that rounds to an infinite bfloat16."""
    L = Layer(lq, torch, 72, 64, M, [8], ids=np.zeros(M, dtype=int))
    A, B, _ = L.adapters[0]
    A.zero_(), L.X.zero_(), B.fill_(2.0 ** -64)
    L.X[:, 0], A[0, 0] = (2 - 2.0 ** -7) * 2.0 ** 63, 2.0 ** 64
    L.X[:, 1], A[0, 1] = 1.5 * 2.0 ** 60, 2.0 ** 59
    L.set = lq.AdapterSet([(A, B, 8.0)])
    L.host = [(f64(A), f64(B), 1.0)]
    _, t = check_forward(lq, torch, L, out)
    assert (f64(t)[:, 0] == 2.0 ** 128 * (1 - 2.0 ** -10)).all() and torch.isinf(t[:, 0].to(torch.bfloat16)).all()


SHARES = [
    # N, K, M, ranks, ids, out: row products in column shares (tiles of 16, 32, 64 and 128 of the adapter's rows), K % 128
    (72, 1088, 4100, [16, 8, 5], "mixed", "bf16"),
    (136, 2048, 4099, [16, 16, 3], "runs", "f32"),
    (200, 1536, 2049, [32, 7], "runs", "bf16"),
    (64, 4160, 1031, [64, 24, 9], "mixed", "f32"),
    (80, 1024, 515, [128, 1], "runs", "f32"),
    # tiles of 256 x 256 with more steps of the contraction than the loads run ahead; K % 64 == 0, begun at an eighth per XCD
    (8184, 1024, 4001, [16, 40, 7], "mixed", "bf16"),
    (8184, 1024, 4001, [16, 40, 7], "mixed", "f32"),
    (8192, 576, 4096, [64], "runs", "bf16"),
    # tiles of 256 x 128 likewise
    # tiles of 256 x 128 likewise, N % 4
    (4090, 1088, 2047, [16, 8, 64, 24], "runs", "bf16"),
    (4090, 1088, 2047, [16, 8, 64, 24], "mixed", "f32"),
]


@pytest.mark.parametrize("case", SHARES, ids=str)
def test_forward_long_contraction(lq, torch, case):
    N, K, M, ranks, ids, out = case
    L = Layer(lq, torch, N, K, M, ranks, ids)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    H, t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=dt)
    (ref, mag, lora), _, _, _ = reference64(torch, L)
    bound = (K + 3 * max(ranks) + 8) * U * (mag + lora) + K * U * lora
    if out == "bf16":
        bound += 2.0 ** -16 * lora + 2.0 ** -8 * ref.abs() + 2.0 ** -130
    assert ((H.double() - ref).abs() <= bound).all()
    X = L.X.double()
    for a, (A, _, _) in enumerate(L.adapters):
        m, r = (L.ids_dev == a).nonzero()[:, 0], A.shape[0]
        want, tmag = X[m] @ A.double().T, X[m].abs() @ A.double().abs().T
        assert ((t[m, :r].double() - want).abs() <= (K + 8) * U * tmag).all()
        assert not t[m, r:].any()
    assert not t[L.ids_dev < 0].any()
    again = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev, out_dtype=dt)
    assert torch.equal(again[0], H) and torch.equal(again[1], t)


@pytest.mark.parametrize("case", [
    # N, K, M, ranks, ids, weight: u and t in column shares of their own lengths
    (1024, 1088, 2051, [32, 16, 7], "runs", "nf4_dq"),
    (2056, 1024, 4100, [16, 5], "mixed", "nf4_f32"),
    (1032, 3136, 1033, [64, 24], "runs", "codebook"),
    (1024, 8192, 4001, [16, 40], "mixed", "nf4_dq"),      # tiles of 256 x 256, begun at an eighth per XCD
], ids=str)
@pytest.mark.parametrize("saved", [False, True])
def test_backward_long_contraction(lq, torch, case, saved):
    N, K, M, ranks, ids, weight = case
    L = Layer(lq, torch, N, K, M, ranks, ids, weight)
    t = lq.adapters_forward(L.qw, L.X, L.set, L.ids_dev)[1] if saved else None
    gx, dA, dB = lq.adapters_backward(L.qw, L.X, L.G, L.set, L.ids_dev, t=t)
    _, (ref, mag, lora), rA, rB = reference64(torch, L, t)
    bound = (N + 3 * max(ranks) + 8) * U * (mag + lora) + N * U * lora + 2.0 ** -16 * lora + 2.0 ** -8 * ref.abs()
    assert ((gx.double() - ref).abs() <= bound + 2.0 ** -130).all()
    for a, (da, db) in enumerate(L.set.split(dA, dB)):
        tokens = int((L.ids == a).sum())
        assert ((da.double() - rA[a][0]).abs() <= (3 * tokens + N + 16) * U * rA[a][1]).all()
        assert ((db.double() - rB[a][0]).abs() <= (3 * tokens + (0 if saved else K) + 16) * U * rB[a][1]).all()
