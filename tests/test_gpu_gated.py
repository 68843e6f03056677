"""GPU parity of the gated pair against the formulas in float64.

Tolerances are derived element by element. A projection's float32 value is off
by the bounds of test_gpu_adapters.py (n 2^-24 of the sum of its terms' absolute
values; two bfloat16 terms of t where H is bfloat16: 2^-16 of the adapters'
part). act' is at most 1.13 in size, so act(g) u is off by 1.13 |u| of g's error
and |act(g)| of u's, and by act's own: e^-x is raised from a product rounded at
|x| 2^-24 (and the gelus' arguments likewise), the hardware's exponential and
reciprocal are good to an ulp. dg and du are products of three or two such
values; grad_X's product takes them rounded to bfloat16, 2^-8 of each term; a
bfloat16 result adds 2^-8 of the value.
"""
import numpy as np
import pytest

from oracle import dropout as odr
from oracle import gated as og
from test_gpu_adapters import U, f64, make_weight

pytestmark = pytest.mark.gpu
SEED, STEP, SITES = 0x123456789ABCDEF0, 0xEEDDCCBBAA998877, (40, 41)


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


class Layer:
    """Inputs of one case. ranks: of the gate's adapters; up's are those reversed."""

    def __init__(self, lq, torch, N, K, M, ranks, ids="mixed", weight="nf4_dq", act="silu", p=0.0, base=0.15, seed=0):
        rng = np.random.default_rng([seed, N, K, M, len(ranks)])
        bf = lambda shape, std=1.0: torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).cuda().to(
            torch.bfloat16)
        self.torch, self.N, self.K, self.M, self.act, n = torch, N, K, M, act, len(ranks)
        weights = weight.split("+")
        self.qw = [make_weight(lq, torch, rng, N, K, weights[i % len(weights)]) for i in range(2)]
        self.W = [lq.dequant(q).double() for q in self.qw]
        self.X, self.G = bf((M, K)), bf((M, N))
        self.g, self.u = bf((M, N), 1.5), bf((M, N), 1.5)
        self.ids = self.set = None
        if n:
            self.adapters = [[(bf((r, K), 0.05), bf((N, r), 0.05), float(rng.uniform(0.5, 3.0) * r)) for r in rs]
                             for rs in (ranks, ranks[::-1])]
            self.set = [lq.AdapterSet(a) for a in self.adapters]
            if isinstance(ids, str) and ids == "mixed":
                host = rng.integers(0, n, M)
                host[rng.random(M) < base] = -1
            elif isinstance(ids, str):
                cuts = np.sort(rng.integers(0, M + 1, n - 1))
                host = np.repeat(rng.permutation(n), np.diff(np.concatenate([[0], cuts, [M]])))
            else:
                host = np.asarray(ids)
            self.ids = torch.from_numpy(host.astype(np.int32)).cuda()
        self.pair = lq.GatedPair(*self.qw, *(self.set or ()), act=act)
        self.drops, self.keep = None, [None, None]
        if p:
            key = lq.dropout_key(SEED, STEP)
            self.drops = tuple(lq.Dropout(p, key, s) for s in SITES)
            for i in range(2):
                mask, factor = odr.kept(SEED, STEP, SITES[i], p, (M, K))
                self.keep[i] = torch.from_numpy(mask).cuda().double() * factor

    def input(self, i):
        X = self.X.double()
        return X if self.keep[i] is None else self.torch.where(self.keep[i] > 0, X, 0.0) * self.keep[i]

    def groups(self, i):
        """(A, B, scale, tokens) of side i's adapters."""
        for a, (A, B, alpha) in enumerate(self.adapters[i] if self.set else ()):
            yield A.double(), B.double(), float(np.float32(alpha / A.shape[0])), (self.ids == a).nonzero()[:, 0]

    def r(self, i):
        return self.set[i].r_max if self.set else 0


def acts(torch, x, kind):
    """act, act', and how far float32 may be off in each."""
    v, s = (torch.from_numpy(a).cuda() for a in og.act(x.cpu().numpy(), kind))
    ax = x.abs()
    # the relative error of the factor that x is multiplied by, in units of 2^-23
    k = {"silu": ax + 8, "gelu": x * x + 16, "gelu_tanh": 8 * (1.6 * ax + 0.08 * ax ** 3) + 8}[kind]
    lever = {"silu": 1 + ax, "gelu": 1 + ax, "gelu_tanh": 1 + 1.6 * ax * (1 + 0.14 * x * x)}[kind]
    return v, s, v.abs() * k * 2.0 ** -23 + 2.0 ** -120, k * lever * 2.0 ** -22


def inside(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(((got.double() - ref).abs() / bound).max())}"


def project(L, i):
    """(value, sum of the base's and of the adapters' absolute terms, t, its absolute sum)."""
    t_ = L.torch
    X, D = L.X.double(), L.input(i)
    H, mag = X @ L.W[i].T, X.abs() @ L.W[i].abs().T
    lora = t_.zeros_like(H)
    T, mT = (t_.zeros(L.M, L.r(i), dtype=t_.float64, device="cuda") for _ in range(2))
    for A, B, s, m in L.groups(i):
        ta, tm = D[m] @ A.T, D[m].abs() @ A.abs().T
        T[m, :A.shape[0]], mT[m, :A.shape[0]] = ta, tm
        H[m] += s * ta @ B.T
        lora[m] = s * tm @ B.abs().T
    return H, mag, lora, T, mT


def check_forward(lq, torch, L, out="bf16", route=None, save=True):
    dt = torch.float32 if out == "f32" else torch.bfloat16
    H, saved = lq.gated_forward(L.pair, L.X, L.ids, out_dtype=dt, save=save, route=route, dropout=L.drops)
    value, err = [], []
    for i in range(2):
        v, mag, lora, T, mT = project(L, i)
        e = (L.K + 3 * L.r(i) + 8) * U * (mag + lora) + (L.K + 2) * U * lora
        if out == "bf16":
            e += 2.0 ** -16 * lora
        value.append(v)
        err.append(e)
        if save:
            inside(saved[i], v, e + 2.0 ** -8 * v.abs() + 2.0 ** -130, "gu"[i])
            if L.set:
                inside(saved[2 + i], T, (L.K + 10) * U * mT, f"t {i}")
            else:
                assert saved[2 + i] is None
    a, _, ea, _ = acts(torch, value[0], L.act)
    ref = a * value[1]
    # (act's own error is taken at the exact g: 2 of it covers the computed one, whose error is small against 1)
    bound = (1.13 * err[0] + 2 * ea) * (value[1].abs() + err[1]) + a.abs() * err[1] + 2 * U * ref.abs()
    if out == "bf16":
        bound += 2.0 ** -8 * ref.abs() + 2.0 ** -8 * bound + 2.0 ** -130
    inside(H, ref, bound, "H")
    return H, saved


def check_backward(lq, torch, L, saved_t=True, route=None):
    ts = [None, None]
    if saved_t and L.set:
        s = lq.gated_forward(L.pair, L.X, L.ids, dropout=L.drops)[1]
        ts = [s.t_gate, s.t_up]
    got = lq.gated_backward(L.pair, L.X, L.G, L.ids, lq.GatedSaved(L.g, L.u, *ts), route=route, dropout=L.drops)
    G, g, u = L.G.double(), L.g.double(), L.u.double()
    a, slope, ea, es = acts(torch, g, L.act)
    d = (G * u * slope, G * a)
    e = ((G * u).abs() * es + 3 * U * d[0].abs() + 2.0 ** -130, G.abs() * ea + 2 * U * d[1].abs() + 2.0 ** -130)
    rX = torch.zeros(L.M, L.K, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(rX)
    for i in range(2):
        W, n, r = L.W[i], 2 * L.N, L.r(i)
        rX += d[i] @ W
        mag = d[i].abs() @ W.abs()
        bound += (n + 8) * U * mag + 2.0 ** -8 * mag + 1.01 * e[i] @ W.abs()
        keep = L.keep[i] if L.keep[i] is not None else 1.0
        D = L.input(i)
        lora, elora = torch.zeros_like(rX), torch.zeros_like(rX)
        parts = L.set[i].split(got[1 + 2 * i], got[2 + 2 * i]) if L.set else []
        for k, (A, B, s, m) in enumerate(L.groups(i)):
            um, ue = d[i][m].abs() @ B.abs(), e[i][m] @ B.abs()
            uv = d[i][m] @ B
            add = torch.zeros_like(rX)
            add[m] = s * uv @ A
            rX += add * keep
            lora[m], elora[m] = s * um @ A.abs(), s * ue @ A.abs()
            tokens = m.numel()
            ref, mA = s * uv.T @ D[m], s * um.T @ D[m].abs()
            inside(parts[k][0], ref, (3 * tokens + L.N + 18) * U * mA + 1.01 * s * ue.T @ D[m].abs(), f"dA {i} {k}")
            tv = D[m] @ A.T if ts[i] is None else ts[i][m, :A.shape[0]].double()
            tm = D[m].abs() @ A.abs().T if ts[i] is None else tv.abs()
            ref, mB = s * d[i][m].T @ tv, s * d[i][m].abs().T @ tm
            inside(parts[k][1], ref, (6 * tokens + (0 if ts[i] is not None else L.K + 2) + 32) * U * mB + 1.01 * s * e[i][m].T @ tm,
                   f"dB {i} {k}")
        bound += ((L.N + 3 * r + n + 8) * U * lora + 2.0 ** -16 * lora + 1.01 * elora) * keep
    inside(got.grad_X, rX, bound + 2.0 ** -8 * (rX.abs() + bound) + 2.0 ** -130, "grad_X")
    return got


CASES = [
    # N, K, M, ranks, ids, weight, act, p
    (64, 64, 1, [8], "mixed", "nf4_dq", "silu", 0.0),
    (80, 128, 1, [16, 4], "mixed", "nf4_f32", "gelu", 0.0),
    (256, 512, 16, [16] * 16, "mixed", "nf4_dq", "silu", 0.0),
    (264, 320, 33, [4, 7, 16, 33, 64], "mixed", "nf4_dq", "gelu_tanh", 0.0),
    (512, 1024, 64, [8, 16, 32], "mixed", "nf4_dq", "silu", 0.0),
    (104, 192, 64, [1, 128], "mixed", "nf4_f32+nf4_dq", "silu", 0.0),
    (64, 128, 7, [], None, "nf4_dq", "silu", 0.0),
    (72, 128, 20, [16, 4, 1], "mixed", "nf4_dq", "silu", 0.3),
    (4168, 192, 64, [128] * 64, "mixed", "nf4_dq", "silu", 0.0),
    (8208, 64, 30, [7, 16], "mixed", "nf4_f32", "gelu", 0.0),
    (16, 16448, 5, [8, 40], "mixed", "nf4_dq", "gelu_tanh", 0.0),
    (72, 192, 65, [5, 24], "runs", "nf4_dq", "silu", 0.1),
    (72, 192, 65, [5, 24], "runs", "codebook", "gelu", 0.5),
    (512, 256, 300, [16, 8, 64, 1, 7], "runs", "nf4_dq", "silu", 0.0),
    (304, 448, 517, [12, 40], "mixed", "codebook+nf4_f32", "gelu_tanh", 0.05),
    (1000, 320, 700, [64, 64, 64], "runs", "nf4_dq", "silu", 0.1),
    (256, 256, 129, [16] * 40, "mixed", "codebook", "gelu", 0.0),
    (128, 64, 1025, [128, 3], "runs", "nf4_dq", "silu", 0.2),
    (200, 256, 333, [], None, "codebook", "gelu_tanh", 0.0),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_forward(lq, torch, case, out):
    check_forward(lq, torch, Layer(lq, torch, *case), out)


@pytest.mark.parametrize("N", [77, 66, 101])
@pytest.mark.parametrize("M", [5, 70, 300])
def test_forward_odd_widths(lq, torch, N, M):
    for out in ("bf16", "f32"):
        check_forward(lq, torch, Layer(lq, torch, N, 192, M, [8, 3], act="gelu"), out)


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("saved_t", [True, False])
def test_backward(lq, torch, case, saved_t):
    check_backward(lq, torch, Layer(lq, torch, *case), saved_t)


LARGE = [
    # forward tiles of 256 x 64 and 256 x 128 outputs, small ones above the CUs' count; backward tiles over [M, K]
    (2056, 64, 2047, [16, 8, 64, 24], "runs", "nf4_dq", "silu", 0.1),
    (2050, 128, 1800, [16] * 9, "mixed", "nf4_f32", "gelu", 0.0),
    (4096, 64, 4001, [64, 16, 128], "runs", "nf4_dq", "gelu_tanh", 0.0),
    (4096, 64, 4096, [32, 7, 16, 8], "mixed", "nf4_dq", "silu", 0.3),
    (520, 192, 1999, [3, 64] * 20, "mixed", "nf4_dq", "silu", 0.0),
    (1096, 128, 2048, [], None, "nf4_dq", "silu", 0.0),
    (72, 4096, 2047, [16, 8, 64, 24], "runs", "nf4_dq", "silu", 0.1),
    (64, 4096, 1800, [16] * 9, "mixed", "codebook", "gelu", 0.0),
    (136, 8192, 4001, [64, 16, 128], "runs", "nf4_dq", "silu", 0.05),
    (64, 8192, 4096, [32, 7, 16, 8], "mixed", "nf4_f32", "gelu_tanh", 0.0),
    (200, 1088, 1999, [3, 64] * 20, "mixed", "nf4_dq", "silu", 0.2),
]


@pytest.mark.parametrize("case", LARGE, ids=str)
def test_large(lq, torch, case):
    L = Layer(lq, torch, *case)
    check_forward(lq, torch, L, "bf16")
    check_forward(lq, torch, L, "f32", save=False)
    if L.N % 8 == 0:
        check_backward(lq, torch, L, saved_t=False)


@pytest.mark.parametrize("case", [
    # grad_X in 64 x 64 tiles above the CUs' count; the forward in 256 x 64 outputs
    (200, 1088, 1500, [3, 64] * 20, "mixed", "nf4_dq", "silu", 0.0),
    (1608, 1088, 1500, [16, 64], "runs", "codebook", "gelu", 0.2),
], ids=str)
def test_more_small_tiles_than_compute_units(lq, torch, case):
    test_large(lq, torch, case)


@pytest.mark.parametrize("M", [3, 64, 70, 300, 2048])
def test_no_token_has_an_adapter(lq, torch, M):
    """Every id outside the set: the result without sets, zero t, zero gradients."""
    N = 2048 if M == 2048 else 128
    L = Layer(lq, torch, N, 128, M, [16, 8], ids=np.full(M, 7), p=0.2 if M > 64 else 0.0)
    H, saved = check_forward(lq, torch, L)
    assert not saved.t_gate.any() and not saved.t_up.any()
    got = check_backward(lq, torch, L)
    assert not any(x.any() for x in got[1:])
    bare = lq.GatedPair(*L.qw, act="silu")
    assert torch.equal(lq.gated_forward(bare, L.X)[0], H)
    assert torch.equal(lq.gated_backward(bare, None, L.G, None, lq.GatedSaved(L.g, L.u)).grad_X, got.grad_X)


@pytest.mark.parametrize("M", [3, 16, 64, 100, 300])
def test_an_adapters_infinities_stay_with_its_tokens(lq, torch, M):
    L = Layer(lq, torch, 136, 128, M, [16, 8, 12], base=0.2, seed=3)
    kept = lq.GatedSaved(L.g, L.u)

    def step():
        H, s = lq.gated_forward(L.pair, L.X, L.ids, out_dtype=torch.float32)
        return H, s, lq.gated_backward(L.pair, L.X, L.G, L.ids, kept)
    H0, s0, b0 = step()
    A, B, _ = L.adapters[0][1]
    A[3, 7] = float("nan")
    L.adapters[1][1][1][5, 2] = float("inf")
    bad = int((L.ids != 0).nonzero()[0, 0])
    L.X[bad, 3] = float("nan")
    L.G[bad, 9] = float("inf")
    H1, s1, b1 = step()
    clean = (L.ids != 1) & (torch.arange(M, device="cuda") != bad)
    assert clean.any()
    for a, b in ((H0, H1), *zip(s0, s1), (b0.grad_X, b1.grad_X)):
        assert torch.equal(a[clean], b[clean])
    for i in range(2):
        p0, p1 = (L.set[i].split(*b[1 + 2 * i:3 + 2 * i]) for b in (b0, b1))
        for a in (0, 2):
            if a != int(L.ids[bad]):
                assert torch.equal(p0[a][0], p1[a][0]) and torch.equal(p0[a][1], p1[a][1])


def test_a_side_that_is_infinite(lq, torch):
    """An infinite t of up's leaves g as it was, whatever tiles and steps the two sides share."""
    for M in (16, 70, 300, 2048):
        L = Layer(lq, torch, 2048 if M == 2048 else 128, 128, M, [16], ids=np.zeros(M), seed=4)
        s0 = lq.gated_forward(L.pair, L.X, L.ids)[1]
        L.adapters[1][0][0].fill_(float("inf"))
        s1 = lq.gated_forward(L.pair, L.X, L.ids)[1]
        assert torch.equal(s0.g, s1.g) and not torch.isfinite(s1.u).any()


def test_extreme_activations(lq, torch):
    """Large |g|, zeros and infinities in g, u and G: what the formulas give in float32."""
    L = Layer(lq, torch, 64, 64, 40, [8], seed=6)
    L.g[:] = torch.linspace(-120, 120, 64, device="cuda").to(torch.bfloat16)
    for kind in ("silu", "gelu", "gelu_tanh"):
        L.act, L.pair = kind, lq.GatedPair(*L.qw, *L.set, act=kind)
        check_backward(lq, torch, L, saved_t=False)
    L.G[3, 5] = 0.0
    L.g[7, 9], L.u[8, 9], L.G[9, 9] = float("inf"), float("inf"), float("nan")
    for kind in ("silu", "gelu", "gelu_tanh"):
        pair = lq.GatedPair(*L.qw, act=kind)
        gx = lq.gated_backward(pair, None, L.G, None, lq.GatedSaved(L.g, L.u)).grad_X
        bad = ~torch.isfinite(gx).all(1)
        assert bad[7:10].all() and not bad[:7].any() and not bad[10:].any()


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_slopes_of_large_finite_values(lq, torch, kind):
    """Past |g| = 100 act' is 1 or 0 to the last bit of float32, up to the largest finite g: up's weight and its adapter
    are zero, so that grad_X and the gate's gradients are those of dg = G u act'(g) alone."""
    sizes = [100.0, 1e4, 1e12, 1e13, 2e13, 1e15, 1e18, 1.8e19, 1e25, 3e38]
    values = [v * sign for v in sizes for sign in (1.0, -1.0)]
    N, K, r = 72, 64, 8
    L = Layer(lq, torch, N, K, len(values), [r], ids=np.zeros(len(values)), act=kind, seed=7)
    up = lq.QWeight.from_weight(torch.zeros(N, K, device="cuda"), double_quantize=False)
    assert not lq.dequant(up).any()
    L.adapters[1][0][1].zero_()
    pair = lq.GatedPair(L.qw[0], up, *L.set, act=kind)
    g = torch.tensor(values, device="cuda")[:, None].expand(-1, N).to(torch.bfloat16).contiguous()
    L.G.div_(8)      # exact; du = G act(3e38) stays below float32's largest (an infinity times up's zeros is NaN)
    assert float(L.G.abs().max()) < 1
    got = lq.gated_backward(pair, L.X, L.G, L.ids, lq.GatedSaved(g, L.u))
    A, B, s, m = next(L.groups(0))
    d = L.G.double() * L.u.double() * (g > 0)      # a product of two bfloat16 values is a float32
    t, X = L.X.double() @ A.T, L.X.double()
    rX = d @ L.W[0] + s * (d @ B) @ A
    mag, lora = d.abs() @ L.W[0].abs(), s * (d.abs() @ B.abs()) @ A.abs()
    bound = (2 * N + 8) * U * mag + 2.0 ** -8 * mag + (3 * N + 3 * r + 8) * U * lora + 2.0 ** -16 * lora
    inside(got.grad_X, rX, bound + 2.0 ** -8 * (rX.abs() + bound) + 2.0 ** -130, "grad_X")
    (dA, dB), = L.set[0].split(got.dA_gate, got.dB_gate)
    M = len(values)
    inside(dA, s * (d @ B).T @ X, (3 * M + N + 18) * U * s * (d.abs() @ B.abs()).T @ X.abs() + 2.0 ** -130, "dA")
    inside(dB, s * d.T @ t, (6 * M + K + 34) * U * s * d.abs().T @ (X.abs() @ A.abs().T) + 2.0 ** -130, "dB")


DECODE_FORMS = [
    # N, K, M, ranks: every form of the projection by row groups, token tiles and waves; N % 4, odd K / 64, rows of
    # a multiple of 64 blocks, ranks % 8
    (4112, 192, 1, [16, 40]),            # flat, one token tile
    (4117, 320, 16, [16, 7, 40]),
    (5000, 1024, 9, [3, 16]),
    (4112, 256, 30, [7, 16]),            # flat, two
    (8206, 64, 17, [24, 8, 128]),
    (264, 192, 20, [8, 33]),             # two row groups, eight waves
    (250, 128, 32, [16] * 20),
    (16400, 128, 5, [16, 24]),           # flat in two rounds
    (16390, 4096, 3, [16, 7]),
    (12310, 128, 5, [16, 24]),           # four row groups, four waves
    (14336, 4096, 3, [16, 7]),
    (16400, 192, 30, [16, 24, 1]),
    (16400, 4096, 20, [8, 33]),
    (4168, 192, 64, [8, 16, 32]),        # ... of four token tiles
    (4166, 4096, 40, [24, 5]),
    (4168, 320, 50, [64, 9, 64]),        # ... eight waves, where t leaves no room for two workgroups
    (4168, 4096, 64, [64, 40] * 8),
]


@pytest.mark.parametrize("case", DECODE_FORMS, ids=str)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("weight", ["nf4_dq", "nf4_f32"])
def test_decode_forms(lq, torch, case, out, weight):
    L = Layer(lq, torch, *case, weight=weight, act=("silu", "gelu", "gelu_tanh")[case[2] % 3], seed=8)
    H, saved = check_forward(lq, torch, L, out)
    again = lq.gated_forward(L.pair, L.X, L.ids, out_dtype=H.dtype)
    assert torch.equal(H, again[0]) and all(torch.equal(a, b) for a, b in zip(saved, again[1]))
    assert torch.equal(H, lq.gated_forward(L.pair, L.X, L.ids, out_dtype=H.dtype, save=False)[0])


def test_partial_outputs(lq, torch):
    L = Layer(lq, torch, 136, 192, 150, [16, 8], p=0.1)
    kept = lq.GatedSaved(L.g, L.u)
    full = lq.gated_backward(L.pair, L.X, L.G, L.ids, kept, dropout=L.drops)
    for need in ([True, False, False], [False, True, False], [False, False, True]):
        got = lq.gated_backward(L.pair, L.X, L.G, L.ids, kept, *need, dropout=L.drops)
        for i, x in enumerate(got):
            wanted = need[0] if i == 0 else need[1] if i % 2 else need[2]
            assert (x is None) == (not wanted) and (x is None or torch.equal(x, full[i]))
    s = lq.gated_forward(L.pair, L.X, L.ids, dropout=L.drops)[1]
    got = lq.gated_backward(L.pair, None, L.G, L.ids, s._replace(g=L.g, u=L.u), need_dA=False, dropout=L.drops)
    assert torch.equal(got.grad_X, full.grad_X) and got.dB_up is not None


def test_one_side_drops(lq, torch):
    """A dropout on one side alone: the other side's t and gradients are those without any."""
    for M in (70, 300):
        L = Layer(lq, torch, 136, 192, M, [16, 8])
        kept = lq.GatedSaved(L.g, L.u)
        d = lq.Dropout(0.5, lq.dropout_key(1), 3)
        s0 = lq.gated_forward(L.pair, L.X, L.ids)[1]
        b0 = lq.gated_backward(L.pair, L.X, L.G, L.ids, kept)
        for drops, other in (((d, None), 1), ((None, d), 0)):
            s1 = lq.gated_forward(L.pair, L.X, L.ids, dropout=drops)[1]
            b1 = lq.gated_backward(L.pair, L.X, L.G, L.ids, kept, dropout=drops)
            assert torch.equal(s0[2 + other], s1[2 + other]) and not torch.equal(s0[3 - other], s1[3 - other])
            assert torch.equal(b0[1 + 2 * other], b1[1 + 2 * other]) and torch.equal(b0[2 + 2 * other], b1[2 + 2 * other])


def test_route_repeats_and_streams(lq, torch):
    for M in (40, 333):
        L = Layer(lq, torch, 264, 320, M, [16, 8, 40], p=0.1)
        route = lq.adapter_route(L.ids, 3)
        runs = []
        torch.cuda.synchronize()
        for r, stream in ((None, torch.cuda.current_stream()), (route, torch.cuda.Stream())):
            with torch.cuda.stream(stream):
                H, s = lq.gated_forward(L.pair, L.X, L.ids, route=r, dropout=L.drops)
                b = lq.gated_backward(L.pair, L.X, L.G, L.ids, s, route=r, dropout=L.drops)
            stream.synchronize()
            runs.append((H, *s, *b))
        assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_graph(lq, torch):
    """Forward and backward captured, replayed on new tokens: each replay is the eager result."""
    for M in (16, 300):
        L = Layer(lq, torch, 264, 320, M, [16, 40], p=0.2 if M > 64 else 0.0)

        def step():
            H, s = lq.gated_forward(L.pair, L.X, L.ids, dropout=L.drops)
            return (H, *s, *lq.gated_backward(L.pair, L.X, L.G, L.ids, s, dropout=L.drops))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        for _ in range(3):
            L.X.copy_(torch.randn_like(L.X))
            L.G.copy_(torch.randn_like(L.G))
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            assert all(torch.equal(a, b) for a, b in zip(got, step()))
            torch.cuda.synchronize()


def test_two_captured_graphs_keep_their_own_workspaces(lq, torch):
    L = Layer(lq, torch, 136, 192, 100, [16, 8])
    outs, graphs = [], []
    for _ in range(2):
        lq.gated_forward(L.pair, L.X, L.ids)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(lq.gated_forward(L.pair, L.X, L.ids)[0])
        graphs.append(graph)
    want = lq.gated_forward(L.pair, L.X, L.ids)[0]
    for _ in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_gradients_against_differences(lq, torch):
    """d/d eps of sum(H R) along directions of X, A and B by central differences in float64 of the formulas; the
    kernels' gradients, from the exact g and u rounded to bfloat16, give the same number."""
    L = Layer(lq, torch, 64, 128, 90, [8, 16], act="gelu_tanh", p=0.25, seed=2)
    G = L.G.double()
    saved = lq.gated_forward(L.pair, L.X, L.ids, dropout=L.drops)[1]
    got = lq.gated_backward(L.pair, L.X, L.G, L.ids, saved, dropout=L.drops)
    rng = np.random.default_rng(3)
    rand = lambda x: torch.from_numpy(rng.standard_normal(tuple(x.shape))).cuda()
    VX = rand(L.X)
    VA = [[rand(A) for A, _, _ in L.adapters[i]] for i in range(2)]
    VB = [[rand(B) for _, B, _ in L.adapters[i]] for i in range(2)]

    def loss(ex=0.0, ea=(0.0, 0.0), eb=(0.0, 0.0)):
        v = []
        for i in range(2):
            X = L.X.double() + ex * VX
            H = X @ L.W[i].T
            for k, (A, B, s, m) in enumerate(L.groups(i)):
                H[m] += s * ((X * L.keep[i])[m] @ (A + ea[i] * VA[i][k]).T) @ (B + eb[i] * VB[i][k]).T
            v.append(H)
        return float((torch.from_numpy(og.act(v[0].cpu().numpy(), L.act)[0]).cuda() * v[1] * G).sum())
    h = 1e-4

    def close(grads, dirs, plus, minus, what):
        value = sum(float((a.double() * b).sum()) for a, b in zip(grads, dirs))
        scale = sum(float((a.double() * b).square().sum()) for a, b in zip(grads, dirs)) ** 0.5
        # g and u are rounded to bfloat16 (2^-8 of each, of random sign), grad_X too: the errors of the terms of the
        # sum are independent and each a few 2^-8 of its term, so sixteen 2^-8 of the root of the sum of squares
        assert abs(value - (plus - minus) / (2 * h)) <= 16 * 2.0 ** -8 * scale + 1e-6 * abs(value), what
    close([got.grad_X], [VX], loss(ex=h), loss(ex=-h), "X")
    for i in range(2):
        e = lambda x: (x, 0.0) if i == 0 else (0.0, x)
        parts = L.set[i].split(got[1 + 2 * i], got[2 + 2 * i])
        close([a for a, _ in parts], VA[i], loss(ea=e(h)), loss(ea=e(-h)), f"A {i}")
        close([b for _, b in parts], VB[i], loss(eb=e(h)), loss(eb=e(-h)), f"B {i}")


@pytest.mark.parametrize("M", [16, 100, 300, 2048])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -3e38])
def test_padding_of_any_value(lq, torch, M, what):
    """Rows without an adapter (a padded batch's) may hold anything: every other row and all gradients of the
    adapters are bit for bit those of zero rows. So may one adapter's tokens: the other adapters' are."""
    N = 1024 if M == 2048 else 136
    L = Layer(lq, torch, N, 192, M, [16, 8, 40], ids="mixed", base=0.3, p=0.2 if M > 64 else 0.0)
    for who in (-1, 1):
        bad = L.ids == who
        assert bad.any() and not bad.all()
        runs = []
        for v in (0.0, what):
            X, G, g, u = (torch.where(bad[:, None], v, x.float()).to(torch.bfloat16) for x in (L.X, L.G, L.g, L.u))
            H, s = lq.gated_forward(L.pair, X, L.ids, dropout=L.drops)
            b = lq.gated_backward(L.pair, X, G, L.ids, lq.GatedSaved(g, u), dropout=L.drops)
            runs.append((H, s, b))
        (H0, s0, b0), (H1, s1, b1) = runs
        for a, c in ((H0, H1), *zip(s0, s1), (b0.grad_X, b1.grad_X)):
            assert torch.equal(a[~bad], c[~bad])
        for i in range(2):
            for k, (x, y) in enumerate(zip(L.set[i].split(b0[1 + 2 * i], b0[2 + 2 * i]), L.set[i].split(b1[1 + 2 * i], b1[2 + 2 * i]))):
                assert k == who or (torch.equal(x[0], y[0]) and torch.equal(x[1], y[1]))


def test_both_sides_alike(lq, torch):
    """One weight, one set and one dropout on both sides: what copies of them give."""
    for M in (20, 300):
        L = Layer(lq, torch, 136, 192, M, [16, 8], p=0.2 if M > 64 else 0.0)
        q, st = L.qw[0], L.set[0]
        drops = L.drops and (L.drops[0], L.drops[0])
        copies = [lq.AdapterSet([(A.clone(), B.clone(), a) for A, B, a in L.adapters[0]]) for _ in range(2)]
        runs = []
        for sets in ((st, st), copies):
            pair = lq.GatedPair(q, q, *sets)
            H, s = lq.gated_forward(pair, L.X, L.ids, dropout=drops)
            runs.append((H, *s, *lq.gated_backward(pair, L.X, L.G, L.ids, s, dropout=drops)))
        assert all(torch.equal(a, b) for a, b in zip(*runs))
        assert torch.equal(runs[0][1], runs[0][2]) and torch.equal(runs[0][3], runs[0][4])


def test_outputs_past_32_bits(lq, torch):
    """M N past 2^31 elements: rows at the end against the formulas, and the adapters' gradients over all rows."""
    N, K, r = 65600, 64, 4
    M = (1 << 31) // N + 300
    L = Layer(lq, torch, N, K, 24, [r], ids=np.zeros(24, dtype=np.int64))
    small = L.M
    X = torch.randn(M, K, dtype=torch.bfloat16, device="cuda")
    G = torch.randn(M, N, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    X[M - small:], G[M - small:] = L.X, L.G
    H, saved = lq.gated_forward(L.pair, X, ids)
    got = lq.gated_backward(L.pair, X, G, ids, saved)
    value, err = [], []
    for i in range(2):
        v, mag, lora, T, mT = project(L, i)
        e = (K + 3 * r + 8) * U * (mag + lora) + (K + 2) * U * lora + 2.0 ** -16 * lora
        inside(saved[i][M - small:], v, e + 2.0 ** -8 * v.abs() + 2.0 ** -130, "gu"[i])
        inside(saved[2 + i][M - small:], T, (K + 10) * U * mT, f"t {i}")
        value.append(v)
        err.append(e)
    a, _, ea, _ = acts(torch, value[0], L.act)
    ref = a * value[1]
    bound = (1.13 * err[0] + 2 * ea) * (value[1].abs() + err[1]) + a.abs() * err[1] + 2 * U * ref.abs()
    inside(H[M - small:], ref, bound + 2.0 ** -8 * ref.abs() + 2.0 ** -8 * bound + 2.0 ** -130, "H")
    dA = [torch.zeros(r, K, dtype=torch.float64, device="cuda") for _ in range(2)]
    mA, dB, mB = [d.clone() for d in dA], [], []
    for i in range(2):
        dB.append(torch.zeros(N, r, dtype=torch.float64, device="cuda"))
        mB.append(dB[i].clone())
    for m in range(0, M, 1024):
        sl = slice(m, min(m + 1024, M))
        g, u, Gd = saved.g[sl].double(), saved.u[sl].double(), G[sl].double()
        sig = torch.sigmoid(g)      # silu and the errors of acts(), on the device
        act, slope, k = g * sig, sig + g * sig * torch.sigmoid(-g), g.abs() + 8
        ea, es = act.abs() * k * 2.0 ** -23 + 2.0 ** -120, k * (1 + g.abs()) * 2.0 ** -22
        d = (Gd * u * slope, Gd * act)
        e = ((Gd * u).abs() * es + 3 * U * d[0].abs() + 2.0 ** -130, Gd.abs() * ea + 2 * U * d[1].abs() + 2.0 ** -130)
        rX = bX = 0.0
        for i in range(2):
            A, B, s, _ = next(L.groups(i))
            um, ue = d[i].abs() @ B.abs(), e[i] @ B.abs()
            dA[i] += s * (d[i] @ B).T @ X[sl].double()
            mA[i] += ((3 * M + N + 18) * U * s * um.T + 1.01 * s * ue.T) @ X[sl].double().abs()
            t = saved[2 + i][sl].double()
            dB[i] += s * d[i].T @ t
            mB[i] += ((6 * M + 32) * U * s * d[i].abs().T + 1.01 * s * e[i].T) @ t.abs()
            mag, lora = d[i].abs() @ L.W[i].abs(), s * um @ A.abs()
            rX = rX + d[i] @ L.W[i] + s * (d[i] @ B) @ A
            bX = bX + ((2 * N + 8) * U * mag + 2.0 ** -8 * mag + 1.01 * e[i] @ L.W[i].abs() +
                       (3 * N + 3 * r + 8) * U * lora + 2.0 ** -16 * lora + 1.01 * s * ue @ A.abs())
        inside(got.grad_X[sl], rX, bX + 2.0 ** -8 * (rX.abs() + bX) + 2.0 ** -130, f"grad_X {m}")
    for i in range(2):
        (a, b), = L.set[i].split(got[1 + 2 * i], got[2 + 2 * i])
        inside(a, dA[i], mA[i], f"dA {i}")
        inside(b, dB[i], mB[i], f"dB {i}")


def test_refusals(lq, torch):
    L = Layer(lq, torch, 64, 128, 20, [8, 4])
    other = Layer(lq, torch, 72, 128, 20, [8, 4])
    S, bad = L.set, pytest.raises(ValueError)
    for args, kw in (((L.qw[0], other.qw[0]), {}), ((*L.qw, S[0]), {}), ((*L.qw, S[0], other.set[1]), {}),
                     ((*L.qw, S[0], lq.AdapterSet(L.adapters[1][:1])), {}), (tuple(L.qw), dict(act="relu"))):
        with bad:
            lq.GatedPair(*args, **kw)
    bare = lq.GatedPair(*L.qw)
    d = lq.Dropout(0.1, lq.dropout_key(0))
    saved = lq.GatedSaved(L.g, L.u)
    for call in (lambda: lq.gated_forward(L.pair, L.X), lambda: lq.gated_forward(bare, L.X, L.ids),
                 lambda: lq.gated_forward(bare, L.X, dropout=(d, None)), lambda: lq.gated_forward(L.pair, L.X[:, :64], L.ids),
                 lambda: lq.gated_forward(L.pair, L.X.float(), L.ids), lambda: lq.gated_forward(L.pair, L.X, L.ids[:7]),
                 lambda: lq.gated_forward(L.pair, L.X, L.ids, out_dtype=torch.float16),
                 lambda: lq.gated_forward(L.pair, L.X.t().contiguous().t(), L.ids),
                 lambda: lq.gated_backward(L.pair, L.X[:5], L.G, L.ids, saved),
                 lambda: lq.gated_backward(L.pair, L.X, L.G, L.ids, saved._replace(g=L.g[:3])),
                 lambda: lq.gated_backward(L.pair, L.X, L.G, L.ids, saved._replace(u=L.u.float())),
                 lambda: lq.gated_backward(L.pair, L.X, L.G, L.ids, saved._replace(t_up=L.g)),
                 lambda: lq.gated_backward(L.pair, L.X, L.G, L.ids, saved, route=lq.adapter_route(L.ids[:9], 2))):
        with bad:
            call()
    with pytest.raises(lq.LqError):
        lq.gated_backward(L.pair, None, L.G, L.ids, saved)      # dA needs X
