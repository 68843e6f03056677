"""The gated half of a layer, as it is trained and served: gated_forward, the down
projection of its result, dropout of the output and their backward, with one
route and one key; eager, captured and as single tokens.

A step is checked stage by stage, each against the formulas in float64 at the
values that the stage before it gave, with that stage's own bounds; what the
block returns must be those stages' outputs bit for bit.
"""
import importlib.util
import os
import types

import numpy as np
import pytest

from oracle import dropout as odr
from oracle import gated as og
import test_gpu_dropout as td
import test_gpu_gated as tg
from test_gpu_adapters import U, f64, make_weight

pytestmark = pytest.mark.gpu
SEED, STEP, SITE = 91, 5, 12


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")
    spec = importlib.util.spec_from_file_location("gated_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Parts:
    """A block of the example and its projections as the layers of test_gpu_gated.py and test_gpu_dropout.py."""

    def __init__(self, lq, torch, example, N, K, M, ranks, p, weight="nf4_dq", act="silu", seed=0):
        L = self.L = tg.Layer(lq, torch, N, K, M, ranks, weight=weight, act=act, seed=seed)
        rng = np.random.default_rng([seed, N, K, M])
        bf = lambda shape, std=1.0: torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).cuda().to(
            torch.bfloat16)
        self.p, self.G = p, bf((M, K))
        down = make_weight(lq, torch, rng, K, N, weight.split("+")[0])
        adapters = [(bf((r, N), 0.05), bf((K, r), 0.05), float(rng.uniform(0.5, 3.0) * r)) for r in ranks]
        D = self.D = types.SimpleNamespace(N=K, K=N, M=M, qw=down, adapters=adapters, set=lq.AdapterSet(adapters),
                                           Wd=f64(lq.dequant(down)), ids=L.ids.cpu().numpy(), ids_dev=L.ids)
        D.host = [(f64(A), f64(B), float(np.float32(a / A.shape[0]))) for A, B, a in adapters]
        self.key = lq.dropout_key(SEED, STEP)
        self.block = example.Block(*L.qw, down, *L.set, D.set, self.key, p=p, site=SITE, act=act)
        self.at_step(STEP)

    def at_step(self, step):
        """The layers' masks of that step."""
        torch, L = self.L.torch, self.L
        L.drops = tuple(self.block.drops[:2])
        masks = [odr.kept(SEED, step, SITE + i, self.p, (L.M, (L.K, L.K, L.N, L.K)[i])) for i in range(4)]
        self.keep = [torch.from_numpy(m).cuda().double() * f for m, f in masks]
        self.down_mask = masks[2]
        L.keep = self.keep[:2]


@pytest.mark.parametrize("case", [
    # N, K, M, ranks, p, weight, act
    (320, 192, 20, [8, 16], 0.1, "nf4_dq", "silu"),
    (512, 256, 300, [16, 8, 64, 1, 7], 0.1, "nf4_dq", "gelu_tanh"),
    (256, 448, 517, [12, 40], 0.3, "codebook+nf4_f32", "silu"),
    (1024, 512, 1100, [64, 64, 64], 0.05, "nf4_dq", "gelu"),
], ids=str)
def test_a_training_step(lq, torch, example, case):
    N, K, M, ranks, p, weight, act = case
    P = Parts(lq, torch, example, N, K, M, ranks, p, weight, act)
    L, D = P.L, P.D
    y, s = P.block.forward(L.X, L.ids)
    grad_X, flat = P.block.backward(P.G, L.ids, s)

    h, saved = tg.check_forward(lq, torch, L, route=s.route)
    assert torch.equal(h, s.h) and all(torch.equal(a, b) for a, b in zip(saved, s.pair))

    D.X = h
    D.G = lq.dropout(P.G, P.block.drops[3])
    want = P.G.double() * P.keep[3]
    assert bool(((D.G.double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
    z, t = lq.adapters_forward(D.qw, h, D.set, L.ids, dropout=P.block.drops[2])
    (rH, mH, lH), (T, mT), (rX, mX, lX), rA, rB = td.reference(torch, D, *P.down_mask, t)
    r, tiny = D.set.r_max, 2.0 ** -130
    tg.inside(t, T, (N + 10) * U * mT, "down's t")
    tg.inside(z, rH, (N + 3 * r + 8) * U * (mH + lH) + (N + 2) * U * lH + 2.0 ** -16 * lH + 2.0 ** -8 * rH.abs() + tiny, "down")
    assert torch.equal(t, s.t_down)
    # kept / (1 - p) and the sum are rounded to bfloat16 once each
    dropped = z.double() * P.keep[3]
    tg.inside(y, dropped + L.X.double(),
              2.0 ** -8 * (dropped.abs() + (dropped + L.X.double()).abs() * (1 + 2.0 ** -8) + 2.0 ** -8 * dropped.abs()) + tiny, "y")

    Gh, dA, dB = lq.adapters_backward(D.qw, h, D.G, D.set, L.ids, t=t, dropout=P.block.drops[2])
    tg.inside(Gh, rX, (K + 3 * r + 8) * U * (mX + lX) + (K + 2) * U * lX + 2.0 ** -16 * lX + 2.0 ** -8 * rX.abs() + tiny, "grad_h")
    for a, (da, db) in enumerate(D.set.split(dA, dB)):
        tokens = int((L.ids == a).sum())
        tg.inside(da, rA[a][0], (3 * tokens + K + 18) * U * rA[a][1], f"down's dA {a}")
        tg.inside(db, rB[a][0], (3 * tokens + 16) * U * rB[a][1], f"down's dB {a}")
    assert torch.equal(dA, flat[2][0]) and torch.equal(dB, flat[2][1])

    L.G, L.g, L.u = Gh, saved.g, saved.u
    g = tg.check_backward(lq, torch, L, route=s.route)
    assert torch.equal(g.grad_X + P.G, grad_X)
    assert all(torch.equal(a, b) for a, b in zip(g[1:], (*flat[0], *flat[1])))


def test_captured_steps(lq, torch, example):
    """Forward, backward and the key's advance captured; replays on new tokens, eager work between them."""
    P = Parts(lq, torch, example, 320, 192, 150, [16, 40], 0.2)
    L = P.L
    route = lq.adapter_route(L.ids, 2)

    def step():
        y, s = P.block.forward(L.X, L.ids, route)
        gx, flat = P.block.backward(P.G, L.ids, s)
        return y, gx, *(t for ab in flat for t in ab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
        P.key[1] += 1
    seen = []
    for k in range(4):
        if k != 2:          # (the second and third replay: the same tokens, other masks)
            L.X.copy_(torch.randn_like(L.X))
            P.G.copy_(torch.randn_like(P.G))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert int(P.key[1]) == STEP + k + 1
        P.key[1] -= 1
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
        P.key[1] += 1
        torch.cuda.synchronize()
        seen.append(got[0])
    assert not torch.equal(seen[1], seen[2])


def test_single_tokens(lq, torch, example):
    """Decode of a batch of one token per request, against the stages' formulas."""
    P = Parts(lq, torch, example, 512, 256, 9, [8, 16, 4, 32], 0.1)
    L, D = P.L, P.D
    L.drops, L.keep = None, [None, None]
    h, _ = tg.check_forward(lq, torch, L, save=False)
    D.X, D.G = h, P.G
    (rH, mH, lH), *_ = td.reference(torch, D, np.ones((9, 512), bool), 1.0)
    z, _ = lq.adapters_forward(D.qw, h, D.set, L.ids, save_t=False)
    r = D.set.r_max
    tg.inside(z, rH, (512 + 3 * r + 8) * U * (mH + lH) + 514 * U * lH + 2.0 ** -16 * lH + 2.0 ** -8 * rH.abs() + 2.0 ** -130, "down")
    assert torch.equal(P.block.decode(L.X, L.ids), z + L.X)


def test_gradients_against_differences(lq, torch, example):
    """d/d eps of sum(y R) along directions of X and of every adapter, by central differences in float64."""
    P = Parts(lq, torch, example, 128, 64, 90, [8, 16], 0.25, act="gelu_tanh", seed=2)
    L, D = P.L, P.D
    _, s = P.block.forward(L.X, L.ids)
    grad_X, flat = P.block.backward(P.G, L.ids, s)
    rng = np.random.default_rng(3)
    rand = lambda x: torch.from_numpy(rng.standard_normal(tuple(x.shape))).cuda()
    sets = (*L.set, D.set)
    VX = rand(L.X)
    V = [[(rand(A), rand(B)) for A, B, _ in st.adapters] for st in sets]
    W = (*L.W, torch.from_numpy(D.Wd).cuda())

    def project(i, X, ea, eb):
        H = X @ W[i].T
        for k, (A, B, alpha) in enumerate(sets[i].adapters):
            m = (L.ids == k).nonzero()[:, 0]
            H[m] += float(np.float32(alpha / A.shape[0])) * ((X * P.keep[i])[m] @ (A.double() + ea * V[i][k][0]).T) @ (
                B.double() + eb * V[i][k][1]).T
        return H

    def loss(ex=0.0, at=None, ea=0.0, eb=0.0):
        X = L.X.double() + ex * VX
        g, u = (project(i, X, *((ea, eb) if at == i else (0.0, 0.0))) for i in range(2))
        h = torch.from_numpy(og.act(g.cpu().numpy(), L.act)[0]).cuda() * u
        y = X + project(2, h, *((ea, eb) if at == 2 else (0.0, 0.0))) * P.keep[3]
        return float((y * P.G.double()).sum())
    e = 1e-4

    def close(grads, dirs, plus, minus, what):
        value = sum(float((a.double() * b).sum()) for a, b in zip(grads, dirs))
        scale = sum(float((a.double() * b).square().sum()) for a, b in zip(grads, dirs)) ** 0.5
        # six roundings to bfloat16 lie on the way (g, u, h, the dropped gradient, grad_h, grad_X or the terms' own),
        # each off by at most 2^-8 of its terms, of random sign: sixteen 2^-8 of the root of the sum of squares
        assert abs(value - (plus - minus) / (2 * e)) <= 16 * 2.0 ** -8 * scale + 1e-6 * abs(value), what
    close([grad_X], [VX], loss(ex=e), loss(ex=-e), "X")
    for i, st in enumerate(sets):
        parts = st.split(*flat[i])
        close([a for a, _ in parts], [a for a, _ in V[i]], loss(at=i, ea=e), loss(at=i, ea=-e), f"A {i}")
        close([b for _, b in parts], [b for _, b in V[i]], loss(at=i, eb=e), loss(at=i, eb=-e), f"B {i}")


def test_example_runs(torch, example):
    losses, out = example.run(steps=5)
    assert len(losses) == 5 and all(np.isfinite(losses)) and bool(torch.isfinite(out.float()).all())


def test_an_example_step_applies_each_gradient_to_its_matrix(lq, torch, example, monkeypatch):
    """The clipped gradients of gate, up and down, adapter by adapter, reach their own matrices with the step's sign and
    size, in float32 and then in the copies that the kernels read; the key counts the steps."""
    keys, lists, steps = [], [], []
    key, clip, backward = lq.dropout_key, lq.clip_grad_norm, example.Block.backward
    monkeypatch.setattr(example.lq, "dropout_key", lambda *a: keys.append(key(*a)) or keys[-1])
    monkeypatch.setattr(example.lq, "clip_grad_norm", lambda grads, *a: lists.append(grads) or clip(grads, *a))

    def recorded(block, *a):
        before = [t.clone() for s in (block.pair.gate_adapters, block.pair.up_adapters, block.down_set)
                  for A, B, _ in s.adapters for t in (A, B)]
        out = backward(block, *a)
        steps.append((block, before, out[1]))
        return out
    monkeypatch.setattr(example.Block, "backward", recorded)
    lr = 0.01
    example.run(steps=1, lr=lr)
    (block, before, flat), (grads,) = steps[0], lists
    sets = (block.pair.gate_adapters, block.pair.up_adapters, block.down_set)
    n = block.pair.n
    own = [g for s, (dA, dB) in zip(sets, flat) for ab in s.split(dA, dB) for g in ab]
    assert [g.data_ptr() for g in grads.tensors] == [g.data_ptr() for g in own]
    assert grads.n_groups == n
    after = [t for s in sets for A, B, _ in s.adapters for t in (A, B)]
    for i, (old, new, g) in enumerate(zip(before, after, own)):      # (the clip worked in place)
        g = g.double()
        if i % 2:      # B began at zero
            assert not old.any() and torch.equal(new, torch.zeros_like(g, dtype=torch.float32).sub_(g.float(), alpha=lr * 10).to(
                torch.bfloat16))
        else:          # A: the float32 value is within half a step of its first copy, and the new copy of the new value
            assert ((new.double() - (old.double() - lr * 10 * g)).abs() <=
                    2.0 ** -8 * (old.double().abs() * 1.01 + new.double().abs()) + 2.0 ** -22 * g.abs()).all()
    assert any(g.any() for g in own[1::2])
    # each adapter's gradients were clipped to norm 1 together
    norms = [sum(float(own[2 * (k * n + a) + j].double().square().sum()) for k in range(3) for j in range(2)) ** 0.5 for a in range(n)]
    assert all(x <= 1 + 1e-5 for x in norms)
    example.run(steps=3)
    assert keys[0].tolist() == [0, 1] and keys[1].tolist() == [0, 3]
