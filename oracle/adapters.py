"""Many adapters over one quantized projection, and gradient clipping, in float64.

QLoRA page, introduction: h = dequant(W0_NF4) x + (alpha / r) B A x; here token
m has the adapter a = ids[m] (or none, for an id outside [0, n)):

    t[m] = A_a X[m],   H[m] = W' X[m] + s_a B_a t[m],   s_a = alpha_a / r_a
    u[m] = B_a^T G[m], dX[m] = W'^T G[m] + s_a A_a^T u[m]
    dA_a = s_a sum_m u[m] X[m]^T,  dB_a = s_a sum_m G[m] t[m]^T  over a's tokens.

Beside each result stands the sum of the absolute values of its terms, from
which the tests derive how far float32 accumulation may be off.
"""
from __future__ import annotations

import numpy as np


def _f64(a):
    return np.asarray(a, dtype=np.float64)


def route(ids, n: int):
    """(off [n + 2], perm [M], sid [M]): tokens stably sorted by adapter, those
    without one last."""
    key = np.array([i if 0 <= i < n else n for i in ids], dtype=np.int64)
    perm = np.argsort(key, kind="stable")
    off = [int((key < a).sum()) for a in range(n + 1)] + [len(key)]
    return np.array(off), perm, key[perm]


def _tokens(ids, a: int):
    return np.nonzero(np.asarray(ids) == a)[0]


def forward(Wd, X, adapters, ids):
    """adapters: list of (A [r, K], B [N, r], scale). Returns (H, t, abs H, abs t, lora abs)
    with t [M, r_max] zero past each token's rank."""
    Wd, X = _f64(Wd), _f64(X)
    r_max = max(A.shape[0] for A, _, _ in adapters)
    H, mag = X @ Wd.T, np.abs(X) @ np.abs(Wd).T
    t, tmag = np.zeros((X.shape[0], r_max)), np.zeros((X.shape[0], r_max))
    lora = np.zeros_like(H)      # sum of |s t' B| with t' = sum |x a|
    for a, (A, B, s) in enumerate(adapters):
        m, r, A, B = _tokens(ids, a), A.shape[0], _f64(A), _f64(B)
        t[m, :r] = X[m] @ A.T
        tmag[m, :r] = np.abs(X[m]) @ np.abs(A).T
        H[m] += s * (t[m, :r] @ B.T)
        lora[m] = abs(s) * (tmag[m, :r] @ np.abs(B).T)
    return H, t, mag, tmag, lora


def backward(Wd, X, G, adapters, ids, t=None):
    """Returns (dX, [dA], [dB]) and, in the same layout, the absolute sums
    (dX base, dX adapter part, [dA], [dB])."""
    Wd, X, G = _f64(Wd), _f64(X), _f64(G)
    dX, mag = G @ Wd, np.abs(G) @ np.abs(Wd)
    lora = np.zeros_like(dX)
    dA, dB, mA, mB = [], [], [], []
    for a, (A, B, s) in enumerate(adapters):
        m, r, A, B = _tokens(ids, a), A.shape[0], _f64(A), _f64(B)
        Xm, Gm = X[m], G[m]
        u, um = Gm @ B, np.abs(Gm) @ np.abs(B)
        tm, tmm = (Xm @ A.T, np.abs(Xm) @ np.abs(A).T) if t is None else (_f64(t)[m, :r], np.abs(_f64(t)[m, :r]))
        dX[m] += s * (u @ A)
        lora[m] = abs(s) * (um @ np.abs(A))
        dA.append(s * (u.T @ Xm))
        dB.append(s * (Gm.T @ tm))
        mA.append(abs(s) * (um.T @ np.abs(Xm)))
        mB.append(abs(s) * (np.abs(Gm).T @ tmm))
    return (dX, dA, dB), (mag, lora, mA, mB)


def clip(tensors, groups, n_groups: int, max_norm: float, eps: float):
    """(norms [n_groups], clipped tensors) in float64."""
    sq = [0.0] * n_groups
    for x, g in zip(tensors, groups):
        sq[g] += float(np.square(_f64(x)).sum())
    norms = np.sqrt(np.array(sq))
    with np.errstate(invalid="ignore"):
        q = max_norm / (norms + eps)
        coef = np.where(q > 1.0, 1.0, q)
        return norms, [_f64(x) * coef[g] for x, g in zip(tensors, groups)]
