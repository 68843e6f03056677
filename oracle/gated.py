"""The gated pair's activations in float64: h = act(g) u, dg = G u act'(g),
du = G act(g)."""
from __future__ import annotations

import numpy as np
from scipy.special import erfc, expit


def act(g, kind: str):
    """(act(g), act'(g))."""
    g = np.asarray(g, dtype=np.float64)
    if kind == "silu":
        s = expit(g)      # keeps its digits where it is small
        return g * s, s + g * s * expit(-g)
    if kind == "gelu":
        phi = 0.5 * erfc(-g / np.sqrt(2.0))
        return g * phi, phi + g * np.exp(-0.5 * g * g) / np.sqrt(2.0 * np.pi)
    if kind == "gelu_tanh":
        c, b = np.sqrt(2.0 / np.pi), 0.044715
        y = 2.0 * c * (g + b * g ** 3)
        s = expit(y)      # (1 + tanh(y / 2)) / 2
        return g * s, s + g * s * expit(-y) * 2.0 * c * (1.0 + 3.0 * b * g * g)
    raise ValueError(kind)
