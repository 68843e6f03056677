"""Fine-tuning and serving the gated half of a layer over frozen weights.

    y = X + dropout(down(act(gate(X)) * up(X)))

gate, up and down are NF4 projections, each with an adapter per job, whose
inputs are dropped in training. One key in device memory stands for the step:
the backward forms every mask again from it, and the step's end advances it, so
that the next one draws anew. The trained adapters then answer single tokens.

    python examples/gated_block.py [--steps 40]
"""
import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_lora_fine_lq_amd as lq  # noqa: E402


class Saved(NamedTuple):
    X: object
    h: object
    pair: object     # GatedSaved
    t_down: object
    route: object


class Block:
    """The block over quantized weights gate, up [N, K] and down [K, N]. p: the
    rate of its four dropouts, at sites site .. site + 3 of key (the adapters'
    inputs of gate, up and down, and the block's output)."""

    def __init__(self, gate, up, down, gate_set, up_set, down_set, key, p=0.1, site=0, act="silu"):
        self.pair = lq.GatedPair(gate, up, gate_set, up_set, act=act)
        self.down, self.down_set = down, down_set
        self.drops = [lq.Dropout(p, key, site + i) for i in range(4)]

    def forward(self, X, ids, route=None):
        """(y, Saved): the training forward."""
        if route is None:
            route = lq.adapter_route(ids, self.pair.n)      # once for the three projections
        h, saved = lq.gated_forward(self.pair, X, ids, route=route, dropout=self.drops[:2])
        y, t = lq.adapters_forward(self.down, h, self.down_set, ids, route=route, dropout=self.drops[2])
        lq.dropout(y, self.drops[3], out=y)
        return y.add_(X), Saved(X, h, saved, t, route)

    def backward(self, G, ids, s: Saved):
        """(grad_X, [(dA, dB) of gate, up, down]) for G = dL/dy, on the key as the
        forward found it."""
        Gd = lq.dropout(G, self.drops[3])
        Gh, dA, dB = lq.adapters_backward(self.down, s.h, Gd, self.down_set, ids, t=s.t_down, route=s.route,
                                          dropout=self.drops[2])
        g = lq.gated_backward(self.pair, s.X, Gh, ids, s.pair, route=s.route, dropout=self.drops[:2])
        return g.grad_X.add_(G), [(g.dA_gate, g.dB_gate), (g.dA_up, g.dB_up), (dA, dB)]

    def decode(self, X, ids):
        """y of single tokens: nothing dropped, nothing kept."""
        h, _ = lq.gated_forward(self.pair, X, ids, save=False)
        return lq.adapters_forward(self.down, h, self.down_set, ids, save_t=False)[0].add_(X)


N, K, TOKENS, RANKS, ALPHA = 768, 256, 320, (8, 16), 16.0


def run(steps: int = 40, lr: float = 0.01, max_norm: float = 1.0, seed: int = 0):
    """Returns (the steps' losses, decode outputs of one token per job)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    bf16, n = torch.bfloat16, len(RANKS)
    shapes = ((N, K), (N, K), (K, N))
    weights = [lq.QWeight.from_weight(randn(*s) / s[1] ** 0.5) for s in shapes]
    master = [[(randn(r, k) / k ** 0.5, torch.zeros(o, r, device="cuda")) for r in RANKS] for o, k in shapes]
    sets = [lq.AdapterSet([(A.to(bf16), B.to(bf16), ALPHA) for A, B in m]) for m in master]
    params = [p for m in master for ab in m for p in ab]
    copies = [c for s in sets for A, B, _ in s.adapters for c in (A, B)]
    moments = [torch.zeros_like(p) for p in params]
    key = lq.dropout_key(seed)
    block = Block(*weights, *sets, key)

    change = [randn(K, K) * (0.3 / K ** 0.5) for _ in RANKS]        # what a job's block is to learn
    X = randn(TOKENS, K).to(bf16)
    ids = torch.randint(0, n, (TOKENS,), generator=gen, device="cuda").int()
    calm = Block(*weights, *sets, key, p=0.0)
    target = calm.forward(X, ids)[0].float()
    for a in range(n):
        target = torch.where((ids == a)[:, None], target + X.float() @ change[a].T, target)
    loss = torch.zeros((), device="cuda")

    def step():
        y, saved = block.forward(X, ids)
        err = y.float() - target
        loss.copy_(err.square().mean())
        G = (err / TOKENS).to(bf16)
        _, flat = block.backward(G, ids, saved)
        grads = [g for s, (dA, dB) in zip(sets, flat) for ab in s.split(dA, dB) for g in ab]
        lq.clip_grad_norm(lq.GradList(grads, [a for _ in sets for a in range(n) for _ in range(2)]), max_norm)
        for p, c, m, g in zip(params, copies, moments, grads):
            m.mul_(0.9).add_(g)
            p.sub_(m, alpha=lr * 10)
            c.copy_(p)
        key[1] += 1

    losses = []
    for _ in range(steps):
        step()
        losses.append(float(loss))
    one = torch.arange(n, device="cuda").int()
    return losses, block.decode(X[:n], one)


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=40)
    losses, _ = run(parser.parse_args().steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
