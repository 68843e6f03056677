"""Fine-tuning jobs and decode requests over one frozen NF4 projection.

Several jobs train an adapter each, their tokens mixed in one batch: the batch
is sorted once (``adapter_route``), ``adapters_forward`` and
``adapters_backward`` run all adapters over the one quantized weight, and
``clip_grad_norm`` clips each job's gradients by its own norm. The trained
adapters then answer single tokens, one per request.

    python examples/many_adapters.py [--steps 60]

Each job's target is the frozen projection plus a low-rank change of its own,
so its loss falls towards zero as its adapter finds that change.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_lora_fine_lq_amd as lq  # noqa: E402

N, K, TOKENS, RANKS, ALPHA = 512, 256, 384, (8, 16, 4), 16.0


def run(steps: int = 60, lr: float = 0.02, max_norm: float = 1.0, seed: int = 0):
    """Returns (first losses, last losses, decode outputs, their targets): losses per job."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    bf16 = torch.bfloat16
    qw = lq.QWeight.from_weight(randn(N, K) * 0.05)
    n = len(RANKS)
    change = [(randn(N, 2) @ randn(2, K)) * (0.5 / K ** 0.5) for _ in RANKS]
    frozen = lq.dequant(qw).float()

    # the jobs' adapters: float32 masters, bfloat16 copies that the kernels read
    master = [(randn(r, K) / K ** 0.5, torch.zeros(N, r, device="cuda")) for r in RANKS]
    adapters = lq.AdapterSet([(A.to(bf16), B.to(bf16), ALPHA) for A, B in master])
    moments = [[torch.zeros_like(p) for p in ab for _ in range(2)] for ab in master]

    def target(X, ids):
        out = X.float() @ frozen.T
        for a in range(n):
            out = torch.where((ids == a)[:, None], out + X.float() @ change[a].T, out)
        return out

    history = []
    for step in range(steps):
        X = randn(TOKENS, K).to(bf16)
        ids = torch.randint(0, n, (TOKENS,), generator=gen, device="cuda").int()
        route = lq.adapter_route(ids, n)                     # once for every projection of the step
        H, t = lq.adapters_forward(qw, X, adapters, ids, route=route)
        err = H.float() - target(X, ids)
        share = torch.zeros(n, device="cuda").index_add_(0, ids.long(), torch.ones(TOKENS, device="cuda"))
        loss = torch.zeros(n, device="cuda").index_add_(0, ids.long(), err.square().mean(1)) / share
        G = (err / share[ids.long()][:, None]).to(bf16)      # of each job's own mean (N / 2 times)
        _, dA, dB = lq.adapters_backward(qw, X, G, adapters, ids, t=t, need_grad_x=False, route=route)
        grads = adapters.split(dA, dB)
        flat = [g for ab in grads for g in ab]
        # by job; a list a step, since adapters_backward returns new tensors
        lq.clip_grad_norm(lq.GradList(flat, [a for a in range(n) for _ in range(2)]), max_norm)
        for a, ab in enumerate(grads):                       # Adam, into the masters and the kernels' copies
            for k, g in enumerate(ab):
                m, v = moments[a][2 * k], moments[a][2 * k + 1]
                m.lerp_(g, 0.1)
                v.lerp_(g.square(), 0.05)
                hat = (m / (1 - 0.9 ** (step + 1))) / ((v / (1 - 0.95 ** (step + 1))).sqrt() + 1e-8)
                master[a][k].sub_(hat, alpha=lr)
                adapters.adapters[a][k].copy_(master[a][k])
        history.append(loss)

    # decode: one token of each job, and one request without an adapter
    x = randn(n + 1, K).to(bf16)
    ids = torch.arange(n + 1, device="cuda").int()
    ids[n] = -1
    h, _ = lq.adapters_forward(qw, x, adapters, ids, out_dtype=torch.float32, save_t=False)
    return history[0].tolist(), history[-1].tolist(), h, target(x, ids)


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=60)
    first, last, h, want = run(parser.parse_args().steps)
    for a, (f, l) in enumerate(zip(first, last)):
        print(f"job {a}: rank {RANKS[a]:3d}  loss {f:.4f} -> {l:.4f}")
    for m in range(h.shape[0]):
        rel = ((h[m] - want[m]).norm() / want[m].norm()).item()
        print(f"decode, {'adapter %d' % m if m < len(RANKS) else 'no adapter'}: relative error {rel:.4f}")
