"""Every launch of the many-adapter, dropout and gated calls goes to their tensors' device, whichever is current.

One GPU stands for all: the calls' way of making a device current is replaced by one that notes for which device it
is asked, and the library by one that notes what it had noted when something was launched.
"""
import contextlib

import pytest

pytestmark = pytest.mark.gpu

HOST_ONLY = ("_workspace", "_bytes", "_build", "lq_check_")


@pytest.fixture(scope="module")
def lq():
    import quantized_lora_fine_lq_amd as mod
    return mod


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available()
    return t


@pytest.fixture
def launches(lq, monkeypatch):
    """[(entry point, device made current for it or None)]"""
    from quantized_lora_fine_lq_amd import adapters, dropouts, gated
    seen, current = [], [None]

    @contextlib.contextmanager
    def on_device(_, dev):
        current[0] = dev
        yield
        current[0] = None

    class Library:
        def __getattr__(self, name):
            call = getattr(lq.lib, name)
            if not any(part in name for part in HOST_ONLY):
                seen.append((name, current[0]))
            return call

    for mod in (adapters, dropouts, gated):
        monkeypatch.setattr(mod, "on_device", on_device)
        monkeypatch.setattr(mod, "lib", Library())
    return seen


def test_launches_go_to_the_tensors_device(lq, torch, launches):
    from quantized_lora_fine_lq_amd import adapters, dropouts, gated
    bf16, dev = torch.bfloat16, torch.device("cuda", torch.cuda.current_device())
    randn = lambda *s: torch.randn(*s, device=dev)
    N, K, M, r = 128, 64, 70, 8
    gate, up = (lq.QWeight.from_weight(randn(N, K)) for _ in range(2))
    sets = [lq.AdapterSet([(randn(r, K).to(bf16), randn(N, r).to(bf16), 16.0) for _ in range(2)]) for _ in range(2)]
    X, G = randn(M, K).to(bf16), randn(M, N).to(bf16)
    ids = torch.randint(0, 2, (M,), device=dev).int()
    drop = lq.Dropout(0.1, lq.dropout_key(3))
    lq.adapter_route(ids, 2)
    for m in (M, 5):
        lq.adapters_forward(gate, X[:m], sets[0], ids[:m])
    lq.adapters_backward(gate, X, G, sets[0], ids)
    lq.adapters_forward(gate, X, sets[0], ids, dropout=drop)
    lq.adapters_backward(gate, X, G, sets[0], ids, dropout=drop)
    lq.dropout(X, drop)
    pair = lq.GatedPair(gate, up, *sets)
    _, saved = lq.gated_forward(pair, X, ids)
    lq.gated_backward(pair, X, G, ids, saved)
    grads = lq.GradList([randn(33), randn(7)])
    lq.grad_norm(grads)
    lq.clip_grad_norm(grads, 1.0)
    assert all(at == dev for _, at in launches), [name for name, at in launches if at != dev]
    launching = {n for mod in (adapters, dropouts, gated) for n in mod.SIGNATURES if not any(part in n for part in HOST_ONLY)}
    assert {name for name, _ in launches} == launching
