"""Cases and plain forms of dropout and of the gated projection pair.

Operators that a program meets when it trains or serves the MLP half of a layer
over frozen quantized weights:

``dropout``        y = x / (1 - p) where the element is kept, else 0. The mask is a
                   function of (seed, step, site, element) and is stored nowhere: the
                   gradient's mask is formed again from the same four.
``lora_forward``   H = X W'^T + s_a (D A_a^T) B_a^T, t = D A_a^T with D = dropout(X): the
                   adapters of a projection see dropped inputs, the frozen weight the
                   inputs themselves; a = ids[m] (a negative id: no adapter).
``lora_backward``  grad_X = G W' + dropout'(s_a (G B_a) A_a), dA_a = s_a (G B_a)^T D,
                   dB_a = s_a G^T t.
``gated_forward``  h = act(g) u with g and u two such projections of the same X.
``gated_backward`` dg = G u act'(g) and du = G act(g), then lora_backward of both with
                   the two gradients of X added.

The generator is Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw:
"Parallel random numbers: as easy as 1, 2, 3", 2011). Elements 8 i .. 8 i + 7 share
the block of counter (low 32 bits of i, site 4096 + high bits of i, low and high
word of step) and key (low and high word of seed); element 8 i + j takes 16 bits,
half j % 2 of word j / 2, and is dropped where they are below T = round(65536 p),
so p counts in steps of 2^-16; the scale is 65536 / (65536 - T).

W' is the bfloat16 weight that the packed codes and block constants stand for
(bfloat16(float32(level * constant))): that rounding belongs to the weight's
definition, so the plain and the 64-bit forms both start from it.
"""
import math
import statistics

import numpy as np
import torch

own = False

DQ_BLOCK = 256
BLOCK = 64
ACTS = ["silu", "gelu", "gelu_tanh"]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a short batch of hidden states of an odd width, half precision
        dict(name="drop_300_odd_f16", op="dropout", rows=300, cols=1021, dtype="f16", p=0.1),
        # the hidden states of an MLP's inner width in training
        dict(name="drop_4096_mlp", op="dropout", rows=4096, cols=11008, dtype="bf16", p=0.05),
        # many small fine-tuning jobs over one small projection, float32 result
        dict(name="lora_fwd_300_small", op="lora_forward", N=1024, K=1024, M=300, adapters=40, ranks="4,7,16,32",
             order="runs", base=0.05, weight="nf4_f32", out="f32", p=0.05),
        # an attention projection of eight jobs, the usual dropout of adapters
        dict(name="lora_fwd_2048", op="lora_forward", N=4096, K=4096, M=2048, adapters=8, ranks="16", order="runs",
             base=0.0, weight="nf4_dq", out="bf16", p=0.1),
        # the same projection's gradients
        dict(name="lora_bwd_2048", op="lora_backward", N=4096, K=4096, M=2048, adapters=8, ranks="16", order="runs",
             base=0.0, weight="nf4_dq", p=0.1, saved_t=True),
        # four jobs' wide projection back to the hidden size, t formed again
        dict(name="lora_bwd_4096_mlp", op="lora_backward", N=4096, K=11008, M=4096, adapters=4, ranks="64", order="runs",
             base=0.0, weight="nf4_dq", p=0.05, saved_t=False),
        # one request answering, one token at a time: pure latency
        dict(name="gated_decode_1", op="gated_forward", N=11008, K=4096, M=1, adapters=8, ranks="16", order="mixed",
             base=0.0, weight="nf4_dq", out="bf16", p=0.0, act="silu", save=False),
        # a large decode batch of a large model's MLP, adapters shared by some requests, some requests without one
        dict(name="gated_decode_64_wide", op="gated_forward", N=28672, K=8192, M=64, adapters=32, ranks="8,16,32",
             order="mixed", base=0.2, weight="nf4_dq", out="bf16", p=0.0, act="silu", save=False),
        # prompts of several requests side by side, ranks of different users
        dict(name="gated_prefill_1999", op="gated_forward", N=11008, K=4096, M=1999, adapters=8, ranks="8,16,32,64",
             order="runs", base=0.15, weight="nf4_dq", out="bf16", p=0.0, act="silu", save=False),
        # a training step of four jobs, everything kept that the backward needs
        dict(name="gated_train_4096", op="gated_forward", N=11008, K=4096, M=4096, adapters=4, ranks="64", order="runs",
             base=0.0, weight="nf4_dq", out="bf16", p=0.05, act="silu", save=True),
        # many small jobs over a small codebook-quantized MLP, another activation, t formed again
        dict(name="gated_bwd_300_small", op="gated_backward", N=1024, K=1024, M=300, adapters=40, ranks="4,7,16,32",
             order="runs", base=0.05, weight="codebook", p=0.0, act="gelu_tanh", saved_t=False),
        # the largest: the gradients of the training step
        dict(name="gated_bwd_4096", op="gated_backward", N=11008, K=4096, M=4096, adapters=4, ranks="64", order="runs",
             base=0.0, weight="nf4_dq", p=0.05, act="silu", saved_t=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "lora_forward", "lora_backward", "gated_forward", "gated_forward", "gated_backward"])
    p = rng.choice([0.0, 0.05, 0.1, 0.5]) if op != "dropout" else round(rng.uniform(0.01, 0.9), 4)
    if op == "dropout":
        return dict(op=op, rows=_log(rng, 1, 4096), cols=_log(rng, 1, 11008), dtype=rng.choice(["f32", "bf16", "f16"]), p=p)
    while True:
        N, K, M = _log(rng, 64, 11008), 64 * _log(rng, 1, 172), _log(rng, 1, 4096)
        if N * K * M <= 4096 * 11008 * 4096:
            break
    ranks = ",".join(str(rng.choice([1, 4, 7, 8, 16, 24, 32, 64])) for _ in range(rng.randint(1, 4)))
    case = dict(op=op, N=N, K=K, M=M, adapters=_log(rng, 1, 64), ranks=ranks, order=rng.choice(["mixed", "runs"]),
                base=rng.choice([0.0, 0.1, 0.5]), weight=rng.choice(["nf4_dq", "nf4_f32", "codebook"]), p=p)
    if op.startswith("gated"):
        case["act"] = rng.choice(ACTS)
    if op.endswith("forward"):
        case["out"] = rng.choice(["bf16", "f32"])
        if op == "gated_forward":
            case["save"] = rng.random() < 0.5
    else:
        case["N"] = 8 * max(1, N // 8)      # the backward reads G's rows in 16-byte pieces
        case["saved_t"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _levels():
    """The 16 NormalFloat values: 8 + 9 normal quantiles, one of the two zeros dropped."""
    q = statistics.NormalDist().inv_cdf
    delta = 1.0 - 0.5 * (1.0 / 32.0 + 1.0 / 30.0)
    top = q(delta)
    pos = [q(0.5 + (delta - 0.5) * j / 8) / top for j in range(1, 9)]
    neg = [-q(0.5 + (delta - 0.5) * j / 7) / top for j in range(1, 8)]
    return np.array(sorted(neg + [0.0] + pos), dtype=np.float32)


def _double_quantize(c):
    """float32 constants [n] -> (E4M3 codes, per-256 scales, mean)."""
    n = c.numel()
    nd = (n + DQ_BLOCK - 1) // DQ_BLOCK
    mu = c.double().mean().float().reshape(1)
    d = torch.zeros(nd * DQ_BLOCK, device=c.device)
    d[:n] = c - mu
    d = d.reshape(nd, DQ_BLOCK)
    scale = d.abs().amax(1) / 448.0
    q = (d / scale.clamp_min(1e-30)[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.reshape(-1)[:n].view(torch.uint8).contiguous(), scale.contiguous(), mu


def _make_weight(case, gen):
    N, K = case["N"], case["K"]
    w = {"N": N, "K": K, "kind": case["weight"]}
    if case["weight"] == "codebook":
        # widths 1..4 per row in the proportions of a 1.75-bit weight, sorted levels per row
        pick = torch.rand(N, generator=gen, device="cuda")
        bits = 1 + (pick < 0.5).int() + (pick < 0.1875).int() + (pick < 0.0625).int()
        code = torch.randint(0, 16, (N, K), generator=gen, device="cuda", dtype=torch.int32) % (1 << bits)[:, None]
        levels = (torch.rand(N, 16, generator=gen, device="cuda") * 2 - 1).sort(1).values
        nb = K // BLOCK
        code = code.reshape(N, nb, BLOCK)
        weights = (1 << torch.arange(8, device="cuda", dtype=torch.int32))
        planes = [(((code >> p) & 1).reshape(N, nb, 8, 8) * weights).sum(3).to(torch.uint8) for p in range(4)]
        bits_host = bits.cpu().tolist()
        offs = [0]
        for b in bits_host:
            offs.append(offs[-1] + K * b // 8)
        packed = torch.empty(offs[-1], dtype=torch.uint8, device="cuda")
        off = torch.tensor(offs, device="cuda")
        for b in (1, 2, 3, 4):
            rows = (bits == b).nonzero()[:, 0]
            if rows.numel():
                body = torch.stack(planes[:b], 2)[rows].reshape(rows.numel(), -1)     # [rows, nb * b * 8]
                at = off[rows][:, None] + torch.arange(body.shape[1], device="cuda")
                packed[at.reshape(-1)] = body.reshape(-1)
        c = 0.02 * (2.0 + 0.5 * torch.rand(N * nb, generator=gen, device="cuda"))
        w.update(codes=packed, row_bits=bits.to(torch.uint8), row_offset=off, levels=levels.contiguous())
    else:
        lv = torch.from_numpy(_levels()).cuda()
        mid = (lv[1:] + lv[:-1]) / 2
        W = torch.randn(N * K // BLOCK, BLOCK, generator=gen, device="cuda") * 0.02
        c = W.abs().amax(1)
        code = torch.bucketize(W / c[:, None], mid, out_int32=True).to(torch.uint8).reshape(-1, 2)
        w.update(codes=((code[:, 0] << 4) | code[:, 1]).contiguous(), levels=lv)
    if case["weight"] == "nf4_f32":
        w["absmax"] = c.contiguous()
    else:
        w["absmax_q"], w["dq_scale"], w["dq_mean"] = _double_quantize(c)
    return w


def _token_ids(case, rng):
    """The adapter of each token: -1 where the request uses the base weight alone."""
    M, n = case["M"], case["adapters"]
    if case["order"] == "mixed":
        ids = rng.integers(0, n, M)
        ids[rng.random(M) < case["base"]] = -1
    else:
        # requests of uneven length, one after the other; not every adapter need have one
        cuts = np.sort(rng.integers(0, M + 1, max(0, n - 1)))
        lens = np.diff(np.concatenate([[0], cuts, [M]]))
        who = rng.permutation(n)
        who = np.where(rng.random(n) < case["base"], -1, who)
        ids = np.repeat(who, lens)
    return ids.astype(np.int32)


def _normal(gen, shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SITES = (5, 6)      # of the two projections' dropout; the first alone where there is one


def _adapters(case, gen):
    ranks = [int(x) for x in case["ranks"].split(",")]
    out = []
    for a in range(case["adapters"]):
        r = ranks[a % len(ranks)]
        out.append((_normal(gen, (r, case["K"]), 0.02), _normal(gen, (case["N"], r), 0.02), 2.0 * r))
    return out


def _qweight(lq, w):
    if w["kind"] == "codebook":
        return lq.QWeight(w["N"], w["K"], w["codes"], absmax_q=w["absmax_q"], dq_scale=w["dq_scale"],
                          dq_mean=w["dq_mean"], fmt=lq.LQ_FMT_CODEBOOK, row_bits=w["row_bits"],
                          row_offset=w["row_offset"], levels=w["levels"])
    if w["kind"] == "nf4_f32":
        return lq.QWeight(w["N"], w["K"], w["codes"], absmax=w["absmax"])
    return lq.QWeight(w["N"], w["K"], w["codes"], absmax_q=w["absmax_q"], dq_scale=w["dq_scale"], dq_mean=w["dq_mean"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    key = torch.from_numpy(rng.integers(0, 1 << 62, 2)).cuda()      # seed and step of the generator
    state = dict(op=case["op"], p=case["p"], key=key, act=case.get("act"), save=case.get("save"))
    if case["op"] == "dropout":
        x = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        state["x"], state["out"] = x, torch.empty_like(x)
        if own:
            import quantized_lora_fine_lq_amd as lq
            state["drop"] = lq.Dropout(case["p"], key, SITES[0])
        return state
    N, K, M = case["N"], case["K"], case["M"]
    n = 2 if case["op"].startswith("gated") else 1
    state["w"] = [_make_weight(case, gen) for _ in range(n)]
    state["adapters"] = [_adapters(case, gen) for _ in range(n)]
    state["ids"] = torch.from_numpy(_token_ids(case, rng)).cuda()
    state["X"] = _normal(gen, (M, K))
    state["out"] = DTYPES[case.get("out", "bf16")]
    if case["op"].endswith("backward"):
        state["G"] = _normal(gen, (M, N))
        if n == 2:      # the two projections' values that the forward kept
            state["gu"] = [_normal(gen, (M, N), 1.3) for _ in range(2)]
        state["t"] = [None] * n
        if case["saved_t"]:
            state["t"] = [_spread(state, _down(state, k), k) for k in range(n)]
    if own:
        import quantized_lora_fine_lq_amd as lq
        qw, sets = [_qweight(lq, w) for w in state["w"]], [lq.AdapterSet(a) for a in state["adapters"]]
        drops = [lq.Dropout(case["p"], key, SITES[k]) for k in range(n)] if case["p"] else None
        if n == 2:
            state["pair"] = lq.GatedPair(qw[0], qw[1], sets[0], sets[1], act=case["act"])
            if case["op"] == "gated_backward":
                state["saved"] = lq.GatedSaved(state["gu"][0], state["gu"][1], state["t"][0], state["t"][1])
            state["drops"] = drops
        else:
            state["qw"], state["set"], state["drops"] = qw[0], sets[0], drops[0] if drops else None
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_bits(key, site, numel):
    """The 16 random bits of elements 0 .. numel - 1, int64."""
    i = torch.arange((numel + 7) // 8, dtype=torch.int64, device=key.device)
    low = 0xFFFFFFFF
    seed, step = key[0], key[1]
    c0, c1, c2, c3 = i & low, (i >> 32) + site * 4096, step & low, (step >> 32) & low
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57      # modulo 2^64
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 1)
    return words.reshape(-1)[:numel]


def _threshold(p):
    return min(int(round(p * 65536)), 65535)


def _plain_dropout(x, p, key, site):
    """float32, not yet rounded to x's type."""
    T = _threshold(p)
    kept = (_plain_bits(key, site, x.numel()) >= T).reshape(x.shape)
    return torch.where(kept, x.float() * (65536.0 / (65536.0 - T)), 0.0)


def _constants(w):
    if "absmax" in w:
        return w["absmax"]
    q = w["absmax_q"].view(torch.float8_e4m3fn).double()
    s = w["dq_scale"].double().repeat_interleave(DQ_BLOCK)[:q.numel()]
    return (q * s + w["dq_mean"].double()).float()      # one rounding, as a fused multiply-add


def _weight(w):
    """W' [N, K] as float32 (exactly bfloat16 values)."""
    N, K = w["N"], w["K"]
    codes = w["codes"]
    if w["kind"] == "codebook":
        k, p = torch.arange(K, device=codes.device), torch.arange(4, device=codes.device)
        b = w["row_bits"].int()[:, None, None]
        at = (k // BLOCK * 8)[None, :, None] * b + (k % BLOCK // 8)[:, None] + 8 * torch.minimum(p, b - 1)
        bit = (codes[at + w["row_offset"][:-1, None, None]] >> (k % 8).to(torch.uint8)[:, None]) & 1
        code = ((bit * (p < b)) << p).sum(2)
        out = torch.gather(w["levels"], 1, code)
    else:
        both = torch.stack([codes >> 4, codes & 15], 1).reshape(-1)
        out = w["levels"][both.int()]
    out = (out.reshape(-1, BLOCK) * _constants(w)[:, None]).to(torch.bfloat16).float()
    return out.reshape(N, K)


def _owners(st, k):
    """Set k's adapters side by side: for column j of all R = sum of r_a columns, its adapter, its place
    in it and its scale; and on [M, R], where the column belongs to the token's adapter."""
    dev = st["ids"].device
    r = torch.tensor([A.shape[0] for A, _, _ in st["adapters"][k]])
    owner = torch.repeat_interleave(torch.arange(len(r)), r)
    place = torch.arange(owner.numel()) - (r.cumsum(0) - r)[owner]
    scale = torch.tensor([alpha / A.shape[0] for A, _, alpha in st["adapters"][k]])[owner]
    owner, place, scale = owner.to(dev), place.to(dev), scale.to(dev)
    return place, scale, (st["ids"][:, None] == owner).float()


def _stacked(st, k):
    return (torch.cat([A for A, _, _ in st["adapters"][k]]).float(),
            torch.cat([B for _, B, _ in st["adapters"][k]], 1).float())


def _dropped(st, k):
    return _plain_dropout(st["X"], st["p"], st["key"], SITES[k]) if st["p"] else st["X"].float()


def _down(st, k):
    """t of every token with its own adapter, in that adapter's columns of all."""
    A, _ = _stacked(st, k)
    return (_dropped(st, k) @ A.T) * _owners(st, k)[2]


def _spread(st, T, k):
    """T's columns moved to the first columns of [M, largest rank]."""
    t = torch.zeros(T.shape[0], max(A.shape[0] for A, _, _ in st["adapters"][k]), device=T.device)
    t.index_add_(1, _owners(st, k)[0], T)      # a token's columns but its own adapter's are zero
    return t


def _plain_projection(st, k):
    _, B = _stacked(st, k)
    T = _down(st, k)
    H = st["X"].float() @ _weight(st["w"][k]).T + (T * _owners(st, k)[1]) @ B.T
    return H, _spread(st, T, k)


def _plain_projection_backward(st, k, G):
    """Gradients for the float32 gradient G of projection k's output: of X in float32, of A and B."""
    A, B = _stacked(st, k)
    place, scale, on = _owners(st, k)
    T = (_down(st, k) if st["t"][k] is None else st["t"][k][:, place] * on) * scale
    U = (G @ B) * on * scale
    gx = U @ A
    if st["p"]:
        gx = _plain_dropout(gx, st["p"], st["key"], SITES[k])
    dB = torch.split(G.T @ T, [B.shape[1] for _, B, _ in st["adapters"][k]], 1)
    return G @ _weight(st["w"][k]) + gx, U.T @ _dropped(st, k), torch.cat([d.reshape(-1) for d in dB])


def _plain_act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c, b = math.sqrt(2.0 / math.pi), 0.044715
    th = torch.tanh(c * (g + b * g * g * g))
    return 0.5 * g * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * (c * (1.0 + 3.0 * b * g * g))


def _plain(st):
    op = st["op"]
    if op == "dropout":
        st["out"].copy_(_plain_dropout(st["x"], st["p"], st["key"], SITES[0]))
        return {"y": st["out"]}
    if op == "lora_forward":
        H, t = _plain_projection(st, 0)
        return {"H": H.to(st["out"]), "t": t}
    if op == "lora_backward":
        gx, dA, dB = _plain_projection_backward(st, 0, st["G"].float())
        return {"grad_X": gx.to(torch.bfloat16), "dA": dA, "dB": dB}
    if op == "gated_forward":
        g, t_gate = _plain_projection(st, 0)
        u, t_up = _plain_projection(st, 1)
        out = {"H": (_plain_act(g, st["act"])[0] * u).to(st["out"])}
        if st["save"]:
            out.update(g=g.to(torch.bfloat16), u=u.to(torch.bfloat16), t_gate=t_gate, t_up=t_up)
        return out
    G, g, u = st["G"].float(), st["gu"][0].float(), st["gu"][1].float()
    a, da = _plain_act(g, st["act"])
    gx0, dA0, dB0 = _plain_projection_backward(st, 0, G * u * da)
    gx1, dA1, dB1 = _plain_projection_backward(st, 1, G * a)
    return {"grad_X": (gx0 + gx1).to(torch.bfloat16), "dA_gate": dA0, "dB_gate": dB0, "dA_up": dA1, "dB_up": dB1}


def run(st):
    if not own:
        return _plain(st)
    import quantized_lora_fine_lq_amd as lq
    op = st["op"]
    if op == "dropout":
        return {"y": lq.dropout(st["x"], st["drop"], out=st["out"])}
    if op == "lora_forward":
        H, t = lq.adapters_forward(st["qw"], st["X"], st["set"], st["ids"], out_dtype=st["out"], dropout=st["drops"])
        return {"H": H, "t": t}
    if op == "lora_backward":
        gx, dA, dB = lq.adapters_backward(st["qw"], st["X"], st["G"], st["set"], st["ids"], t=st["t"][0],
                                          dropout=st["drops"])
        return {"grad_X": gx, "dA": dA, "dB": dB}
    if op == "gated_forward":
        H, saved = lq.gated_forward(st["pair"], st["X"], st["ids"], out_dtype=st["out"], save=st["save"],
                                    dropout=st["drops"])
        return {"H": H} if saved is None else {"H": H, "g": saved.g, "u": saved.u, "t_gate": saved.t_gate,
                                               "t_up": saved.t_up}
    grads = lq.gated_backward(st["pair"], st["X"], st["G"], st["ids"], st["saved"], dropout=st["drops"])
    return {"grad_X": grads.grad_X, "dA_gate": grads.dA_gate, "dB_gate": grads.dB_gate, "dA_up": grads.dA_up,
            "dB_up": grads.dB_up}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_weight(w):
    """W' [N, K] in float64, decoded code by code from the stored bytes."""
    N, K = w["N"], w["K"]
    j = torch.arange(N * K // BLOCK, device=w["codes"].device)
    if "absmax" in w:
        const = w["absmax"].double()
    else:
        byte = w["absmax_q"].int()
        sign = 1.0 - 2.0 * (byte >> 7).double()
        e, m = (byte >> 3) & 15, (byte & 7).double()
        mag = torch.where(e > 0, (1.0 + m / 8.0) * torch.exp2(e.double() - 7.0), m * 2.0 ** -9)
        const = (sign * mag * w["dq_scale"].double()[j // DQ_BLOCK] + w["dq_mean"].double()).float().double()
    value = torch.empty(N, K, dtype=torch.float64, device=const.device)
    step = max(1, (1 << 24) // K)
    for i in range(0, N, step):
        rows = torch.arange(i, min(N, i + step), device=const.device)
        k = torch.arange(K, device=const.device)
        if w["kind"] == "codebook":
            b = w["row_bits"][rows].long()[:, None]
            code = torch.zeros(rows.numel(), K, dtype=torch.long, device=const.device)
            for p in range(4):
                at = w["row_offset"][rows][:, None] + (k // BLOCK) * 8 * b + 8 * torch.clamp(b - 1, max=p) + (k % BLOCK) // 8
                bit = (w["codes"][at].long() >> (k % 8)) & 1
                code += torch.where(b > p, bit << p, torch.zeros_like(bit))
            lv = w["levels"].double()[rows[:, None], code]
        else:
            at = rows[:, None] * (K // 2) + k // 2
            byte = w["codes"][at].int()
            lv = w["levels"].double()[torch.where(k % 2 == 0, byte >> 4, byte & 15)]
        c = const[rows[:, None] * (K // BLOCK) + k // BLOCK]
        value[rows] = (lv * c).float().to(torch.bfloat16).double()
    return value


def _exact_kept(key, site, numel, p):
    """Which elements dropout keeps and their factor, by the generator's definition in whole numbers on the host."""
    word, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    seed, step = (v & 0xFFFFFFFFFFFFFFFF for v in key.cpu().tolist())
    block = np.arange((numel + 7) // 8, dtype=np.uint64)
    x = [block & word, (block >> half) + np.uint64(site * 4096), np.full_like(block, step & 0xFFFFFFFF),
         np.full_like(block, step >> 32)]
    for r in range(10):
        a = np.uint64((seed + r * 0x9E3779B9) & 0xFFFFFFFF)
        b = np.uint64(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        first, second = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(second >> half) ^ x[1] ^ a, second & word, (first >> half) ^ x[3] ^ b, first & word]
    out = np.empty((block.size, 8), dtype=np.uint16)
    for w in range(4):
        out[:, 2 * w], out[:, 2 * w + 1] = x[w] & np.uint64(0xFFFF), x[w] >> np.uint64(16)
    limit = min(int(round(p * 65536)), 65535)
    return torch.from_numpy(out.reshape(-1)[:numel] >= limit).to(key.device), 65536.0 / (65536 - limit)


def _exact_act(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    if act == "gelu":
        phi = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    inner = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(2 * inner)      # (1 + tanh) / 2
    return g * s, s + g * 2 * s * (1 - s) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    key, p = st["key"], st["p"]

    def drop(x, k):
        if not p and case["op"] != "dropout":
            return x.double()
        kept, factor = _exact_kept(key, SITES[k], x.numel(), p)
        return torch.where(kept.reshape(x.shape), x.double() * factor, torch.zeros((), dtype=torch.float64, device=x.device))

    if case["op"] == "dropout":
        return {"y": drop(st["x"], 0)}
    X, ids = st["X"].double(), st["ids"]

    def member(a):
        return (ids == a).double()[:, None]

    def forward(k):
        H = X @ _exact_weight(st["w"][k]).T
        D = drop(st["X"], k)
        t = torch.zeros(X.shape[0], max(A.shape[0] for A, _, _ in st["adapters"][k]), dtype=torch.float64, device=X.device)
        for a, (A, B, alpha) in enumerate(st["adapters"][k]):
            ta = (D @ A.double().T) * member(a)
            t[:, :A.shape[0]] += ta
            H += (ta @ B.double().T) * (alpha / A.shape[0])
        return H, t

    def backward(k, G):
        D = drop(st["X"], k)
        gx = torch.zeros_like(X)
        dA, dB = [], []
        for a, (A, B, alpha) in enumerate(st["adapters"][k]):
            r = A.shape[0]
            u = (G @ B.double()) * member(a) * (alpha / r)
            t = D @ A.double().T if st["t"][k] is None else st["t"][k][:, :r].double()
            gx += u @ A.double()
            dA.append(u.T @ D)
            dB.append((G.T @ (t * member(a) * (alpha / r))).reshape(-1))
        return G @ _exact_weight(st["w"][k]) + drop(gx, k), torch.cat(dA), torch.cat(dB)

    if case["op"] == "lora_forward":
        H, t = forward(0)
        return {"H": H, "t": t}
    if case["op"] == "lora_backward":
        gx, dA, dB = backward(0, st["G"].double())
        return {"grad_X": gx, "dA": dA, "dB": dB}
    if case["op"] == "gated_forward":
        (g, t_gate), (u, t_up) = forward(0), forward(1)
        H = _exact_act(g, st["act"])[0] * u
        return {"H": H, "g": g, "u": u, "t_gate": t_gate, "t_up": t_up} if st["save"] else {"H": H}
    G, g, u = st["G"].double(), st["gu"][0].double(), st["gu"][1].double()
    value, slope = _exact_act(g, st["act"])
    gx0, dA0, dB0 = backward(0, G * u * slope)
    gx1, dA1, dB1 = backward(1, G * value)
    return {"grad_X": gx0 + gx1, "dA_gate": dA0, "dB_gate": dB0, "dA_up": dA1, "dB_up": dB1}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "f32" else 2), "flops": n}
    N, K, M, n = case["N"], case["K"], case["M"], case["adapters"]
    both = 2 if case["op"].startswith("gated") else 1
    bits = {"nf4_dq": 4 + 8 / 64 + 32 / 16384, "nf4_f32": 4.5, "codebook": 1.75 + 8 / 64 + 32 / 16384}[case["weight"]]
    ranks = [int(x) for x in case["ranks"].split(",")]
    rs = [ranks[a % len(ranks)] for a in range(n)]
    mean_r = sum(rs) / n
    used = n * (1.0 - (1.0 - 1.0 / n) ** M) * (1.0 - case["base"])      # adapters that some token needs, on average
    tokens = M * (1.0 - case["base"])
    small = both * (N * K * bits / 8 + used * mean_r * (N + K) * 2) + 4 * M
    if case["op"].endswith("forward"):
        kept = 4 * M * max(rs) if both == 1 else 2 * (2 * M * N + 4 * M * max(rs)) if case["save"] else 0
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": int(small + 2 * M * K + size * M * N + kept),
                "flops": int(both * (2 * M * N * K + 2 * tokens * mean_r * (N + K)))}
    flops = both * (2 * M * N * K + 4 * tokens * mean_r * (N + K) + (0 if case["saved_t"] else 2 * tokens * mean_r * K))
    saved = both * 4 * M * max(rs) if case["saved_t"] else 0
    acts = 2 * M * (2 * K + (3 * N if both == 2 else N))      # X and its gradient; G, and g and u
    return {"bytes": int(small + saved + acts + both * 4 * sum(rs) * (N + K)), "flops": int(flops)}
