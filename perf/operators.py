"""Cases and plain forms of the many-adapter operators.

Three operators that a program meets when it serves or trains several low-rank
adapters over one frozen quantized projection:

``forward``   H = X W'^T + s_a (X A_a^T) B_a^T with a = ids[m] the adapter of
              token m (a negative id: the base projection alone), and
              t[m] = A_a X[m], kept for the backward.
``backward``  grad_X = G W' + s_a (G B_a) A_a and, per adapter over its own
              tokens, dA_a = s_a (G B_a)^T X and dB_a = s_a G^T t.
``clip``      the L2 norm of each job's gradients over its many tensors, and
              the gradients scaled by min(1, max_norm / (norm + 1e-6)).

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
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request answering, one token at a time: pure latency
        dict(name="decode_1", op="forward", N=4096, K=4096, M=1, adapters=8, ranks="16", order="mixed",
             base=0.0, weight="nf4_dq", out="bf16"),
        # a full decode batch, nearly every request with an adapter of its own
        dict(name="decode_16", op="forward", N=4096, K=4096, M=16, adapters=16, ranks="16", order="mixed",
             base=0.1, weight="nf4_dq", out="bf16"),
        # a large decode batch over a wide projection, adapters shared by some requests, some requests without one
        dict(name="decode_64_wide", op="forward", N=28672, K=8192, M=64, adapters=32, ranks="8,16,32", order="mixed",
             base=0.2, weight="nf4_dq", out="bf16"),
        # a per-channel codebook weight, a batch of decoded tokens, float32 result
        dict(name="decode_250_codebook", op="forward", N=4096, K=4096, M=250, adapters=20, ranks="16", order="mixed",
             base=0.1, weight="codebook", out="f32"),
        # prompts of several requests side by side, ranks of different users
        dict(name="prefill_1999", op="forward", N=4096, K=4096, M=1999, adapters=8, ranks="8,16,32,64", order="runs",
             base=0.15, weight="nf4_dq", out="bf16"),
        # fine-tuning jobs batched over one MLP projection
        dict(name="train_fwd_4096", op="forward", N=11008, K=4096, M=4096, adapters=4, ranks="64", order="runs",
             base=0.0, weight="nf4_dq", out="bf16"),
        # many small jobs, some without a token in this batch, t recomputed
        dict(name="bwd_300_small", op="backward", N=1024, K=1024, M=300, adapters=40, ranks="4,7,16,32", order="runs",
             base=0.05, weight="nf4_f32", saved_t=False),
        # attention projection of eight jobs
        dict(name="bwd_2048", op="backward", N=4096, K=4096, M=2048, adapters=8, ranks="16", order="runs",
             base=0.0, weight="nf4_dq", saved_t=True),
        # the largest: four jobs' MLP projection
        dict(name="bwd_4096_mlp", op="backward", N=4096, K=11008, M=4096, adapters=4, ranks="64", order="runs",
             base=0.0, weight="nf4_dq", saved_t=True),
        # one layer's adapter gradients
        dict(name="clip_layer", op="clip", layers=1, hidden=4096, inner=11008, rank=16, groups=1, dtype="f32",
             odd=False, clipped=True),
        # all layers of four jobs, each clipped by its own norm
        dict(name="clip_model", op="clip", layers=32, hidden=4096, inner=11008, rank=16, groups=4, dtype="f32",
             odd=False, clipped=True),
        # bfloat16 gradients of uneven sizes at unaligned addresses, below the limit
        dict(name="clip_odd_bf16", op="clip", layers=24, hidden=1021, inner=2749, rank=7, groups=3, dtype="bf16",
             odd=True, clipped=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "clip"])
    if op == "clip":
        hidden = _log(rng, 64, 4096)
        return dict(op="clip", layers=_log(rng, 1, 32), hidden=hidden, inner=int(hidden * rng.uniform(1.0, 2.7)),
                    rank=rng.choice([1, 4, 8, 15, 16]), groups=rng.randint(1, 4), dtype=rng.choice(["f32", "bf16", "f16"]),
                    odd=rng.random() < 0.5, clipped=rng.random() < 0.7)
    while True:
        N, K, M = _log(rng, 64, 11008), 64 * _log(rng, 1, 172), _log(rng, 1, 4096)
        if N * K * M <= 4096 * 11008 * 4096:
            break
    ranks = ",".join(str(rng.choice([1, 4, 7, 8, 16, 24, 32, 64])) for _ in range(rng.randint(1, 4)))
    case = dict(op=op, N=N, K=K, M=M, adapters=_log(rng, 1, 64), ranks=ranks, order=rng.choice(["mixed", "runs"]),
                base=rng.choice([0.0, 0.1, 0.5]), weight=rng.choice(["nf4_dq", "nf4_f32", "codebook"]))
    if op == "forward":
        case["out"] = rng.choice(["bf16", "f32"])
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


def _clip_shapes(case):
    h, i, r = case["hidden"], case["inner"], case["rank"]
    layer = []
    for n, k in [(h, h)] * 4 + [(i, h)] * 2 + [(h, i)]:
        layer += [(r, k), (n, r)]
    shapes, groups = [], []
    for g in range(case["groups"]):
        for _ in range(case["layers"]):
            shapes += layer
            groups += [g] * len(layer)
    return shapes, groups


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    if case["op"] == "clip":
        dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[case["dtype"]]
        shapes, groups = _clip_shapes(case)
        total = sum(a * b for a, b in shapes)
        gap = 1 if case["odd"] else 0      # an element between tensors: addresses aligned to the element alone
        flat = torch.zeros(total + gap * len(shapes), dtype=dtype, device="cuda")
        out_flat = torch.zeros_like(flat)
        values = torch.randn(total, generator=gen, device="cuda").mul_(1e-2).to(dtype)
        grads, out, pos, taken = [], [], 0, 0
        for a, b in shapes:
            pos += gap
            grads.append(flat[pos:pos + a * b].view(a, b))
            out.append(out_flat[pos:pos + a * b].view(a, b))
            grads[-1].copy_(values[taken:taken + a * b].view(a, b))
            pos, taken = pos + a * b, taken + a * b
        norm = 1e-2 * math.sqrt(total / case["groups"])
        state = dict(op="clip", grads=grads, out=out, flat=flat, out_flat=out_flat, groups=groups, n_groups=case["groups"],
                     max_norm=norm * (0.3 if case["clipped"] else 3.0))
        if own:
            import quantized_lora_fine_lq_amd as lq
            state["list"] = lq.GradList(grads, groups)
            state["out_list"] = lq.GradList(out, groups)
        return state

    N, K, M = case["N"], case["K"], case["M"]
    w = _make_weight(case, gen)
    ranks = [int(x) for x in case["ranks"].split(",")]
    adapters = []
    for a in range(case["adapters"]):
        r = ranks[a % len(ranks)]
        adapters.append((_normal(gen, (r, K), 0.02), _normal(gen, (N, r), 0.02), 2.0 * r))
    ids = torch.from_numpy(_token_ids(case, rng)).cuda()
    state = dict(op=case["op"], w=w, X=_normal(gen, (M, K)), adapters=adapters, ids=ids,
                 out=torch.float32 if case.get("out") == "f32" else torch.bfloat16)
    if case["op"] == "backward":
        state["G"] = _normal(gen, (M, N))
        state["t"] = None
        if case["saved_t"]:
            t = torch.zeros(M, max(ranks[:case["adapters"]]), device="cuda")
            for a, (A, _, _) in enumerate(adapters):
                rows = (ids == a).nonzero()[:, 0]
                t[rows, :A.shape[0]] = state["X"][rows].float() @ A.float().T
            state["t"] = t
    if own:
        import quantized_lora_fine_lq_amd as lq
        if w["kind"] == "codebook":
            state["qw"] = lq.QWeight(N, K, w["codes"], absmax_q=w["absmax_q"], dq_scale=w["dq_scale"],
                                     dq_mean=w["dq_mean"], fmt=lq.LQ_FMT_CODEBOOK, row_bits=w["row_bits"],
                                     row_offset=w["row_offset"], levels=w["levels"])
        elif w["kind"] == "nf4_f32":
            state["qw"] = lq.QWeight(N, K, w["codes"], absmax=w["absmax"])
        else:
            state["qw"] = lq.QWeight(N, K, w["codes"], absmax_q=w["absmax_q"], dq_scale=w["dq_scale"],
                                     dq_mean=w["dq_mean"])
        state["set"] = lq.AdapterSet(adapters)
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
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


def _owners(st):
    """The adapters side by side: for column j of all R = sum of r_a columns, its adapter, its place
    in it and its scale; and on [M, R], where the column belongs to the token's adapter."""
    dev = st["ids"].device
    r = torch.tensor([A.shape[0] for A, _, _ in st["adapters"]])
    owner = torch.repeat_interleave(torch.arange(len(r)), r)
    place = torch.arange(owner.numel()) - (r.cumsum(0) - r)[owner]
    scale = torch.tensor([alpha / A.shape[0] for A, _, alpha in st["adapters"]])[owner]
    owner, place, scale = owner.to(dev), place.to(dev), scale.to(dev)
    return owner, place, scale, (st["ids"][:, None] == owner).float()


def _plain_forward(st):
    X = st["X"].float()
    A = torch.cat([A for A, _, _ in st["adapters"]]).float()
    B = torch.cat([B for _, B, _ in st["adapters"]], 1).float()
    owner, place, scale, on = _owners(st)
    T = (X @ A.T) * on
    H = X @ _weight(st["w"]).T + (T * scale) @ B.T
    t = torch.zeros(X.shape[0], max(A.shape[0] for A, _, _ in st["adapters"]), device=X.device)
    t.index_add_(1, place, T)      # a token's columns but its own adapter's are zero
    return {"H": H.to(st["out"]), "t": t}


def _plain_backward(st):
    X, G = st["X"].float(), st["G"].float()
    A = torch.cat([A for A, _, _ in st["adapters"]]).float()
    B = torch.cat([B for _, B, _ in st["adapters"]], 1).float()
    owner, place, scale, on = _owners(st)
    T = (X @ A.T if st["t"] is None else st["t"][:, place]) * on * scale
    U = (G @ B) * on * scale
    gx = G @ _weight(st["w"]) + U @ A
    dB = torch.split(G.T @ T, [B.shape[1] for _, B, _ in st["adapters"]], 1)
    return {"grad_X": gx.to(torch.bfloat16), "dA": U.T @ X, "dB": torch.cat([d.reshape(-1) for d in dB])}


def _plain_clip(st):
    # the jobs' gradients are equal shares of one buffer (zeros between the tensors)
    x = st["flat"].float().view(st["n_groups"], -1)
    norms = (x * x).sum(1).sqrt()
    coef = (st["max_norm"] / (norms + EPS)).clamp(max=1.0)
    st["out_flat"].copy_((x * coef[:, None]).view(-1))
    return {"norms": norms, "grads": st["out_flat"]}


def run(st):
    if not own:
        return {"forward": _plain_forward, "backward": _plain_backward, "clip": _plain_clip}[st["op"]](st)
    import quantized_lora_fine_lq_amd as lq
    if st["op"] == "forward":
        H, t = lq.adapters_forward(st["qw"], st["X"], st["set"], st["ids"], out_dtype=st["out"])
        return {"H": H, "t": t}
    if st["op"] == "backward":
        gx, dA, dB = lq.adapters_backward(st["qw"], st["X"], st["G"], st["set"], st["ids"], t=st["t"])
        return {"grad_X": gx, "dA": dA, "dB": dB}
    norms = lq.clip_grad_norm(st["list"], st["max_norm"], out=st["out_list"])
    return {"norms": norms, "grads": st["out_flat"]}


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


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "clip":
        total = [0.0] * st["n_groups"]
        for g, x in zip(st["groups"], st["grads"]):
            total[g] = total[g] + x.double().pow(2).sum()
        norms = torch.stack([torch.as_tensor(v).sqrt() for v in total])
        scale = torch.minimum(torch.ones_like(norms), st["max_norm"] / (norms + EPS))
        grads = torch.zeros(st["out_flat"].numel(), dtype=torch.float64, device=norms.device)
        for g, x, o in zip(st["groups"], st["grads"], st["out"]):
            at = o.storage_offset()
            grads[at:at + x.numel()] = (x.double() * scale[g]).reshape(-1)
        return {"norms": norms, "grads": grads}
    W, X, ids = _exact_weight(st["w"]), st["X"].double(), st["ids"]
    n = len(st["adapters"])
    member = [(ids == a).double()[:, None] for a in range(n)]
    if st["op"] == "forward":
        H = X @ W.T
        t = torch.zeros(X.shape[0], max(A.shape[0] for A, _, _ in st["adapters"]), dtype=torch.float64, device=X.device)
        for (A, B, alpha), on in zip(st["adapters"], member):
            ta = (X @ A.double().T) * on
            t[:, :A.shape[0]] += ta
            H += (ta @ B.double().T) * (alpha / A.shape[0])
        return {"H": H, "t": t}
    G = st["G"].double()
    gx = G @ W
    dA, dB = [], []
    for (A, B, alpha), on in zip(st["adapters"], member):
        r = A.shape[0]
        u = (G @ B.double()) * on * (alpha / r)
        t = X @ A.double().T if st["t"] is None else st["t"][:, :r].double()
        gx += u @ A.double()
        dA.append(u.T @ X)
        dB.append(G.T @ (t * on * (alpha / r)))
    return {"grad_X": gx, "dA": torch.cat(dA), "dB": torch.cat([d.reshape(-1) for d in dB])}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "clip":
        shapes, _ = _clip_shapes(case)
        n = sum(a * b for a, b in shapes)
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * size + 4 * case["groups"], "flops": 3 * n}
    N, K, M, n = case["N"], case["K"], case["M"], case["adapters"]
    bits = {"nf4_dq": 4 + 8 / 64 + 32 / 16384, "nf4_f32": 4.5, "codebook": 1.75 + 8 / 64 + 32 / 16384}[case["weight"]]
    ranks = [int(x) for x in case["ranks"].split(",")]
    rs = [ranks[a % len(ranks)] for a in range(n)]
    mean_r = sum(rs) / n
    used = n * (1.0 - (1.0 - 1.0 / n) ** M) * (1.0 - case["base"])      # adapters that some token needs, on average
    tokens = M * (1.0 - case["base"])
    small = N * K * bits / 8 + used * mean_r * (N + K) * 2 + 4 * M
    if case["op"] == "forward":
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": int(small + 2 * M * K + size * M * N + 4 * M * max(rs)),
                "flops": int(2 * M * N * K + 2 * tokens * mean_r * (N + K))}
    flops = 2 * M * N * K + 4 * tokens * mean_r * (N + K) + (0 if case["saved_t"] else 2 * tokens * mean_r * K)
    saved = 4 * M * max(rs) if case["saved_t"] else 0
    return {"bytes": int(small + saved + 2 * M * (2 * K + N) + 4 * sum(rs) * (N + K)), "flops": int(flops)}
