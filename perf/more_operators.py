"""Workloads of the 16-bit layers and of the output head around the experts: a
matrix product with its epilogue, the gated feed-forward block, the scores of
given tokens, and distillation from a teacher's top logits.

Each case is one call, or one training step (forward and backward), in its
plain form (elementary torch operations in 32 or 64 bits, rounded once) or, with
`own` set, through the library.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through an attention output projection kept in 16 bits, the residual added
        dict(name="dense_token", op="dense", M=1, N=6144, K=2048, x="bf16", y="bf16", bias=False, act="none",
             residual=True, train=False),
        # a verify batch through one rank's share of the output head, logits in fp32
        dict(name="dense_head", op="dense", M=16, N=16384, K=6144, x="bf16", y="fp32", bias=False, act="none",
             residual=False, train=False),
        # a training step of odd sizes, everything in the epilogue
        dict(name="dense_odd", op="dense", M=77, N=1543, K=1448, x="fp16", y="fp16", bias=True, act="silu",
             residual=True, train=True),
        # a training step of a square layer on a chunk of 4096 tokens
        dict(name="dense_train", op="dense", M=4096, N=6144, K=6144, x="bf16", y="bf16", bias=True, act="gelu",
             residual=False, train=True),
        # a decode step of a dense feed-forward block (one rank's share of it)
        dict(name="gated_decode", op="gated", M=4, H=6144, I=2048, x="bf16", act="silu", train=False),
        # a training step of odd sizes
        dict(name="gated_odd", op="gated", M=333, H=2056, I=1159, x="fp16", act="gelu_tanh", train=True),
        # a training step of the block on a chunk of 4096 tokens
        dict(name="gated_train", op="gated", M=4096, H=6144, I=2048, x="bf16", act="silu", train=True),
        # the drafted tokens of a verify batch scored against the whole vocabulary
        dict(name="scores_verify", op="scores", M=16, V=131072, x="fp32", k=8),
        # a small vocabulary of odd size with banned tokens, an odd batch
        dict(name="scores_odd", op="scores", M=77, V=30011, x="fp16", k=5),
        # the tokens of a prompt chunk, with the teacher's alternatives kept for distillation
        dict(name="scores_prompt", op="scores", M=2048, V=131072, x="bf16", k=32),
        # a training step on few rows of odd size, forward and backward by themselves
        dict(name="distill_odd", op="distill", M=61, V=30011, x="fp32", k=20, T=2.0, fused=False),
        # a training step of the head on a chunk of 2048 tokens
        dict(name="distill_train", op="distill", M=2048, V=131072, x="bf16", k=32, T=1.0, fused=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("dense", "gated", "scores", "distill"))
    x = rng.choice(("bf16", "bf16", "fp16"))
    train = rng.random() < 0.5
    if op == "dense":
        while True:
            M, N, K = _log(rng, 1, 4096), _log(rng, 16, 32768), 8 * _log(rng, 16, 1024)
            if M * N * K <= (1 if train else 3) * 4096 * 6144 * 6144 and N * K <= 16384 * 6144:
                return dict(op=op, M=M, N=N, K=K, x=x, y=x if train else rng.choice((x, "fp32")),
                            bias=rng.random() < 0.5, act=rng.choice(("none", "none", "relu", "silu", "gelu", "gelu_tanh")),
                            residual=rng.random() < 0.5, train=train)
    if op == "gated":
        while True:
            M, H, I = _log(rng, 1, 4096), 8 * _log(rng, 16, 1024), _log(rng, 16, 8192)
            if M * H * I <= 4096 * 6144 * 2048 and H * I <= 6144 * 8192:
                return dict(op=op, M=M, H=H, I=I, x=x, act=rng.choice(("silu", "silu", "relu", "gelu", "gelu_tanh")),
                            train=train)
    x = rng.choice(("bf16", "fp16", "fp32"))
    while True:
        M, V = _log(rng, 1, 4096), _log(rng, 64, 262144)
        if M * V * BYTES[x] <= 2048 * 131072 * 2:
            break
    if op == "scores":
        return dict(op=op, M=M, V=V, x=x, k=rng.randint(0, 32))
    return dict(op=op, M=M, V=V, x=x, k=rng.randint(1, 64), T=rng.choice((1.0, 1.0, 2.0, 0.7)),
                fused=rng.random() < 0.5)


def work(case):
    c = case
    M = c["M"]
    if c["op"] == "dense":
        N, K, b, train = c["N"], c["K"], BYTES[c["y"]], c["train"]
        moved = 2 * (M * K + N * K) + b * M * N * (2 if c["residual"] else 1) + (2 * N if c["bias"] else 0)
        if train:  # dy in; dx, dw and the bias's gradient out
            moved += 2 * (M * N + M * K + N * K) + (2 * N if c["bias"] else 0)
        return {"bytes": moved, "flops": (6 if train else 2) * M * N * K}
    if c["op"] == "gated":
        H, I = c["H"], c["I"]
        moved = 2 * (M * H + 2 * I * H + M * I)
        if c["train"]:  # dh in; dx and dw out
            moved += 2 * (M * I + M * H + 2 * I * H)
        return {"bytes": moved, "flops": (12 if c["train"] else 4) * M * H * I}
    V, k = c["V"], c["k"]
    if c["op"] == "scores":
        return {"bytes": M * (V * BYTES[c["x"]] + 12 + 8 * k), "flops": 6 * M * V}
    return {"bytes": M * (2 * V * BYTES[c["x"]] + 8 * k + 8), "flops": 8 * M * V}


# ------------------------------------------------------------------ inputs
def _inputs(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    M = c["M"]
    if c["op"] == "dense":
        N, K, t = c["N"], c["K"], TYPES[c["x"]]
        d = {"x": normal(M, K).to(t), "w": (normal(N, K) / math.sqrt(K)).to(t)}
        d["bias"] = normal(N).to(t) if c["bias"] else None
        d["residual"] = normal(M, N).to(TYPES[c["y"]]) if c["residual"] else None
        d["dy"] = normal(M, N).to(t) if c["train"] else None
        return d
    if c["op"] == "gated":
        H, I, t = c["H"], c["I"], TYPES[c["x"]]
        return {"x": normal(M, H).to(t), "w": (normal(2 * I, H) / math.sqrt(H)).to(t),
                "dy": normal(M, I).to(t) if c["train"] else None}
    V, k = c["V"], c["k"]
    # logits of a row: a spread of its own, some tokens banned, and the vocabulary's
    # last entries padding
    z = torch.empty((M, V), dtype=TYPES[c["x"]], device=DEV)
    for a in range(0, M, 256):
        part = normal(min(256, M - a), V) * (1 + 3 * uniform(min(256, M - a), 1))
        part[uniform(*part.shape) < 0.002] = -math.inf
        part[:, V - V // 512:] = -math.inf
        z[a:a + 256] = part
    if c["op"] == "scores":
        return {"z": z, "tokens": (uniform(M) * (V - V // 512)).int().clamp_(max=V - 1)}
    # distinct tokens of the teacher's: one in each of k equal stretches; some
    # rows hold fewer than k, every 16th none (padding)
    width = max((V - V // 512) // k, 1)
    ids = (torch.arange(k, device=DEV) * width + (uniform(M, k) * width).long()).clamp_(max=V - 1).int()
    z.scatter_(1, ids.long(), (normal(M, k) * 2 + 4).to(z.dtype))  # none of them is banned
    held = (uniform(M, 1) * 1.5 * k + 1).long()
    held[15::16] = 0
    ids[torch.arange(k, device=DEV)[None] >= held] = -1
    t = torch.sort(normal(M, k) * 2 + 6, dim=1, descending=True)[0]
    return {"z": z, "ids": ids.contiguous(), "t": t.contiguous(), "weight": (uniform(M) + 0.5)}


def prepare(case, seed):
    c = case
    d = dict(_inputs(c, seed), case=c)
    if not own:
        return d
    # what a program keeps: the handle on its weights, output buffers, a workspace
    from quantized_moe_expert_route_amd import binding as B

    M = c["M"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=DEV)

    def scratch(n):
        return empty(max(n, 16), torch.uint8)

    if c["op"] == "dense":
        t = TYPES[c["x"]]
        d["op"] = B.Dense(d["w"], bias=d["bias"], activation=c["act"], max_M=M)
        d["out"] = empty((M, c["N"]), TYPES[c["y"]])
        d["ws"] = scratch(d["op"].workspace_bytes(M, train=c["train"]))
        d["pre"] = empty((M, c["N"]), t) if c["train"] and c["act"] != "none" else None
        if c["train"]:
            d["dx"], d["dw"] = torch.empty_like(d["x"]), torch.empty_like(d["w"])
            d["dbias"] = torch.empty_like(d["bias"]) if c["bias"] else None
    elif c["op"] == "gated":
        t = TYPES[c["x"]]
        d["op"] = B.Gated(d["w"], activation=c["act"], max_M=M)
        d["out"] = empty((M, c["I"]), t)
        d["ws"] = scratch(d["op"].workspace_bytes(M, train=c["train"]))
        if c["train"]:
            d["pre"] = empty((M, 2 * c["I"]), t)
            d["dx"], d["dw"] = torch.empty_like(d["x"]), torch.empty_like(d["w"])
    elif c["op"] == "scores":
        d["op"] = B.TokenScores(c["V"], top_k=c["k"], dtype=d["z"].dtype, max_M=M)
        d["ws"] = scratch(d["op"].workspace_bytes(M))
        d["lp"], d["entropy"] = empty((M,), torch.float32), empty((M,), torch.float32)
        if c["k"]:
            d["top"], d["top_ids"] = empty((M, c["k"]), torch.float32), empty((M, c["k"]), torch.int32)
    else:
        d["op"] = B.Distill(c["V"], c["k"], dtype=d["z"].dtype, temperature=c["T"], max_M=M)
        d["ws"] = scratch(d["op"].workspace_bytes(M))
        d["loss"], d["lse"], d["grad"] = empty((M,), torch.float32), empty((M,), torch.float32), torch.empty_like(d["z"])
    return d


def _run_own(d, c):
    op = d["op"]
    if c["op"] == "dense":
        op.forward(d["x"], d["out"], residual=d["residual"], pre=d["pre"], workspace=d["ws"])
        if not c["train"]:
            return d["out"]
        op.backward(d["dy"], d["x"], dx=d["dx"], dw=d["dw"], dbias=d["dbias"], pre=d["pre"], workspace=d["ws"])
        return (d["out"], d["dx"], d["dw"]) + ((d["dbias"],) if c["bias"] else ())
    if c["op"] == "gated":
        if not c["train"]:
            return op.forward(d["x"], d["out"], workspace=d["ws"])
        op.forward(d["x"], d["out"], pre=d["pre"], workspace=d["ws"])
        op.backward(d["dy"], d["x"], d["pre"], dx=d["dx"], dw=d["dw"], workspace=d["ws"])
        return d["out"], d["dx"], d["dw"]
    if c["op"] == "scores":
        if not c["k"]:
            op.forward(d["z"], d["tokens"], d["lp"], entropy=d["entropy"], workspace=d["ws"])
            return d["lp"], d["entropy"]
        op.forward(d["z"], d["tokens"], d["lp"], entropy=d["entropy"], top_logprobs=d["top"], top_ids=d["top_ids"],
                   workspace=d["ws"])
        return d["lp"], d["entropy"], d["top"], d["top_ids"]
    if c["fused"]:
        op.forward_backward(d["z"], d["ids"], d["t"], d["weight"], d["loss"], d["grad"], workspace=d["ws"])
    else:
        op.forward(d["z"], d["ids"], d["t"], d["loss"], d["lse"], workspace=d["ws"])
        op.backward(d["z"], d["ids"], d["t"], d["lse"], d["weight"], d["grad"])
    return d["loss"], d["grad"]


# ------------------------------------------------------------------ plain form
def _act(name, z):
    """The activation and its derivative, elementwise."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return z * cdf, cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    a, b = math.sqrt(2 / math.pi), 0.044715  # gelu_tanh
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * b * z * z)


def _plain_dense(d, c):
    t = TYPES[c["x"]]
    x, w = d["x"].float(), d["w"].float()
    z = x @ w.t()
    if d["bias"] is not None:
        z = z + d["bias"].float()
    y, slope = _act(c["act"], z)
    if d["residual"] is not None:
        y = y + d["residual"].float()
    y = y.to(TYPES[c["y"]])
    if not c["train"]:
        return y
    dz = d["dy"].float() * slope
    out = (y, (dz @ w).to(t), (dz.t() @ x).to(t))
    return out + ((dz.sum(0).to(t),) if c["bias"] else ())


def _plain_gated(d, c):
    t = TYPES[c["x"]]
    x, w, I = d["x"].float(), d["w"].float(), c["I"]
    gu = x @ w.t()
    g, u = gu[:, :I], gu[:, I:]
    a, slope = _act(c["act"], g)
    h = (a * u).to(t)
    if not c["train"]:
        return h
    dh = d["dy"].float()
    dz = torch.cat((dh * u * slope, dh * a), 1)
    return h, (dz @ w).to(t), (dz.t() @ x).to(t)


def _plain_scores(d, c):
    k = c["k"]
    parts = []
    for a in range(0, c["M"], 256):
        z = d["z"][a:a + 256].float()
        token = d["tokens"][a:a + 256].long()[:, None]
        top = z.max(1, keepdim=True)[0]
        e = torch.exp(z - top)
        total = e.double().sum(1, keepdim=True)
        lse = top.double() + torch.log(total)
        # entropy = lse - sum p z, banned tokens without a part in it
        mean = torch.where(e > 0, e * (z - top), 0.0).double().sum(1, keepdim=True) / total
        part = [(z.gather(1, token).double() - lse)[:, 0].float(), (torch.log(total) - mean)[:, 0].float()]
        if k:
            v, ids = torch.sort(z, dim=1, descending=True, stable=True)
            part += [(v[:, :k].double() - lse).float(), ids[:, :k].int()]
        parts.append(part)
    return tuple(torch.cat(p) for p in zip(*parts))


def _plain_distill(d, c):
    T = c["T"]
    ids, held = d["ids"].long().clamp(min=0), d["ids"] >= 0
    t = torch.where(held, d["t"].double() / T, -math.inf)
    some = held.any(1, keepdim=True)
    e = torch.where(some, torch.exp(t - torch.where(some, t.max(1, keepdim=True)[0], 0.0)), 0.0)
    p = e / torch.where(some, e.sum(1, keepdim=True), 1.0)
    loss = torch.empty(c["M"], dtype=torch.float32, device=DEV)
    grad = torch.empty_like(d["z"])
    for a in range(0, c["M"], 256):
        s = slice(a, a + 256)
        z = d["z"][s].float() / T
        top = z.max(1, keepdim=True)[0]
        e = torch.exp(z - top)
        total = e.double().sum(1, keepdim=True)
        logq = z.gather(1, ids[s]).double() - top.double() - torch.log(total)
        logp = torch.where(p[s] > 0, torch.log(p[s]), 0.0)
        loss[s] = torch.where(p[s] > 0, p[s] * (logp - logq), 0.0).sum(1).float()
        q = torch.where(some[s], (e / total.float()), 0.0)
        q.scatter_add_(1, ids[s], -p[s].float())
        grad[s] = (q * (d["weight"][s, None] / T)).to(grad.dtype)
    return loss, grad


def run(state):
    d, c = state, state["case"]
    if own:
        return _run_own(d, c)
    return {"dense": _plain_dense, "gated": _plain_gated, "scores": _plain_scores, "distill": _plain_distill}[c["op"]](d, c)


# ------------------------------------------------------------------ 64 bits
def _value(name, z):
    """The activation, and its slope as the quotient rule or the density gives it."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.relu(z), torch.heaviside(z, torch.zeros_like(z))
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    if name == "gelu":
        normal = torch.distributions.Normal(0.0, 1.0, validate_args=False)
        return z * torch.special.ndtr(z), torch.special.ndtr(z) + z * torch.exp(normal.log_prob(z))
    # z (1 + tanh u) / 2 = z sigmoid(2 u)
    u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(u2)
    return z * s, s + z * s * torch.sigmoid(-u2) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    if c["op"] in ("dense", "gated"):
        x, w = d["x"].double(), d["w"].double()
        z = torch.cat([x @ part.t() for part in w.split(4096)], 1)
        if c["op"] == "dense":
            if c["bias"]:
                z += d["bias"].double()
            y, slope = _value(c["act"], z)
            if c["residual"]:
                y = y + d["residual"].double()
            dz = d["dy"].double() * slope if c["train"] else None
        else:
            g, u = z.chunk(2, 1)
            a, slope = _value(c["act"], g)
            y = a * u
            dz = torch.cat((slope * u, a), 1) * d["dy"].double().repeat(1, 2) if c["train"] else None
        if not c["train"]:
            return y
        dw = torch.cat([part.t() @ x for part in dz.split(4096, 1)])
        out = (y, dz @ w, dw)
        return out + (dz.sum(0),) if c["op"] == "dense" and c["bias"] else out
    M, V, k = c["M"], c["V"], c["k"]
    if c["op"] == "scores":
        lp = torch.empty(M, dtype=torch.float64, device=DEV)
        entropy = torch.empty_like(lp)
        top = torch.empty((M, k), dtype=torch.float64, device=DEV)
        for a in range(0, M, 128):
            s = slice(a, a + 128)
            lq = torch.log_softmax(d["z"][s].double(), 1)
            lp[s] = lq.gather(1, d["tokens"][s, None].long())[:, 0]
            entropy[s] = torch.special.entr(torch.exp(lq)).sum(1)
            top[s] = torch.topk(lq, k, dim=1)[0] if k else 0
        # the tokens' numbers are no computed value
        return (lp, entropy, top, None) if k else (lp, entropy)
    loss = torch.zeros(M, dtype=torch.float64, device=DEV)
    grad = torch.empty((M, V), dtype=torch.float64, device=DEV)
    for a in range(0, M, 128):
        s = slice(a, a + 128)
        n = d["z"][s].shape[0]
        lq = torch.log_softmax(d["z"][s].double() / c["T"], 1)
        held = d["ids"][s] >= 0
        # the teacher's distribution over the whole vocabulary, one column more for the slots that hold none
        col = torch.where(held, d["ids"][s].long(), V)
        raw = torch.full((n, V + 1), -math.inf, dtype=torch.float64, device=DEV)
        raw.scatter_(1, col, d["t"][s].double() / c["T"])
        p = torch.nan_to_num(torch.softmax(raw[:, :V], 1), nan=0.0)
        loss[s] = (-torch.special.entr(p) - torch.where(p > 0, p * lq, 0.0)).sum(1)
        mass = p.sum(1, keepdim=True).round()
        grad[s] = (torch.exp(lq) * mass - p) * d["weight"][s, None].double() / c["T"]
    return loss, grad
