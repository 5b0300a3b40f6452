"""Workloads of the operators around the routed-MoE call: the router's logits,
a linear layer on MXFP4 weights, and a whole MoE layer of a few tokens from its
hidden states.

Each case is one call, in its plain form (elementary torch operations in 32 or
64 bits, rounded once) or, with `own` set, through the library. Weights are
drawn directly as MXFP4 codes (E2M1 elements, two to a byte, element 2i in the
low nibble; one E8M0 scale per 32) with about the code distribution that
N(0, 0.02) takes under per-32 block quantization.
"""

import math

import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALING = 2.5  # the routing weights of a token sum to this
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's router: 4 tokens, the gate kept in fp32
        dict(name="router_decode", op="router", M=4, E=256, H=6144, x="bf16", w="fp32"),
        # the router of a prefill chunk
        dict(name="router_prefill", op="router", M=4096, E=256, H=6144, x="bf16", w="bf16"),
        # odd sizes: a batch of ragged decodes on a model of other widths
        dict(name="router_odd", op="router", M=77, E=161, H=2056, x="fp16", w="bf16"),
        # one token through an attention output projection with the residual added
        dict(name="linear_token", op="linear", M=1, N=6144, K=2048, x="bf16", y="bf16", bias=False, residual=True),
        # a verify batch (16 tokens) through a dense layer's gate/up projection
        dict(name="linear_verify", op="linear", M=16, N=8192, K=6144, x="bf16", y="bf16", bias=False, residual=False),
        # 4 tokens through an output head, logits in fp32
        dict(name="linear_head", op="linear", M=4, N=131072, K=6144, x="bf16", y="fp32", bias=False, residual=False),
        # odd sizes, fp16 activations, a bias
        dict(name="linear_odd", op="linear", M=37, N=1543, K=1440, x="fp16", y="fp16", bias=True, residual=False),
        # a prefill chunk through a square projection with the residual added
        dict(name="linear_prefill", op="linear", M=4096, N=6144, K=6144, x="bf16", y="bf16", bias=False, residual=True),
        # whole layer, one token
        dict(name="layer_token", op="layer", M=1, H=6144, E=256, I=256, k=8, w="bf16", alike=0.0),
        # whole layer, the 4-token decode of a rank of eight, the gate in fp32
        dict(name="layer_decode", op="layer", M=4, H=6144, E=256, I=256, k=8, w="fp32", alike=0.0),
        # whole layer, a 16-token verify batch: each group of 4 tokens drafted in a row, so alike
        dict(name="layer_verify", op="layer", M=16, H=6144, E=256, I=256, k=8, w="bf16", alike=0.8),
        # whole layer of other widths, an odd batch
        dict(name="layer_odd", op="layer", M=13, H=2560, E=60, I=384, k=6, w="bf16", alike=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("router", "linear", "layer"))
    if op == "router":
        while True:
            M, E, H = _log(rng, 1, 4096), _log(rng, 8, 512), 8 * _log(rng, 32, 1024)
            if M * E * H <= 4096 * 256 * 6144:
                return dict(op=op, M=M, E=E, H=H, x=rng.choice(("bf16", "fp16")), w=rng.choice(("bf16", "fp32")))
    if op == "linear":
        while True:
            M, N, K = _log(rng, 1, 4096), _log(rng, 16, 65536), 32 * _log(rng, 4, 512)
            if M * N * K <= 4096 * 6144 * 6144 and N * K <= 131072 * 6144:
                x = rng.choice(("bf16", "bf16", "fp16"))
                return dict(op=op, M=M, N=N, K=K, x=x, y=rng.choice((x, x, "fp32")), bias=rng.random() < 0.3,
                            residual=rng.random() < 0.4)
    while True:
        H, E, I = 512 * rng.randint(1, 16), _log(rng, 8, 384), 128 * rng.randint(1, 4)
        if E * I * H <= 384 * 256 * 6144:
            return dict(op=op, M=rng.randint(1, 16), H=H, E=E, I=I, k=rng.randint(1, min(E, 8)),
                        w=rng.choice(("bf16", "fp32")), alike=rng.choice((0.0, 0.5, 0.8)))


def _active(c):
    """Distinct experts of a layer case, expected: every group of four tokens
    picks like 4 - 3 alike^2.5 independent ones."""
    eff = c["M"] if c["alike"] == 0 else 0.0
    if c["alike"]:
        m = c["M"]
        while m > 0:
            eff += 1 + (min(m, 4) - 1) * (1 - c["alike"] ** 2.5)
            m -= 4
    return c["E"] * (1 - (1 - c["k"] / c["E"]) ** eff)


def work(case):
    c = case
    b = {"bf16": 2, "fp16": 2, "fp32": 4}
    if c["op"] == "router":
        M, E, H = c["M"], c["E"], c["H"]
        return {"bytes": M * H * 2 + E * H * b[c["w"]] + 4 * M * E, "flops": 2 * M * E * H}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K // 2 + N * K // 32 + 2 * M * K + b[c["y"]] * M * N * (2 if c["residual"] else 1)
                + (b[c["x"]] * N if c["bias"] else 0), "flops": 2 * M * N * K}
    M, H, E, I, k = c["M"], c["H"], c["E"], c["I"], c["k"]
    return {"bytes": int(_active(c) * 3 * I * H * 17 / 32) + E * H * b[c["w"]] + 4 * M * H + 8 * M * k,
            "flops": 2 * M * E * H + 6 * M * k * I * H}


# ------------------------------------------------------------------ inputs
def _codes(gen, shape):
    """Random MXFP4 bytes: each nibble from a 256-entry table that holds the
    eight magnitudes at the shares below, half of them negative."""
    share = (0.081, 0.159, 0.147, 0.131, 0.162, 0.150, 0.118, 0.052)
    table = torch.zeros(256, dtype=torch.uint8)
    edges = [0]
    for s in share:
        edges.append(edges[-1] + s * 128)
    for i in range(256):
        mag = max(m for m in range(8) if edges[m] <= i % 128)
        table[i] = mag | (8 if i >= 128 else 0)
    table = table.to(DEV)
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for a in range(0, flat.numel(), step):
        n = min(step, flat.numel() - a)
        lo = torch.randint(0, 256, (n,), generator=gen, device=DEV, dtype=torch.int32)
        hi = torch.randint(0, 256, (n,), generator=gen, device=DEV, dtype=torch.int32)
        flat[a:a + n] = table[lo] | (table[hi] << 4)
    return out


def _scales(gen, shape):
    """E8M0 bytes 119, 120, 121 at shares .02, .92, .06."""
    u = torch.rand(shape, generator=gen, device=DEV)
    return (119 + (u > 0.02).to(torch.uint8) + (u > 0.94).to(torch.uint8)).to(torch.uint8)


def _inputs(c, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    if c["op"] == "router":
        return {"x": normal(c["M"], c["H"]).to(TYPES[c["x"]]),
                "w": (normal(c["E"], c["H"]) / math.sqrt(c["H"])).to(TYPES[c["w"]])}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        d = {"x": normal(M, K).to(TYPES[c["x"]]), "w": _codes(gen, (N, K // 2)), "s": _scales(gen, (N, K // 32))}
        d["bias"] = normal(N).to(TYPES[c["x"]]) if c["bias"] else None
        d["residual"] = normal(M, N).to(TYPES[c["y"]]) if c["residual"] else None
        return d
    M, H, E, I = c["M"], c["H"], c["E"], c["I"]
    base = normal((M + 3) // 4, H).repeat_interleave(4, 0)[:M]
    x = math.sqrt(c["alike"]) * base + math.sqrt(1 - c["alike"]) * normal(M, H)
    return {"x": x.to(torch.bfloat16), "rw": (normal(E, H) / math.sqrt(H)).to(TYPES[c["w"]]),
            "w13": _codes(gen, (E, 2 * I, H // 2)), "s13": _scales(gen, (E, 2 * I, H // 32)),
            "w2": _codes(gen, (E, H, I // 2)), "s2": _scales(gen, (E, H, I // 32))}


def prepare(case, seed):
    c = case
    d = dict(_inputs(c, seed), case=c, mag=torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV))
    if own:
        # what a program keeps: the weights laid out once, the plan with its
        # workspace, the output buffers
        from quantized_moe_expert_route_amd import binding as B

        if c["op"] == "router":
            d["router"] = B.Router(d["w"], x_dtype=TYPES[c["x"]], max_M=c["M"])
            d["out"] = torch.empty((c["M"], c["E"]), dtype=torch.float32, device=DEV)
        elif c["op"] == "linear":
            d["linear"] = B.Linear(d["w"], d["s"], bias=d["bias"], x_dtype=TYPES[c["x"]], max_M=c["M"])
            d["out"] = torch.empty((c["M"], c["N"]), dtype=TYPES[c["y"]], device=DEV)
            del d["w"], d["s"]
        else:
            d["plan"] = B.Plan(c["M"], c["H"], c["E"], c["I"], c["k"], SCALING)
            d["w13"], d["s13"] = B.pack_w13(d["w13"], d["s13"])
            d["router"] = B.Router(d["rw"], x_dtype=torch.bfloat16, max_M=c["M"])
            d["out"] = torch.empty((c["M"], c["H"]), dtype=torch.bfloat16, device=DEV)
            d["ids"] = d["plan"].view("topk_ids", torch.int32, (c["M"], c["k"]))
    return d


# ------------------------------------------------------------------ plain form
def _dequant(mag, q, s):
    """MXFP4 codes [..., n/2] and E8M0 scales [..., n/32] -> fp32 [..., n] (the
    scale byte is the exponent field of a power of two; exact)."""
    v = torch.stack((mag[(q & 15).int()], mag[(q >> 4).int()]), -1)
    scale = (s.int() << 23).view(torch.float32)
    return (v.view(*s.shape, 32) * scale[..., None]).view(*q.shape[:-1], 2 * q.shape[-1])


def _plain_layer(d):
    c = d["case"]
    M, k, I = c["M"], c["k"], c["I"]
    # 64 bits: two logits next to the selection's border must not swap places
    logits = (d["x"].double() @ d["rw"].double().t()).float()
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    sig = (1 / (1 + torch.exp(-top.double()))).float()
    w = sig / (sig.sum(1, keepdim=True) + 1e-20) * SCALING
    e = ids.reshape(-1)
    x = d["x"].float().repeat_interleave(k, 0)[:, :, None]
    gu = (_dequant(d["mag"], d["w13"][e], d["s13"][e]) @ x)[:, :, 0]
    h = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
    y = (_dequant(d["mag"], d["w2"][e], d["s2"][e]) @ h[:, :, None])[:, :, 0]
    out = (y.view(M, k, -1) * w[:, :, None]).sum(1)
    return out.to(torch.bfloat16), ids.int()


def run(state):
    d, c = state, state["case"]
    if own:
        if c["op"] == "router":
            return d["router"].forward(d["x"], d["out"])
        if c["op"] == "linear":
            return d["linear"].forward(d["x"], d["out"], residual=d["residual"])
        return d["plan"].layer(d["x"], d["router"], d["w13"], d["s13"], d["w2"], d["s2"], d["out"]), d["ids"]
    if c["op"] == "router":
        return d["x"].float() @ d["w"].float().t()
    if c["op"] == "linear":
        y = d["x"].float() @ _dequant(d["mag"], d["w"], d["s"]).t()
        if d["bias"] is not None:
            y = y + d["bias"].float()
        if d["residual"] is not None:
            y = y + d["residual"].float()
        return y.to(TYPES[c["y"]])
    return _plain_layer(d)


# ------------------------------------------------------------------ 64 bits
def _value(q, s):
    """The 64-bit values, from the bits: sign, two exponent bits, one mantissa
    bit (exponent bits 0: the mantissa alone is a half)."""
    n = torch.stack((q % 16, q // 16), -1).reshape(*q.shape[:-1], -1).long()
    e, m = (n // 2) % 4, (n % 2).double()
    mag = torch.where(e > 0, (1 + m / 2) * torch.pow(2.0, (e - 1).double()), m / 2)
    mag = torch.where(n >= 8, -mag, mag)
    return mag * torch.pow(2.0, s.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    c, d = case, _inputs(case, seed)
    x = d["x"].double()
    if c["op"] == "router":
        return x @ d["w"].double().t()
    if c["op"] == "linear":
        y = torch.cat([x @ _value(q, s).t() for q, s in zip(d["w"].split(8192), d["s"].split(8192))], 1)
        y = y if d["bias"] is None else y + d["bias"].double()
        return y if d["residual"] is None else y + d["residual"].double()
    M, k, I = c["M"], c["k"], c["I"]
    logits = (x @ d["rw"].double().t()).cpu().tolist()
    out = torch.zeros((M, c["H"]), dtype=torch.float64, device=DEV)
    for t in range(M):
        pick = sorted(range(c["E"]), key=lambda e: (-logits[t][e], e))[:k]
        sig = [1 / (1 + math.exp(-logits[t][e])) for e in pick]
        for e, g in zip(pick, sig):
            gu = _value(d["w13"][e], d["s13"][e]) @ x[t]
            h = gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]
            out[t] += SCALING * g / sum(sig) * (_value(d["w2"][e], d["s2"][e]) @ h)
    return out, None
