"""64-bit references of the layers in 16 bits and of the operators on the output
head's logits, in torch on the CPU, from their formulas, with bounds on what
binary32 arithmetic may be off."""

from __future__ import annotations

import math

import torch

from ops_ref import half_step, sum_error

U = 2.0 ** -24  # half a step of binary32, relative
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s + z * s * (1 - s)
    if name == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z ** 3))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


# Activations and slopes in binary32: sigmoid and the normal distribution function
# within 8 roundings of values up to 1 (of an exponent's argument a: a more, with
# a s (1 - s) < 1), the products with z within 4 more of values up to |z|.
def act_error(z):
    return 16 * U * z.abs()


def slope_error(z):
    return 16 * U * (1 + z.abs())


MAX_SLOPE = 1.13  # of all activations; gelu's is 1.129


def rounding(t, v):
    """One rounding to type t: half a step, of fp16 at least half a subnormal one."""
    return half_step(t) * v.abs() + (2.0 ** -25 if t == "fp16" else 2.0 ** -134)


def dense(x, w, bias, name, residual, t, yt, pt=None):
    """(y, bound, z, bound of z saved in type pt, t by itself)."""
    pt = pt or t
    z, mag = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, mag = z + bias, mag + bias.abs()
    ez = sum_error(x.shape[1]) * mag
    y = act(name, z)
    ey = ez if name == "none" else MAX_SLOPE * ez + act_error(z.abs() + ez)
    if residual is not None:
        y = y + residual
        ey = ey + U * (y.abs() + ey)
    return y, ey * (1 + half_step(yt)) + rounding(yt, y), z, ez * (1 + half_step(pt)) + rounding(pt, z)


def products(dz, edz, x, w, t):
    """dx = dz w and dw = dz^T x with their bounds, for dz off by up to edz."""
    out = []
    for a, ea, b in ((dz, edz, w), (dz.T, edz.T, x)):
        v, mag = a @ b, (a.abs() + ea) @ b.abs()
        err = ea @ b.abs() + sum_error(a.shape[1]) * mag
        out.append((v, err * (1 + half_step(t)) + rounding(t, v)))
    return out


def dense_backward(dy, pre, x, w, name, t):
    """[(dx, bound), (dw, bound), (dbias, bound)]"""
    dz = dy * slope(name, pre) if name != "none" else dy
    raw = torch.zeros_like(dz) if name == "none" else dy.abs() * slope_error(pre) + U * dz.abs()
    edz = raw if name == "none" else raw * (1 + half_step(t)) + rounding(t, dz)
    db = dz.sum(0)
    eb = raw.sum(0) + sum_error(32 * dz.shape[0]) * (dz.abs() + raw).sum(0)
    return products(dz, edz, x, w, t) + [(db, eb * (1 + half_step(t)) + rounding(t, db))]


def gated(x, w13, name, t, pt=None):
    """(h, bound, pre, bound of pre in type pt, t by itself)."""
    pt = pt or t
    gu, mag = x @ w13.T, x.abs() @ w13.abs().T
    e = sum_error(x.shape[1]) * mag
    (g, u), (eg, eu) = gu.chunk(2, 1), e.chunk(2, 1)
    a = act(name, g)
    ea = MAX_SLOPE * eg + act_error(g.abs() + eg)
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + U * h.abs()
    return h, eh * (1 + half_step(t)) + rounding(t, h), gu, e * (1 + half_step(pt)) + rounding(pt, gu)


def gated_backward(dh, pre, x, w13, name, t):
    """[(dx, bound), (dw13, bound)]"""
    g, u = pre.chunk(2, 1)
    dg, du = dh * u * slope(name, g), dh * act(name, g)
    dz = torch.cat((dg, du), 1)
    raw = torch.cat(((dh * u).abs() * slope_error(g) + 2 * U * dg.abs(), dh.abs() * act_error(g) + U * du.abs()), 1)
    return products(dz, raw * (1 + half_step(t)) + rounding(t, dz), x, w13, t)


# ------------------------------------------------------------------ the head
def lse_error(z, lse):
    """Of log sum exp of rows z: an exponent's argument off by 2 U of itself, exp by 4
    U, sums in chains of at most V/256 + 64, the result rounded once."""
    q = torch.softmax(z, 1)
    far = (lse[:, None] - z).clamp(min=0)
    mean = torch.where(q > 0, q * far, 0.0).sum(1)
    return U * (2 * mean + 4 + z.shape[1] / 256 + 64)


def scores(z, tokens, k):
    """lse, logprobs, entropy, top logprobs, top ids and the bounds of the first four."""
    lse = torch.logsumexp(z, 1)
    lq = torch.log_softmax(z, 1)
    ok = (tokens >= 0) & (tokens < z.shape[1])
    lp = torch.where(ok, lq.gather(1, tokens.clamp(0, z.shape[1] - 1).long()[:, None])[:, 0], math.nan)
    q = torch.exp(lq)
    ent = -torch.where(q > 0, q * lq, 0.0).sum(1)
    ids = torch.from_numpy((-z.numpy()).argsort(axis=1, kind="stable"))[:, :k]
    top = lq.gather(1, ids)
    e = lse_error(z, lse)
    # the entropy's sum: of terms q |log q|, each off by a few U (1 + |log q|)
    mag = torch.where(q > 0, q * (1 + lq.abs()) ** 2, 0.0).sum(1)
    ee = 2 * e + U * (8 + z.shape[1] / 256 + 64) * (mag + 1)
    rnd = lambda v: U * v.abs() + 2.0 ** -149
    return dict(lse=(lse, e + rnd(lse)), logprobs=(lp, e + rnd(lp)), entropy=(ent, ee + rnd(ent)),
                top=(top, e[:, None] + rnd(top)), ids=ids.int())


def distill(z, ids, t, weight, T):
    """loss and gradient with their bounds (of the gradient before its rounding)."""
    M, V = z.shape
    held = (ids >= 0) & (ids < V) & (t != -math.inf)
    some = held.any(1)
    s = torch.where(held, t / T, -math.inf)
    p = torch.softmax(torch.where(some[:, None], s, 0.0), 1) * some[:, None]
    lse = torch.logsumexp(z / T, 1)
    lq = torch.log_softmax(z / T, 1)
    at = lq.gather(1, torch.where(held, ids, 0).long())
    lp = torch.where(p > 0, torch.log(p), 0.0)
    loss = torch.where(p > 0, p * (lp - at), 0.0).sum(1)
    el = lse_error(z / T, lse) + U * 2 * lse.abs()
    mag = torch.where(p > 0, p * (lp.abs() + at.abs() + lse.abs()[:, None] + (t / T).abs()), 0.0).sum(1)
    q = torch.exp(lq) * some[:, None]
    target = torch.zeros_like(z).scatter_add_(1, torch.where(held, ids, 0).long(), p)
    f = (weight / T)[:, None]
    grad = f * (q - target)
    # (an exponential below the least normal number 2^-126 may come as 0, before f multiplies it)
    eg = f.abs() * (2.0 ** -126 + q * (el[:, None] + U * (8 + 4 * lq.abs().clamp(max=1e4) + 4 * lse.abs()[:, None])) + 16 * U * target) + 4 * U * grad.abs()
    return loss, torch.where(some, el + 16 * U * (mag + 1), 0.0), grad, torch.where(some[:, None], eg, 0.0)
