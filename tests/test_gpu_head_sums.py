"""Long sums of the output head's operators: rows of many like logits, whose sums have
closed forms, by one workgroup a row."""

import math

import pytest
import torch

import dense_ref as R
from test_gpu_head import DT

pytestmark = pytest.mark.gpu

M = 520  # more than two rows a CU: no row is split


def _rows(kind, t, V):
    """z [M, V] on the GPU, log sum exp z and the entropy, by their closed forms."""
    z = torch.zeros(M, V, dtype=DT[t], device="cuda")
    if kind == "like":  # every thread's first elements pass the others, which add exp(-0.7) each
        d, n = 0.69921875, 16384
        z[:, :n] = d
        top, total = d, n + (V - n) * math.exp(-d)
        mean = (V - n) * math.exp(-d) * -d / total
    else:  # rising by 2^-20 a token: sums of exp(-i h), i < V
        h = 2.0 ** -20
        z[:] = torch.arange(V, device="cuda") * h
        top, x, V1 = (V - 1) * h, math.exp(-h), math.exp(-V * h)
        total = -math.expm1(-V * h) / -math.expm1(-h)
        mean = -h * (x * (1 - V * V1 / x + (V - 1) * V1) / (1 - x) ** 2) / total
    return z, top + math.log(total), math.log(total) - mean, -mean


def _checked(got, want, units):
    assert got.isfinite().all()
    off = (got.double() - want).abs().max().item() / R.U
    assert off <= units, (off, units)


# An exponential's argument is off by 4 U of itself (of |z - m|, whose mean is `mean` and 6
# log 2 more where m lags), the exponential by 2 U, 16 of them added by 16, the sums of
# sixteens, carried, by 4; the rest is in 64 bits and rounded once.
def _units(mean):
    return 24 + 4 * (mean + 4.2)


CASES = [("like", "bf16", 1 << 24), ("like", "fp16", 3000001), ("rising", "fp32", 1 << 22)]


@pytest.mark.parametrize("kind,t,V", CASES)
@pytest.mark.parametrize("k", [0, 1])
def test_scores(kind, t, V, k):
    from quantized_moe_expert_route_amd.binding import TokenScores

    z, lse, entropy, mean = _rows(kind, t, V)
    op = TokenScores(V, top_k=k, dtype=DT[t])
    assert op.workspace_bytes(M) == 0  # a row a workgroup
    tokens = torch.full((M,), V - 1, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.full(s, math.nan, device="cuda")
    lp, ent, ls, top, ids = f(M), f(M), f(M), f(M, 1), torch.full((M, 1), -1, dtype=torch.int32, device="cuda")
    op.forward(z, tokens, lp, entropy=ent, lse=ls, **(dict(top_logprobs=top, top_ids=ids) if k else {}))
    last, first = z[0, V - 1].double().item(), z[0].max().double().item()
    _checked(ls, lse, _units(mean) + abs(lse))
    _checked(lp, last - lse, _units(mean) + abs(last - lse))
    # (terms q |log q| of the entropy move with the exponents' errors once more)
    _checked(ent, entropy, 2 * _units(mean) * (1 + mean) + abs(entropy))
    if k:
        _checked(top, first - lse, _units(mean) + abs(first - lse))
        assert (ids == (0 if kind == "like" else V - 1)).all()


@pytest.mark.parametrize("kind,t,V", CASES)
@pytest.mark.parametrize("fused", [False, True])
def test_distill(kind, t, V, fused):
    """One slot: the loss is the token's, minus its log probability; the gradient in 16 or 32
    bits of two stretches against its closed form."""
    from quantized_moe_expert_route_amd.binding import Distill

    z, lse, _, mean = _rows(kind, t, V)
    op = Distill(V, 1, dtype=DT[t])
    ids = torch.full((M, 1), V - 1, dtype=torch.int32, device="cuda")
    tl, weight = torch.zeros(M, 1, device="cuda"), torch.full((M,), float(1 << 20), device="cuda")
    loss, ls, ws = torch.empty(M, device="cuda"), torch.empty(M, device="cuda"), torch.empty(max(op.workspace_bytes(M), 256), dtype=torch.uint8, device="cuda")
    last = z[0, V - 1].double().item()
    parts = [slice(0, 1000), slice(V - 1001, V - 1)]
    want = [torch.exp(z[:1, p].double() - lse) * (1 << 20) for p in parts]
    if fused:
        op.forward_backward(z, ids, tl, weight, loss, z, workspace=ws)
    else:
        op.forward(z, ids, tl, loss, lse=ls, workspace=ws)
        _checked(ls, lse, _units(mean) + abs(lse))
        op.backward(z, ids, tl, ls, weight, z)
    _checked(loss, lse - last, _units(mean) + abs(lse - last) + 1)
    for p, w in zip(parts, want):
        # (an exponent again; lse rounded to 32 bits where it was saved)
        rel = R.U * (_units(mean) + 8 + 4 * mean + 2 * abs(lse))
        assert ((z[:, p].double() - w).abs() <= rel * w + R.rounding(t, w)).all()
