"""The 64-bit references of the 16-bit layers and of the head's operators: their
gradients against differences of their values. No GPU."""

import math

import pytest
import torch

import dense_ref as R


def _differences(f, v, h=1e-6):
    """Central differences of a scalar function by every element of v."""
    out = torch.zeros_like(v)
    flat, o = v.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + h
        hi = f()
        flat[i] = keep - h
        lo = f()
        flat[i] = keep
        o[i] = (hi - lo) / (2 * h)
    return out


def _close(a, b):
    assert torch.allclose(a, b, rtol=1e-6, atol=1e-7), (a - b).abs().max()


@pytest.mark.parametrize("name", R.ACTS)
def test_dense_gradients(name):
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    x, w, b, res, dy = n(3, 8), n(5, 8), n(5), n(3, 5), n(3, 5)
    f = lambda: (R.dense(x, w, b, name, res, "bf16", "bf16")[0] * dy).sum().item()
    z = R.dense(x, w, b, name, res, "bf16", "bf16")[2]
    (dx, _), (dw, _), (db, _) = R.dense_backward(dy, z, x, w, name, "bf16")
    _close(dx, _differences(f, x))
    _close(dw, _differences(f, w))
    _close(db, _differences(f, b))
    _close(dy, _differences(f, res))


@pytest.mark.parametrize("name", R.ACTS[1:])
def test_gated_gradients(name):
    gen = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    x, w, dh = n(3, 8), n(10, 8), n(3, 5)
    f = lambda: (R.gated(x, w, name, "bf16")[0] * dh).sum().item()
    (dx, _), (dw, _) = R.gated_backward(dh, R.gated(x, w, name, "bf16")[2], x, w, name, "bf16")
    _close(dx, _differences(f, x))
    _close(dw, _differences(f, w))


@pytest.mark.parametrize("T", [1.0, 2.0, 0.7])
def test_distill_gradients(T):
    """Empty slots, a row of none, a token in two slots."""
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)
    z, t, weight = n(4, 9), n(4, 3), n(4).abs()
    ids = torch.tensor([[1, 4, 7], [2, -1, 2], [-1, -1, 9], [0, 8, -1]], dtype=torch.int32)
    f = lambda: (R.distill(z, ids, t, weight, T)[0] * weight).sum().item()
    loss, _, grad, _ = R.distill(z, ids, t, weight, T)
    _close(grad, _differences(f, z))
    assert loss[2] == 0 and (grad[2] == 0).all()
    # a token in two slots: the same loss as the divergence of the two slots' parts by hand
    p = torch.softmax(t[1, [0, 2]] / T, 0)
    lq = torch.log_softmax(z[1] / T, 0)[2]
    assert abs(loss[1] - (p * (torch.log(p) - lq)).sum()) < 1e-12


def test_scores_definition():
    z = torch.tensor([[0.0, 2.0, 2.0, -math.inf], [1.0, 1.0, 1.0, 1.0]], dtype=torch.float64)
    s = R.scores(z, torch.tensor([2, 4], dtype=torch.int32), 3)
    total = 1 + 2 * math.exp(2.0)
    assert abs(s["logprobs"][0][0] - math.log(math.exp(2.0) / total)) < 1e-12 and math.isnan(s["logprobs"][0][1])
    p = [1 / total, math.exp(2.0) / total, math.exp(2.0) / total]
    assert abs(s["entropy"][0][0] + sum(v * math.log(v) for v in p)) < 1e-12
    assert abs(s["entropy"][0][1] - math.log(4)) < 1e-12
    assert s["ids"].tolist() == [[1, 2, 0], [0, 1, 2]]
