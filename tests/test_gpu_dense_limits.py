"""The 16-bit layers at far arguments: infinities, given or from sums past the saved
type's range."""

import math

import pytest
import torch

import dense_ref as R
from test_gpu_dense import DT, _backward, _case, _dense, _f64, _forward, _nan, _within, _ws

pytestmark = pytest.mark.gpu

BIG = 131072.0  # = 64 products of 32 and 64, past fp16's 65504


@pytest.mark.parametrize("act", R.ACTS[1:])
def test_saved_past_the_range(act):
    """Sums of +-131072 are saved in fp16 as infinities; y (in 32 bits) and all
    gradients are those of the sums: slopes 0 and 1."""
    d = _case(5, 20, 48, 64, "fp16", act, yt="fp32", bias=False)
    d["x"][3:7] = 32.0
    d["w"][5:9], d["w"][11] = -64.0, 64.0
    op = _dense(d)
    y, pre = _forward(d, op)
    ye, bound, z, _ = R.dense(_f64(d["x"]), _f64(d["w"]), None, act, _f64(d["residual"]), "fp16", "fp32")
    assert (z[3:7, 5:9] == -BIG).all() and pre.cpu()[3:7, 5:9].isneginf().all() and pre.cpu()[3:7, 11].isposinf().all()
    _within(y, ye, bound, "y")
    assert torch.equal(y.cpu()[3:7, 5:9], d["residual"][3:7, 5:9])
    bounded = pre.cpu().clamp(-100, 100).double()  # (the same slopes to 2^-100)
    grads = R.dense_backward(_f64(d["dy"]), bounded, _f64(d["x"]), _f64(d["w"]), act, "fp16")
    for got, (want, e), what in zip(_backward(d, op, pre), grads, ("dx", "dw", "dbias")):
        _within(got, want, e, what)


@pytest.mark.parametrize("act", R.ACTS[1:])
@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_infinite_bias(t, act):
    """z of -inf: y and slope 0; of +inf: y infinite, slope 1. NaN stays."""
    d = _case(6, 20, 48, 64, t, act, residual=False)
    d["bias"][4], d["bias"][5], d["bias"][6] = -math.inf, math.inf, math.nan
    d["pt"] = "fp32"
    op = _dense(d)
    y, pre = _forward(d, op)
    assert (y[:, 4] == 0).all() and y[:, 5].isposinf().all() and y[:, 6].isnan().all() and pre[:, 6].isnan().all()
    pre[:, 6] = 0.25
    bounded = pre.cpu().clamp(-100, 100).double()  # (the same slopes to 2^-100)
    grads = R.dense_backward(_f64(d["dy"]), bounded, _f64(d["x"]), _f64(d["w"]), act, t)
    for got, (want, e), what in zip(_backward(d, op, pre), grads, ("dx", "dw", "dbias")):
        _within(got, want, e, what)


@pytest.mark.parametrize("act", R.ACTS[1:])
@pytest.mark.parametrize("pt", ["fp16", "fp32"])
def test_gated_past_the_range(act, pt):
    """Gates of -131072 pass nothing, whatever stands beside them: h and the gradients of
    both projections are 0 there."""
    from quantized_moe_expert_route_amd.binding import Gated

    M, I, H = 37, 40, 64
    gen = torch.Generator().manual_seed(8)
    x = torch.full((M, H), 32.0, dtype=torch.float16)
    w = (torch.randn(2 * I, H, generator=gen) / 256).to(torch.float16)
    dh = torch.randn(M, I, generator=gen).to(torch.float16)
    shut = [0, 1, 3]
    w[shut] = -64.0
    w[I + 1], w[I + 3] = 64.0, -64.0
    op = Gated(w.cuda(), activation=act)
    h, pre = _nan((M, I), torch.float16), _nan((M, 2 * I), DT[pt])
    ws = _ws(op.workspace_bytes(M, train=True))
    op.forward(x.cuda(), h, pre=pre, workspace=ws)
    assert (h[:, shut] == 0).all()
    dx, dw = _nan((M, H), torch.float16), _nan((2 * I, H), torch.float16)
    op.backward(dh.cuda(), x.cuda(), pre, dx=dx, dw=dw, workspace=ws)
    rows = shut + [I + s for s in shut]
    assert (dw[rows] == 0).all()
    keep = [i for i in range(I) if i not in shut]  # the shut ones add nothing to dx
    both = torch.tensor(keep + [I + i for i in keep])
    (want, bound), _ = R.gated_backward(_f64(dh[:, keep]), _f64(pre.cpu()[:, both]), _f64(x), _f64(w[both]), act, "fp16")
    _within(dx, want, bound, "dx")
    dh[5, 1], dh[6, 3] = math.nan, math.inf  # a gradient that is none stays none
    op.backward(dh.cuda(), x.cuda(), pre, dx=dx, dw=dw, workspace=ws)
    assert dx[5:7].isnan().all() and not dx[:5].isnan().any() and dw[[1, 3, I + 1, I + 3]].isnan().all()


# Relative errors of the activations' lower tails in binary32, in U. silu and gelu_tanh: an
# exponent's argument a off by 2 (z's product, the constant) or 6 (2u besides, of four more
# roundings) of itself, the exponential, reciprocal, sum and product by 8. gelu: as beside
# its code.
TAILS = {
    "silu": (-80.0, lambda z: 8 + 2 * z.abs()),
    "gelu": (-12.5, lambda z: 12 + 2 * z * z),
    "gelu_tanh": (-9.5, lambda z: 8 + 7 * (1.6 * z.abs() + 0.0714 * z.abs() ** 3)),
}


@pytest.mark.parametrize("act", list(TAILS))
@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("wide", [False, True])
def test_lower_tail(t, act, wide):
    """act(z) of negative z, which falls to the least numbers, to its own size."""
    from quantized_moe_expert_route_amd.binding import Dense

    low, units = TAILS[act]
    M = 3001
    x = torch.zeros(M, 8, dtype=DT[t])
    x[:, 0] = torch.cat((torch.linspace(low, -1.0, 2000), -torch.logspace(-5, 0, 1001))).to(DT[t])
    w = torch.zeros(1, 8, dtype=DT[t])
    w[0, 0] = 1.0  # z = x
    yt = "fp32" if wide else t
    y = _nan((M, 1), DT[yt])
    Dense(w.cuda(), activation=act).forward(x.cuda(), y)
    z = x[:, :1].double()
    want = R.act(act, z)  # (gelu by erfc; torch's ndtr is 1 + erf, which cancels here)
    if act == "gelu_tanh":  # (1 + tanh u) / 2 would cancel
        want = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    bound = (units(z) * R.U * (1 + R.half_step(yt))) * want.abs() + R.rounding(yt, want)
    _within(y, want, bound, act)
