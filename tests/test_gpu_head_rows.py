"""Rows of the output head's operators that are few and long, many and held in registers,
written over, or of nothing but the lowest number."""

import math

import pytest
import torch

import dense_ref as R
from test_gpu_head import DT, INF, _check_distill, _check_scores, _distill, _logits, _place, _scores, _teacher, _within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,V", [("bf16", 40001), ("bf16", 70001), ("fp16", 131072), ("fp32", 20003), ("fp32", 40004), ("fp32", 65536)])
@pytest.mark.parametrize("M,in_place", [(300, True), (530, False)])
def test_held_rows(t, V, M, in_place):
    """More rows than CUs."""
    z, gen = _logits(V, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 33)
    _check_distill(z, ids, tl, weight, 2.0, _distill(z.cuda(), ids, tl, weight, 2.0, fused=True, in_place=in_place), t)


@pytest.mark.parametrize("t,M,V", [("bf16", 500, 40001), ("bf16", 1000, 40001), ("bf16", 500, 70001), ("fp16", 512, 131072),
                                   ("fp32", 1000, 20003), ("fp32", 500, 40004), ("fp32", 700, 65536)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rounds_of_rows(t, M, V, in_place):
    """One to three rounds of rows over the workgroups."""
    z, gen = _logits(V, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 9)
    _check_distill(z, ids, tl, weight, 2.0, _distill(z.cuda(), ids, tl, weight, 2.0, fused=True, in_place=in_place), t)


@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["normal", "ties", "rising", "falling", "masked", "lowest", "one"])
def test_alternatives_of_many_long_rows(t, kind):
    M, V = 258, 33001
    z, gen = _logits(7, M, V, t, kind)
    for k in (1, 64):
        _check_scores(z, torch.randint(0, V, (M,), generator=gen).int(), k)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_rows_not_alike(t):
    """Many long rows whose gradient lies otherwise than they do."""
    M, V = 290, 36001
    z, gen = _logits(1, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 5)
    _, view = _place(z, V + 3, 1)
    _check_distill(z, ids, tl, weight, 1.0, _distill(view, ids, tl, weight, 1.0, fused=True), t)


@pytest.mark.parametrize("M,V", [(1, 70001), (2, 300007), (90, 100003), (40, 20001)])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_few_rows_in_place(M, V, fused, t):
    z, gen = _logits(2, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 20)
    _check_distill(z, ids, tl, weight, 1.5, _distill(z.cuda(), ids, tl, weight, 1.5, fused=fused, in_place=True), t)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_longest_row(t):
    V = 1 << 24
    z, gen = _logits(3, 1, V, t)
    z[0, V - 1], z[0, 5] = 40.0, 41.0
    _check_scores(z, torch.tensor([V - 1], dtype=torch.int32), 64)
    ids, tl, weight = _teacher(gen, 1, V, 64)
    ids[0, :2] = torch.tensor([V - 1, 5], dtype=torch.int32)
    tl[0, :2] = 1.0
    for fused in (False, True):
        _check_distill(z, ids, tl, weight, 1.0, _distill(z.cuda(), ids, tl, weight, 1.0, fused=fused), t)


SIZES = [(1, 3), (5, 500), (3, 30011), (2, 131072), (300, 5003), (300, 20011)]


@pytest.mark.parametrize("M,V", SIZES)
@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
def test_rows_of_the_lowest_number(M, V, t):
    """A mask of the type's lowest number that leaves nothing: all tokens are alike. The log
    probability is -log V, off by its rounding and the logarithm's; the gradient, of an
    exact sum V, by the roundings of 1/T, weight/T, the quotient and q (4) and p's (16)."""
    z = torch.full((M, V), torch.finfo(DT[t]).min, dtype=DT[t])
    gen = torch.Generator().manual_seed(M)
    tokens = torch.randint(0, V, (M,), generator=gen).int()
    k = min(V, 7)
    o = _scores(z.cuda(), tokens, k)
    want = torch.full((M,), -math.log(V), dtype=torch.float64)
    _within(o["logprobs"], want, 2 * R.U * want.abs(), "logprobs")
    _within(o["entropy"], -want, 2 * R.U * want.abs(), "entropy")
    _within(o["top"], want[:, None].expand(M, k), 2 * R.U * want.abs()[:, None], "top")
    assert torch.equal(o["ids"].cpu(), torch.arange(k).int().expand(M, k))
    ids, tl, weight = _teacher(gen, M, V, 4)
    tl = torch.where(tl == -INF, -1.0, tl)
    for T in (0.5, 1.0, 3.0):
        some = (ids >= 0).any(1).double()
        p = torch.softmax(torch.where(ids >= 0, tl.double() / T, -INF), 1).nan_to_num(0.0)  # (NaN: no slot)
        target = torch.zeros(M, V, dtype=torch.float64).scatter_add_(1, ids.clamp(min=0).long(), p)
        f = weight.double()[:, None] / T
        q = some[:, None] / V
        grad = f * (q - target)
        loss = torch.where(p > 0, p * p.clamp(min=1e-300).log(), 0.0).sum(1) + some * math.log(V)
        for fused in (False, True):
            gl, gg = _distill(z.cuda(), ids, tl, weight, T, fused=fused)
            _within(gl, loss, R.U * (16 + loss.abs() + math.log(V)), "loss")
            _within(gg, grad, 1.01 * f * R.U * (4 * q + 16 * target) + R.rounding(t, grad), "grad")


@pytest.mark.parametrize("T", [1e-6, 1e-3, 0.02])
@pytest.mark.parametrize("M,V", [(3, 300), (2, 70001), (300, 9001)])
def test_small_temperatures(M, V, T):
    """lse of hundreds to millions, whose rounding would show in the gradient: both forms
    within the arithmetic's bound that counts lse from the largest logit."""
    gen = torch.Generator().manual_seed(V)
    # steps of T / 4 below one token, so that several tokens share the probability
    z = (1.0 - torch.randint(0, 4000, (M, V), generator=gen).double() * (T / 4)).float()
    z[:, V // 3] = 1.0
    ids, tl, weight = _teacher(gen, M, V, 6)
    tl = torch.where(tl == -INF, -1.0, tl) * T
    Tf = float(torch.tensor(T, dtype=torch.float32))
    c = 1.0 / Tf
    for fused in (False, True):
        got = _distill(z.cuda(), ids, tl, weight, T, fused=fused)
        loss, _, grad, _ = R.distill(z.double(), ids, torch.where(ids >= 0, tl.double(), 0.0), weight.double(), Tf)
        # an exponent x = (z - m) / T is off by 4 U |x| (1/T, log2 e, the difference, the
        # product), e^x by that and U; sums as a logarithm's. e^x itself may come as 0 below
        # the least normal number 2^-126, before weight / T multiplies it
        lq = torch.log_softmax(z.double() / Tf, 1)
        x = ((z.double() - z.double().max(1, True)[0]) * c).abs()
        q = lq.exp()
        off = U_of(q, x, V)
        f = weight.double()[:, None] * c
        slot = torch.zeros(M, V, dtype=torch.float64).scatter_add_(
            1, ids.clamp(min=0).long(), torch.where(ids >= 0, (tl.double() / Tf).abs().nan_to_num(0.0, 0.0, 0.0) + 1, 0.0))
        some = (ids >= 0).any(1).double()
        eg = f * some[:, None] * (q * (off + R.U * (8 + 4 * x)) + 2.0 ** -126 + 16 * R.U * slot) + 4 * R.U * grad.abs()
        _within(got[1], grad, 1.01 * eg + R.rounding("fp32", grad), "grad")


def U_of(q, x, V):
    """Relative error of a row's sum."""
    return R.U * (4 * (q * x).sum(1, keepdim=True) + 8 + V / 256 + 64)


@pytest.mark.parametrize("M,V", [(5, 300), (3, 70001), (300, 9001), (300, 20001)])
@pytest.mark.parametrize("fused", [False, True])
def test_teachers_of_minus_infinity(M, V, fused):
    """Slots of t = -inf are empty: a row of nothing else has loss and gradient 0, whatever
    its logits hold."""
    z, gen = _logits(4, M, V, "fp32")
    ids = torch.randint(0, V, (M, 3), generator=gen).int()
    tl = torch.randn(M, 3, generator=gen) * 1e38
    tl[:, 1] = -INF
    tl[1::2] = -INF
    z[1, 0] = math.nan
    weight = torch.rand(M, generator=gen) + 0.5
    loss, grad = _distill(z.cuda(), ids, tl, weight, 0.25, fused=fused)
    assert (loss[1::2] == 0).all() and (grad[1::2] == 0).all()
    _check_distill(z[::2], ids[::2], tl[::2], weight[::2], 0.25, (loss[::2], grad[::2]), "fp32")
