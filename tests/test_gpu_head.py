"""Scores of given tokens and distillation on the GPU against their 64-bit
definitions."""

import math

import pytest
import torch

import dense_ref as R

pytestmark = pytest.mark.gpu

DT = R.DT
INF = math.inf


def _f32(*shape):
    return torch.full(shape, math.nan, device="cuda")


def _ws(n):
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")


def _within(got, want, bound, what=""):
    g = got.double().cpu()
    assert torch.equal(g.isnan(), want.isnan()), what
    same = g == want  # infinities
    bad = (~same & ~want.isnan() & ~((g - want).abs() <= bound)).nonzero()
    assert len(bad) == 0, (what, len(bad), bad[:4].tolist(), g[tuple(bad[0])], want[tuple(bad[0])])


def _logits(seed, M, V, t, kind="normal"):
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn(M, V, generator=gen) * 3
    if kind == "ties":
        z = torch.randint(-2, 3, (M, V), generator=gen).float()
    elif kind == "rising":
        z = torch.sort(z, dim=1)[0]
    elif kind == "falling":
        z = torch.sort(z, dim=1, descending=True)[0]
    elif kind == "masked":
        z[torch.rand(M, V, generator=gen) < 0.9] = -INF
        z[:, V // 2] = 0.5
    elif kind == "lowest":  # masked by the type's lowest value
        z[torch.rand(M, V, generator=gen) < 0.9] = torch.finfo(DT[t]).min
        z[:, V // 2] = 0.5
    elif kind == "one":
        z[:] = -INF
        z[torch.arange(M), torch.randint(0, V, (M,), generator=gen)] = 2.0
    elif kind == "far":
        z = z * 1e4 if t != "fp16" else z * 3e3
    return z.to(DT[t]), gen


def _place(z, ld=None, off=0):
    """z on the GPU with rows ld apart from element `off` on."""
    M, V = z.shape
    ld = ld or V
    buf = torch.full((off + M * ld,), math.nan, dtype=z.dtype, device="cuda")
    view = buf.as_strided((M, V), (ld, 1), off)
    view.copy_(z)
    return buf, view


def _scores(z, tokens, k, **kw):
    from quantized_moe_expert_route_amd.binding import TokenScores

    M, V = z.shape
    op = TokenScores(V, top_k=k, dtype=z.dtype, max_M=M)
    o = dict(logprobs=_f32(M), entropy=_f32(M), lse=_f32(M))
    if k:
        o.update(top=_f32(M, k), ids=torch.full((M, k), -7, dtype=torch.int32, device="cuda"))
    op.forward(z, tokens.cuda(), o["logprobs"], entropy=o["entropy"], lse=o["lse"], top_logprobs=o.get("top"),
               top_ids=o.get("ids"), workspace=_ws(op.workspace_bytes(M)), **kw)
    return o


def _check_scores(z, tokens, k, view=None):
    o = _scores(z.cuda() if view is None else view, tokens, k)
    want = R.scores(z.double(), tokens, k)
    if k:
        assert torch.equal(o["ids"].cpu(), want["ids"]), "ids"
    for name in ("lse", "logprobs", "entropy") + (("top",) if k else ()):
        _within(o[name], *want[name], name)


ROWS = [(1, 1), (1, 7), (3, 64), (2, 65), (5, 255), (1, 1000), (4, 4099), (17, 2048), (1, 131072), (2, 30011), (300, 515),
        (33, 8193), (1, 262144), (2, 400003), (300, 20011)]


@pytest.mark.parametrize("M,V", ROWS)
@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
def test_scores(M, V, t):
    for k in sorted({0, 1, min(V, 5), min(V, 64)}):
        z, gen = _logits(M + V + k, M, V, t)
        _check_scores(z, torch.randint(0, V, (M,), generator=gen).int(), k)


@pytest.mark.parametrize("kind", ["ties", "rising", "falling", "masked", "lowest", "one", "far"])
@pytest.mark.parametrize("t", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,V", [(3, 100), (2, 5003), (40, 3001), (1, 70001), (2, 350001), (260, 5001)])
def test_scores_distributions(kind, t, M, V):
    z, gen = _logits(V, M, V, t, kind)
    _check_scores(z, torch.randint(0, V, (M,), generator=gen).int(), 20)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("ld,off", [(1003, 0), (1003, 1), (1024, 3), (4000, 8)])
def test_scores_strides(t, ld, off):
    z, gen = _logits(ld + off, 9, 1000, t)
    buf, view = _place(z, ld, off)
    _check_scores(z, torch.randint(0, 1000, (9,), generator=gen).int(), 7, view)


def test_scores_bad_rows_and_tokens():
    """Rows that hold a NaN, +inf or nothing but -inf are NaN and disturb no other;
    so are tokens outside the vocabulary."""
    V, k = 3001, 4
    for M in (6, 200):
        z, _ = _logits(3, M, V, "fp32")
        z[0, 17], z[1, 5], z[2] = math.nan, INF, -INF
        z[4, 11] = -INF
        tokens = torch.tensor([0, 5, 1, -1, 11, V], dtype=torch.int32)
        tokens = torch.cat((tokens, torch.zeros(M - 6, dtype=torch.int32)))
        o = _scores(z.cuda(), tokens, k)
        lse = o["lse"].cpu()
        assert lse[0].isnan() and lse[1] == INF and lse[2] == -INF
        for name in ("logprobs", "entropy", "top"):
            assert o[name][:3].isnan().all(), name
        assert (o["ids"] >= 0).all() and (o["ids"] < V).all()
        want = R.scores(z[3:].double(), tokens[3:], k)
        assert torch.equal(o["ids"][3:].cpu(), want["ids"])
        for name in ("lse", "logprobs", "entropy", "top"):
            _within(o[name][3:], *want[name], name)
        assert o["logprobs"][3].isnan() and o["logprobs"][5].isnan() and o["logprobs"][4] == -INF


def test_scores_rows_past_M_stay_and_optional_outputs():
    from quantized_moe_expert_route_amd.binding import TokenScores

    z, _ = _logits(4, 10, 500, "bf16")
    op = TokenScores(500, top_k=3, dtype=torch.bfloat16, max_M=10)
    top, ids, lp = _f32(10, 3), torch.full((10, 3), -7, dtype=torch.int32, device="cuda"), _f32(10)
    ws = _ws(op.workspace_bytes(10))
    op.forward(z.cuda(), None, None, top_logprobs=top, top_ids=ids, workspace=ws, M=6)
    assert top[6:].isnan().all() and (ids[6:] == -7).all() and not top[:6].isnan().any()
    op.forward(z.cuda(), torch.zeros(10, dtype=torch.int32, device="cuda"), lp, top_logprobs=top, top_ids=ids, workspace=ws, M=0)
    assert lp.isnan().all()


# ------------------------------------------------------------------ distillation
def _teacher(gen, M, V, k):
    ids = torch.randint(0, V, (M, k), generator=gen).int()  # a token may come twice
    ids[torch.rand(M, k, generator=gen) < 0.2] = -1
    ids[3::5] = -1
    t = torch.randn(M, k, generator=gen) * 2
    if k > 2:
        t[:, 2] = -INF
    t[ids < 0] = math.nan  # not read
    return ids, t, torch.rand(M, generator=gen) + 0.1


def _distill(z, ids, t, weight, T, gt=None, fused=False, in_place=False):
    from quantized_moe_expert_route_amd.binding import Distill

    M, V = z.shape
    gt = gt or z.dtype
    op = Distill(V, ids.shape[1], dtype=z.dtype, grad_dtype=gt, temperature=T, max_M=M)
    loss, lse = _f32(M), _f32(M)
    grad = z if in_place else torch.full((M, V), math.nan, dtype=gt, device="cuda")
    ids, t, weight, ws = ids.cuda(), t.cuda(), weight.cuda(), _ws(op.workspace_bytes(M))
    if fused:
        op.forward_backward(z, ids, t, weight, loss, grad, workspace=ws)
    else:
        op.forward(z, ids, t, loss, lse, workspace=ws)
        op.backward(z, ids, t, lse, weight, grad)
    return loss, grad


def _name(dtype):
    return {v: k for k, v in DT.items()}[dtype]


def _check_distill(z, ids, t, weight, T, got, gt):
    loss, el, grad, eg = R.distill(z.double(), ids, torch.where(ids >= 0, t.double(), 0.0), weight.double(), T)
    _within(got[0], loss, el + R.U * loss.abs(), "loss")
    _within(got[1], grad, eg * 1.01 + R.rounding(gt, grad), "grad")


@pytest.mark.parametrize("M,V", ROWS)
@pytest.mark.parametrize("t,gt", [("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp16")])
def test_distill(M, V, t, gt):
    T = (1.0, 2.0, 0.7)[V % 3]
    for k in (1, 20, 64):
        z, gen = _logits(M + V + k, M, V, t)
        ids, tl, weight = _teacher(gen, M, V, k)
        for fused in (False, True):
            _check_distill(z, ids, tl, weight, T, _distill(z.cuda(), ids, tl, weight, T, DT[gt], fused), gt)


@pytest.mark.parametrize("kind", ["ties", "masked", "one", "far", "lowest"])
@pytest.mark.parametrize("M,V", [(6, 900), (40, 5001), (270, 17001)])
def test_distill_distributions(kind, M, V):
    for t in ("bf16", "fp32"):
        z, gen = _logits(V, M, V, t, kind)
        ids, tl, weight = _teacher(gen, M, V, 9)
        for fused in (False, True):
            _check_distill(z, ids, tl, weight, 1.0, _distill(z.cuda(), ids, tl, weight, 1.0, fused=fused), t)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("ld,off", [(2100, 0), (2101, 3), (2112, 8)])
def test_distill_in_place_and_strides(fused, t, ld, off):
    """dz over z itself; what lies between the rows stays."""
    M, V = 21, 2099
    z, gen = _logits(5, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 33)
    buf, view = _place(z, ld, off)
    loss, grad = _distill(view, ids, tl, weight, 1.0, fused=fused, in_place=True)
    _check_distill(z, ids, tl, weight, 1.0, (loss, grad), t)
    gap = torch.ones_like(buf, dtype=torch.bool)
    gap.as_strided((M, V), (ld, 1), off).fill_(False)
    assert buf[gap].isnan().all()


def test_distill_bad_rows():
    """NaN rows, weights of zero, padding rows of garbage."""
    V, M = 1000, 8
    z, gen = _logits(6, M, V, "fp32")
    ids = torch.randint(0, V, (M, 5), generator=gen).int()
    tl, weight = torch.randn(M, 5, generator=gen), torch.ones(M)
    z[0, 3], z[1, 4], z[2] = math.nan, INF, -INF
    z[3] = math.nan
    ids[3] = torch.tensor([-1, V, -5, 1 << 30, -(1 << 31)], dtype=torch.int64).int()
    weight[4] = 0.0
    for fused in (False, True):
        loss, grad = _distill(z.cuda(), ids, tl, weight, 1.0, fused=fused)
        assert loss[:3].isnan().all() and grad[:3].isnan().all()
        assert loss[3] == 0 and (grad[3] == 0).all() and (grad[4] == 0).all()
        want = R.distill(z[4:].double(), ids[4:], tl[4:].double(), weight[4:].double(), 1.0)
        _within(loss[4:], want[0], want[1] + R.U * want[0].abs())
        _within(grad[4:], want[2], want[3] * 1.01 + R.rounding("fp32", want[2]))
