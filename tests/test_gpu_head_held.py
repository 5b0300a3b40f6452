"""Distillation at once on rows that are held in registers between the sums and the
gradient: rows of every kind, layouts and types; each test says which kernel it is on."""

import math

import pytest
import torch

import dense_ref as R
import test_gpu_head_rows as rows
from test_gpu_head import DT, INF, _check_distill, _distill, _f32, _logits, _place, _scores, _teacher, _within, _ws

pytestmark = pytest.mark.gpu

HELD = "rows held in registers"
# up to 128 KB two rows a CU, above one; one and two rounds of rows over 256 CUs
SIZES = [("bf16", 500, 33001), ("fp16", 1000, 33000), ("bf16", 250, 66001), ("fp16", 500, 65544), ("fp32", 500, 16501), ("fp32", 250, 33002)]


def _kernel(t, M, V, k, gt=None):
    from quantized_moe_expert_route_amd.binding import Distill

    return Distill(V, k, dtype=DT[t], grad_dtype=DT[gt or t], max_M=M).kernel(M)


def _mixed(seed, M, V, t):
    """Row i of kind i % 9: the distributions, an infinity, a NaN, nothing but -inf."""
    kinds = ("normal", "ties", "rising", "falling", "masked", "one")
    z = torch.empty(M, V, dtype=DT[t])
    for i, kind in enumerate(kinds):
        part, gen = _logits(seed + i, len(range(i, M, 9)), V, t, kind)
        z[i::9] = part
    z[6::9], z[7::9], z[8::9] = z[0], z[0], -INF
    z[6::9, V // 3], z[7::9, V - 1] = INF, math.nan
    return z, gen


def _check(z, ids, tl, weight, T, got, gt):
    """Rows without a slot are 0 whatever they hold: their logits are no part of the definition."""
    filled = ((ids >= 0) & (ids < z.shape[1]) & (tl != -INF)).any(1)
    assert (got[0][~filled.cuda()] == 0).all() and (got[1][~filled.cuda()] == 0).all()
    _check_distill(torch.where(filled[:, None], z, torch.zeros((), dtype=z.dtype)), ids, tl, weight, T, got, gt)


@pytest.mark.parametrize("t,M,V", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_of_all_kinds(t, M, V, in_place):
    k = 33
    assert _kernel(t, M, V, k) == HELD
    z, gen = _mixed(V, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, k)
    weight[5::7] = 0.0
    weight[~(ids >= 0).any(1)] = math.nan  # not read
    ids[4::11, 3] = torch.tensor(V, dtype=torch.int32)
    tl[4::11, 3] = 1.0
    for T in (1.0, 0.6):
        _check(z, ids, tl, weight.nan_to_num(0.0), T, _distill(z.cuda(), ids, tl, weight, T, fused=True, in_place=in_place), t)


@pytest.mark.parametrize("t,M,V", [("bf16", 500, 33001), ("fp32", 250, 33002)])
def test_rows_of_the_lowest_number(t, M, V):
    assert _kernel(t, M, V, 4) == HELD
    rows.test_rows_of_the_lowest_number(M, V, t)


def test_teachers_of_minus_infinity():
    """Slots of t = -inf are empty; large differences of t."""
    M, V = 500, 16501
    assert _kernel("fp32", M, V, 3) == HELD
    z, gen = _logits(4, M, V, "fp32")
    ids = torch.randint(0, V, (M, 3), generator=gen).int()
    tl = torch.randn(M, 3, generator=gen) * 1e37
    tl[:, 1] = -INF
    tl[1::2] = -INF
    z[1, 0] = math.nan
    weight = torch.rand(M, generator=gen) + 0.5
    _check(z, ids, tl, weight, 0.25, _distill(z.cuda(), ids, tl, weight, 0.25, fused=True), "fp32")


@pytest.mark.parametrize("M,V", [(5, 901), (300, 5003), (500, 16501), (3, 70001)])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("bad", [math.nan, INF])
def test_teachers_without_a_number(M, V, fused, bad):
    """A slot of NaN or +inf: the row's loss and the gradient at its slots' tokens are NaN,
    the rest of the gradient is the logits' alone."""
    z, gen = _logits(4, M, V, "fp32")
    ids = (torch.arange(4) * (V // 4))[None].expand(M, 4).contiguous().int()
    tl, weight = torch.randn(M, 4, generator=gen), torch.rand(M, generator=gen) + 0.5
    tl[::2, 1] = bad
    ids[::2, 3] = -1
    loss, grad = _distill(z.cuda(), ids, tl, weight, 2.0, fused=fused)
    assert loss[::2].isnan().all() and grad[::2][:, ids[0, :3].long().cuda()].isnan().all()
    want = R.distill(z.double(), ids, tl.nan_to_num(0.0, 0.0).double(), weight.double(), 2.0)
    keep = torch.ones(V, dtype=torch.bool)
    keep[ids[0, :3].long()] = False
    for rows_, columns in ((slice(0, None, 2), keep), (slice(1, None, 2), slice(None))):
        _within(grad[rows_].cpu()[:, columns], want[2][rows_][:, columns], want[3][rows_][:, columns] * 1.01 + R.rounding("fp32", want[2][rows_][:, columns]))
    _within(loss[1::2], want[0][1::2], want[1][1::2] + R.U * want[0][1::2].abs())


@pytest.mark.parametrize("t,gt,M,V", [("bf16", "fp16", 500, 33001), ("fp16", "bf16", 250, 66001)])
def test_other_gradients(t, gt, M, V):
    assert _kernel(t, M, V, 9, gt) == HELD
    z, gen = _mixed(2, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 9)
    _check(z, ids, tl, weight, 2.0, _distill(z.cuda(), ids, tl, weight, 2.0, gt=DT[gt], fused=True), gt)


@pytest.mark.parametrize("t,gt", [("fp32", "fp16"), ("fp16", "bf16"), ("fp32", "bf16"), ("bf16", "fp16")])
@pytest.mark.parametrize("M,V", [(5, 901), (300, 5003), (500, 33003), (3, 70001)])
def test_types(t, gt, M, V):
    """Every pair of types that differ, by every kernel."""
    z, gen = _logits(M, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 20)
    for fused in (False, True):
        _check_distill(z, ids, tl, weight, 1.5, _distill(z.cuda(), ids, tl, weight, 1.5, gt=DT[gt], fused=fused), gt)


def _run(view, grad, ids, tl, weight, T):
    from quantized_moe_expert_route_amd.binding import Distill

    M, V = view.shape
    op = Distill(V, ids.shape[1], dtype=view.dtype, grad_dtype=grad.dtype, temperature=T, max_M=M)
    loss = _f32(M)
    op.forward_backward(view, ids.cuda(), tl.cuda(), weight.cuda(), loss, grad, workspace=_ws(op.workspace_bytes(M)))
    return loss, grad


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("gap,off,ggap,goff", [(0, 0, 0, 0), (7, 3, 7, 3), (24, 8, 8, 0), (5, 1, 13, 9), (16, 2, 0, 2)])
def test_strides(t, gap, off, ggap, goff):
    """Rows apart, their gradient's at the same distance from 16 bytes: held. What lies
    between rows stays."""
    M, V = (500, 33001) if t == "bf16" else (250, 33002)
    assert _kernel(t, M, V, 9) == HELD
    z, gen = _logits(gap, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 9)
    _, view = _place(z, V + gap, off)
    buf, grad = _place(z, V + ggap, goff)
    _check_distill(z, ids, tl, weight, 1.0, _run(view, grad, ids, tl, weight, 1.0), t)
    between = torch.ones_like(buf, dtype=torch.bool)
    between.as_strided((M, V), (V + ggap, 1), goff).fill_(False)
    assert buf[between].isnan().all()


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("gap,off", [(3, 0), (0, 1), (3, 1)])
def test_not_alike(t, gap, off):
    """As many rows, whose gradient lies otherwise than they do: another kernel's."""
    M, V = (500, 33001) if t == "bf16" else (250, 33002)
    assert _kernel(t, M, V, 5) == HELD
    z, gen = _logits(off, M, V, t)
    ids, tl, weight = _teacher(gen, M, V, 5)
    _, view = _place(z, V + gap, off)
    _check_distill(z, ids, tl, weight, 1.0, _distill(view, ids, tl, weight, 1.0, fused=True), t)


# ------------------------------------------------------------------ which kernel
def test_kernels():
    """Names by sizes, and refusals."""
    from quantized_moe_expert_route_amd.binding import Distill, TokenScores

    def scores(M, V, k):
        return TokenScores(V, top_k=k, max_M=1 << 20).kernel(M)

    assert scores(4096, 1000, 5) == "128 threads" and scores(77, 30011, 5) == "1024 threads"
    assert scores(2048, 131072, 8) == "512 threads, in stretches" and scores(2048, 131072, 0) == "512 threads"
    assert scores(600, 300000, 8) == "512 threads, long sums" and scores(16, 131072, 8) == "parts of a row, 512 threads"

    def distill(M, V, step, dtype=torch.bfloat16, **kw):
        return Distill(V, 5, dtype=dtype, max_M=1 << 20, **kw).kernel(M, step)

    assert distill(2048, 131072, 2) == HELD and distill(2048, 131072, 0) == "512 threads"
    assert distill(16, 131072, 2) == "parts of a row, 512 threads" and distill(16, 131072, 1) == "parts of a row, 512 threads"
    assert distill(300, 131072, 2) == "1024 threads" and distill(500, 33001, 2, torch.float32, grad_dtype=torch.float16) != HELD
    op = Distill(100, 2, max_M=4)
    for bad in ((0,), (5,), (1, 3), (1, -1)):
        with pytest.raises(ValueError):
            op.kernel(*bad)
    with pytest.raises(ValueError):
        TokenScores(100, max_M=4).kernel(5)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V,k", [(257, 40001, 64), (520, 131072, 3), (513, 98304, 17), (520, 70003, 1)])
def test_alternatives_in_stretches(t, M, V, k):
    """Rows whose alternatives are looked for in quarters of the threads' pieces: whole and
    ragged tiles and quarters."""
    from quantized_moe_expert_route_amd.binding import TokenScores

    assert TokenScores(V, top_k=k, dtype=DT[t], max_M=M).kernel(M) == "512 threads, in stretches"
    z = torch.cat([_logits(i, n, V, t, kind)[0] for i, (n, kind) in enumerate(
        [(M - 20, "normal"), (4, "ties"), (4, "rising"), (4, "falling"), (4, "masked"), (4, "one")])])
    gen = torch.Generator().manual_seed(k)
    some = torch.cat((torch.arange(20), torch.arange(M - 40, M)))
    tokens = torch.randint(0, V, (M,), generator=gen).int()
    o = _scores(z.cuda(), tokens, k)
    want = R.scores(z[some].double(), tokens[some], k)
    assert torch.equal(o["ids"].cpu()[some], want["ids"])
    for name in ("lse", "logprobs", "entropy", "top"):
        _within(o[name][some.cuda()], *want[name], name)
