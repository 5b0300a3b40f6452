"""The matrix product with its epilogue and the gated block on the GPU, forward and
backward, against their 64-bit definitions: bitwise on inputs whose sums are
representable, within the arithmetic's bound on random ones."""

import math

import pytest
import torch

import dense_ref as R

pytestmark = pytest.mark.gpu

DT = R.DT


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen)


def _ints(gen, *shape):
    return torch.randint(-2, 3, shape, generator=gen).float()


def _cuda(t):
    return None if t is None else t.cuda()


def _nan(shape, dtype):
    return torch.full(shape, math.nan, dtype=dtype, device="cuda")


def _ws(n):
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, whatever it is read as


def _within(got, want, bound, what=""):
    g = got.double().cpu()
    assert not g.isnan().any(), what
    bad = ((g - want).abs() > bound).nonzero()
    assert len(bad) == 0, (what, len(bad), bad[:4].tolist(), ((g - want).abs() / bound).max().item())


def _dense(d, **kw):
    from quantized_moe_expert_route_amd.binding import Dense

    return Dense(_cuda(d["w"]), bias=_cuda(d["bias"]), activation=d["act"], **kw)


def _case(seed, M, N, K, t, act, yt=None, bias=True, residual=True, ints=False):
    gen = torch.Generator().manual_seed(seed)
    f = _ints if ints else _normal
    scale = 1.0 if ints else 1 / math.sqrt(K)
    yt = yt or t
    return dict(x=f(gen, M, K).to(DT[t]), w=(f(gen, N, K) * scale).to(DT[t]), bias=f(gen, N).to(DT[t]) if bias else None,
                residual=f(gen, M, N).to(DT[yt]) if residual else None, dy=f(gen, M, N).to(DT[t]), act=act, t=t, yt=yt)


def _f64(t):
    return None if t is None else t.double()


def _forward(d, op):
    M, N = d["dy"].shape
    y, pre = _nan((M, N), DT[d["yt"]]), _nan((M, N), DT[d.get("pt", d["t"])])
    op.forward(_cuda(d["x"]), y, residual=_cuda(d["residual"]), pre=pre, workspace=_ws(op.workspace_bytes(M)))
    return y, pre


def _backward(d, op, pre, which="xwb"):
    M, N = d["dy"].shape
    t = DT[d["t"]]
    dx, dw, db = _nan((M, d["x"].shape[1]), t), _nan(tuple(d["w"].shape), t), _nan((N,), t)
    op.backward(_cuda(d["dy"]), _cuda(d["x"]), dx=dx if "x" in which else None, dw=dw if "w" in which else None,
                dbias=db if "b" in which else None, pre=pre, workspace=_ws(op.workspace_bytes(M, train=True)))
    return dx, dw, db


SIZES = [(1, 1, 8), (1, 16, 64), (2, 17, 72), (3, 40, 136), (15, 33, 1056), (16, 130, 512), (17, 64, 2056), (31, 257, 96),
         (32, 48, 320), (33, 24, 4104), (64, 128, 128), (65, 300, 672), (77, 1543, 264), (127, 129, 200), (128, 256, 64),
         (130, 520, 1280), (200, 96, 1544), (257, 200, 264), (300, 1030, 480)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("t", ["bf16", "fp16"])
def test_exact_sums_are_bitwise(M, N, K, t):
    """Small whole numbers: binary32 sums are exact in any order, so forward and
    all gradients are one rounding of the exact value."""
    yt = "fp32" if (M + N) % 3 == 0 else t
    d = _case(M * 7 + N, M, N, K, t, ("none", "relu")[N % 2], yt, bias=M % 2 == 0, residual=K % 16 == 0, ints=True)
    op = _dense(d, max_M=M)
    y, pre = _forward(d, op)
    ye, _, z, _ = R.dense(_f64(d["x"]), _f64(d["w"]), _f64(d["bias"]), d["act"], _f64(d["residual"]), t, yt)
    assert torch.equal(y.cpu(), ye.float().to(DT[yt]))
    assert torch.equal(pre.cpu(), z.float().to(DT[t]))
    grads = R.dense_backward(_f64(d["dy"]), _f64(pre.cpu()), _f64(d["x"]), _f64(d["w"]), d["act"], t)
    for got, (want, _), what in zip(_backward(d, op, pre), grads, ("dx", "dw", "dbias")):
        assert torch.equal(got.cpu(), want.float().to(DT[t])), what


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("t,yt,act", [("bf16", "bf16", "gelu"), ("fp16", "fp32", "silu"), ("bf16", "fp32", "none"),
                                      ("fp16", "fp16", "gelu_tanh"), ("bf16", "bf16", "relu")])
def test_random_within_the_bound(M, N, K, t, yt, act):
    d = _case(M + N, M, N, K, t, act, yt, bias=N % 2 == 0, residual=M % 2 == 1)
    op = _dense(d, max_M=M)
    y, pre = _forward(d, op)
    ye, ey, z, ez = R.dense(_f64(d["x"]), _f64(d["w"]), _f64(d["bias"]), act, _f64(d["residual"]), t, yt)
    _within(y, ye, ey, "y")
    _within(pre, z, ez, "pre")
    grads = R.dense_backward(_f64(d["dy"]), _f64(pre.cpu()), _f64(d["x"]), _f64(d["w"]), act, t)
    for got, (want, bound), what in zip(_backward(d, op, pre), grads, ("dx", "dw", "dbias")):
        _within(got, want, bound, what)


@pytest.mark.parametrize("M,N,K", [(5, 24, 72), (40, 83, 264), (130, 200, 328)])
@pytest.mark.parametrize("t,act", [("bf16", "gelu"), ("fp16", "silu")])
def test_pre_in_32_bits(M, N, K, t, act):
    d = dict(_case(M, M, N, K, t, act), pt="fp32")
    op = _dense(d, max_M=M)
    y, pre = _forward(d, op)
    ye, ey, z, ez = R.dense(_f64(d["x"]), _f64(d["w"]), _f64(d["bias"]), act, _f64(d["residual"]), t, t, pt="fp32")
    _within(y, ye, ey, "y")
    _within(pre, z, ez, "pre")
    grads = R.dense_backward(_f64(d["dy"]), _f64(pre.cpu()), _f64(d["x"]), _f64(d["w"]), act, t)
    for got, (want, bound), what in zip(_backward(d, op, pre), grads, ("dx", "dw", "dbias")):
        _within(got, want, bound, what)


@pytest.mark.parametrize("act", ["none", "silu"])
def test_each_gradient_alone(act):
    d = _case(5, 50, 72, 136, "bf16", act)
    op = _dense(d, max_M=50)
    _, pre = _forward(d, op)
    full = _backward(d, op, pre)
    for i, which in enumerate("xwb"):
        part = _backward(d, op, pre, which)
        assert torch.equal(part[i], full[i])
        assert all(part[j].isnan().all() for j in range(3) if j != i)


def test_no_rows():
    """M = 0: forward writes nothing, the gradients of the weights are zero."""
    d = _case(6, 4, 24, 64, "bf16", "gelu")
    op = _dense(d)
    ws = _ws(op.workspace_bytes(0, train=True))
    y = _nan((4, 24), torch.bfloat16)
    op.forward(_cuda(d["x"]), y, M=0)
    assert y.isnan().all()
    dx, dw, db = _nan((4, 64), torch.bfloat16), _nan((24, 64), torch.bfloat16), _nan((24,), torch.bfloat16)
    op.backward(_cuda(d["dy"]), _cuda(d["x"]), dx=dx, dw=dw, dbias=db, pre=_cuda(d["dy"]), workspace=ws, M=0)
    assert dx.isnan().all() and (dw == 0).all() and (db == 0).all()


def _wide(t, left, right):
    """t's values as a view into wider rows of NaN."""
    w = torch.full((t.shape[0], left + t.shape[1] + right), math.nan, dtype=t.dtype, device="cuda")
    w[:, left:left + t.shape[1]] = t.cuda()
    return w, w[:, left:left + t.shape[1]]


@pytest.mark.parametrize("M,N", [(5, 83), (40, 83), (140, 88)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_strides_and_in_place_residual(M, N, act):
    """Rows apart in every matrix, odd offsets where the elements' alignment is
    enough; what lies between the rows stays as it was."""
    K, t = 352, "bf16"
    d = _case(M, M, N, K, t, act)
    op = _dense(d, max_M=M + 3)
    ye, ey, z, ez = R.dense(_f64(d["x"]), _f64(d["w"]), _f64(d["bias"]), act, _f64(d["residual"]), t, t)
    _, x = _wide(d["x"], 8, 24)
    yw, y = _wide(d["residual"], 5, 7)
    pw, pre = _wide(d["dy"], 3, 2)
    ws = _ws(op.workspace_bytes(M, train=True))
    op.forward(x, y, residual=y, pre=pre, workspace=ws)
    _within(y, ye, ey, "y")
    _within(pre, z, ez, "pre")
    for w, left, n in ((yw, 5, N), (pw, 3, N)):
        assert w[:, :left].isnan().all() and w[:, left + n:].isnan().all()
    grads = R.dense_backward(_f64(d["dy"]), _f64(pre.cpu()), _f64(d["x"]), _f64(d["w"]), act, t)
    _, dy = _wide(d["dy"], 1, 4)
    dxw, dx = _wide(torch.zeros(M, K, dtype=torch.bfloat16), 3, 6)
    dw, db = _nan((N, K), torch.bfloat16), _nan((N,), torch.bfloat16)
    op.backward(dy, x, dx=dx, dw=dw, dbias=db, pre=pre, workspace=ws)
    for got, (want, bound), what in zip((dx, dw, db), grads, ("dx", "dw", "dbias")):
        _within(got, want, bound, what)
    assert dxw[:, :3].isnan().all() and dxw[:, 3 + K:].isnan().all()


def test_rows_past_M_stay():
    d = _case(9, 100, 64, 128, "fp16", "silu")
    op = _dense(d, max_M=100)
    ws = _ws(op.workspace_bytes(100, train=True))
    for M in (1, 16, 17, 40, 65, 99):
        y, pre, dx = (_nan((100, c), torch.float16) for c in (64, 64, 128))
        op.forward(_cuda(d["x"]), y, residual=_cuda(d["residual"]), pre=pre, workspace=ws, M=M)
        dw = _nan((64, 128), torch.float16)
        op.backward(_cuda(d["dy"]), _cuda(d["x"]), dx=dx, dw=dw, pre=pre, workspace=ws, M=M)
        for t in (y, pre, dx):
            assert t[M:].isnan().all() and not t[:M].isnan().any()
        x, dy, p = (_f64(v[:M].cpu()) for v in (d["x"], d["dy"], pre))
        for got, (want, bound) in zip((dx[:M], dw), R.dense_backward(dy, p, x, _f64(d["w"]), "silu", "fp16")):
            _within(got, want, bound)


@pytest.mark.parametrize("act", R.ACTS)
def test_infinities_and_nan(act):
    """A NaN or infinity reaches its row of y and dx and nothing else; far arguments
    take the activation's limits."""
    M, N, K = 20, 40, 64
    d = _case(11, M, N, K, "bf16", act, bias=True, residual=False)
    d["x"][3, 5] = math.nan
    d["bias"][7], d["bias"][8], d["bias"][9] = 1e4, -1e4, 1e15
    op = _dense(d)
    y, pre = _forward(d, op)
    y = y.float().cpu()
    assert y[3].isnan().all()
    rest = torch.arange(M) != 3
    assert not y[rest].isnan().any()
    want = R.dense(_f64(d["x"][rest]), _f64(d["w"]), _f64(d["bias"]), act, None, "bf16", "bf16")
    _within(y[rest], want[0], want[1])
    d["x"][3, 5] = 0.0
    pre[3] = 0.5
    dx, dw, db = _backward(d, op, pre)
    for got, (w, b) in zip((dx, dw, db), R.dense_backward(_f64(d["dy"]), _f64(pre.cpu()), _f64(d["x"]), _f64(d["w"]), act, "bf16")):
        _within(got, w, b)


# ------------------------------------------------------------------ gated
GATED = [(1, 1, 8), (1, 40, 264), (4, 100, 1024), (16, 33, 2056), (17, 64, 136), (40, 129, 264), (64, 65, 512),
         (129, 200, 328), (260, 150, 200), (333, 579, 264)]


def _gated_case(seed, M, I, H, t, ints=False):
    gen = torch.Generator().manual_seed(seed)
    f = _ints if ints else _normal
    return dict(x=f(gen, M, H).to(DT[t]), w=(f(gen, 2 * I, H) * (1 if ints else 1 / math.sqrt(H))).to(DT[t]),
                dh=f(gen, M, I).to(DT[t]))


@pytest.mark.parametrize("M,I,H", GATED)
@pytest.mark.parametrize("t,act,pt", [("bf16", "silu", "bf16"), ("fp16", "gelu_tanh", "fp32"), ("bf16", "gelu", "fp32"),
                                      ("fp16", "relu", "fp16")])
def test_gated_within_the_bound(M, I, H, t, act, pt):
    from quantized_moe_expert_route_amd.binding import Gated

    d = _gated_case(M + I, M, I, H, t)
    op = Gated(_cuda(d["w"]), activation=act, max_M=M)
    h, pre, dx, dw = _nan((M, I), DT[t]), _nan((M, 2 * I), DT[pt]), _nan((M, H), DT[t]), _nan((2 * I, H), DT[t])
    ws = _ws(op.workspace_bytes(M, train=True))
    op.forward(_cuda(d["x"]), h, pre=pre, workspace=ws)
    he, eh, gu, egu = R.gated(_f64(d["x"]), _f64(d["w"]), act, t, pt)
    _within(h, he, eh, "h")
    _within(pre, gu, egu, "pre")
    op.backward(_cuda(d["dh"]), _cuda(d["x"]), pre, dx=dx, dw=dw, workspace=ws)
    for got, (want, bound), what in zip((dx, dw), R.gated_backward(_f64(d["dh"]), _f64(pre.cpu()), _f64(d["x"]), _f64(d["w"]), act, t), ("dx", "dw")):
        _within(got, want, bound, what)
    alone = _nan((M, I), DT[t])
    op.forward(_cuda(d["x"]), alone, workspace=ws)  # without pre
    assert torch.equal(alone, h)


@pytest.mark.parametrize("M,I,H", GATED)
def test_gated_exact(M, I, H):
    """relu on small whole numbers: everything is exact up to the roundings."""
    from quantized_moe_expert_route_amd.binding import Gated

    t = "bf16"
    d = _gated_case(M, M, I, H, t, ints=True)
    op = Gated(_cuda(d["w"]), activation="relu", max_M=M)
    h, pre, dx, dw = _nan((M, I), DT[t]), _nan((M, 2 * I), DT[t]), _nan((M, H), DT[t]), _nan((2 * I, H), DT[t])
    ws = _ws(op.workspace_bytes(M, train=True))
    op.forward(_cuda(d["x"]), h, pre=pre, workspace=ws)
    he, _, gu, _ = R.gated(_f64(d["x"]), _f64(d["w"]), "relu", t)
    assert torch.equal(h.cpu(), he.float().to(DT[t])) and torch.equal(pre.cpu(), gu.float().to(DT[t]))
    op.backward(_cuda(d["dh"]), _cuda(d["x"]), pre, dx=dx, dw=dw, workspace=ws)
    g, u = _f64(pre.cpu()).chunk(2, 1)
    dz = torch.cat((_f64(d["dh"]) * u * (g > 0), _f64(d["dh"]) * g.clamp(min=0)), 1).float().to(DT[t]).double()
    if (dz.abs() @ _f64(d["w"]).abs()).max() < 2 ** 24 and (dz.T.abs() @ _f64(d["x"]).abs()).max() < 2 ** 24:
        assert torch.equal(dx.cpu(), (dz @ _f64(d["w"])).float().to(DT[t]))
        assert torch.equal(dw.cpu(), (dz.T @ _f64(d["x"])).float().to(DT[t]))


def test_gated_strides_rows_and_no_rows():
    from quantized_moe_expert_route_amd.binding import Gated

    M, I, H, t = 37, 51, 136, "bf16"
    d = _gated_case(3, M, I, H, t)
    op = Gated(_cuda(d["w"]), max_M=M + 9)
    _, x = _wide(d["x"], 8, 8)
    hw, h = _wide(d["dh"], 1, 2)
    pre = _nan((M + 9, 2 * I), torch.bfloat16)
    ws = _ws(op.workspace_bytes(M, train=True))
    op.forward(x, h, pre=pre, workspace=ws, M=M)
    he, eh, _, _ = R.gated(_f64(d["x"]), _f64(d["w"]), "silu", t)
    _within(h, he, eh)
    assert hw[:, :1].isnan().all() and hw[:, 1 + I:].isnan().all() and pre[M:].isnan().all()
    _, dh = _wide(d["dh"], 3, 2)
    dxw, dx = _wide(torch.zeros(M, H, dtype=torch.bfloat16), 1, 2)
    dw = _nan((2 * I, H), torch.bfloat16)
    op.backward(dh, x, pre, dx=dx, dw=dw, workspace=ws, M=M)
    for got, (want, bound) in zip((dx, dw), R.gated_backward(_f64(d["dh"]), _f64(pre[:M].cpu()), _f64(d["x"]), _f64(d["w"]), "silu", t)):
        _within(got, want, bound)
    assert dxw[:, :1].isnan().all() and dxw[:, 1 + H:].isnan().all()
    op.backward(dh, x, pre, dw=dw, workspace=ws, M=0)
    assert (dw == 0).all()
