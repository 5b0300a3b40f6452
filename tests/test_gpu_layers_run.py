"""The 16-bit layers and the head's operators run together, as a training step and a
decode step use them; every kernel of the products at sizes that choose it; graphs,
streams, workspaces, far rows."""

import math

import pytest
import torch

import dense_ref as R

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _B():
    from quantized_moe_expert_route_amd import binding

    return binding


def _ws(n):
    return torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")


def _empty(*shape, dtype=BF):
    return torch.full(shape, math.nan if dtype.is_floating_point else -7, dtype=dtype, device="cuda")


def _within(got, want, bound, what=""):
    g = got.double().cpu()
    assert not g.isnan().any(), what
    bad = ((g - want).abs() > bound).nonzero()
    assert len(bad) == 0, (what, len(bad), bad[:4].tolist(), ((g - want).abs() / bound).max().item())


# ------------------------------------------------------------------ kernels
# rows, columns and K of a product, and the kernel that it chooses
PRODUCTS = [
    (2050, 6200, 72, "256 x 256 tile"), (700, 4104, 4104, "256 x 256 tile"),  # the second of each: K split
    (4100, 2056, 72, "256 x 192 tile"), (4100, 520, 4104, "256 x 192 tile"),
    (2050, 2056, 72, "128 x 128 tile"), (1030, 2056, 2056, "128 x 128 tile"),
    (130, 6200, 72, "64 x 64 tile"), (130, 2056, 4104, "64 x 64 tile"),
    (130, 40, 72, "64 x 64 tile, two groups of waves"), (130, 40, 4104, "64 x 64 tile, two groups of waves"),
    (333, 2056, 2320, "64 x 64 tile, two groups of waves"),
]
WAVES = [(5, 40, 72, "16 x 16, K split over the waves"), (5, 4104, 72, "16 x 32, K split over the waves"),
         (16, 16000, 1032, "16 x 32, K split over the waves"), (3, 300, 9000, "16 x 16, K split over the waves"),
         (20, 40, 72, "32 x 16, K split over the waves"), (40, 2056, 72, "32 x 32, K split over the waves"),
         (32, 20000, 264, "32 x 32, K split over the waves")]


def _ints(seed, *shape):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-2, 3, shape, generator=gen, device="cuda").float()


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,K,kernel", PRODUCTS + WAVES)
def test_forward_kernels(rows, cols, K, kernel, t):
    x, w = _ints(1, rows, K).to(R.DT[t]), _ints(2, cols, K).to(R.DT[t])
    op = _B().Dense(w, activation="relu", max_M=rows)
    assert op.kernel(rows) == kernel
    y, pre = _empty(rows, cols, dtype=R.DT[t]), _empty(rows, cols, dtype=F32)
    op.forward(x, y, pre=pre, workspace=_ws(op.workspace_bytes(rows)))
    want = x.double() @ w.double().t()
    assert torch.equal(pre, want.float()) and torch.equal(y, want.clamp(min=0).float().to(R.DT[t]))


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,K,kernel", PRODUCTS)
def test_gradient_kernels(rows, cols, K, kernel, t):
    dt = R.DT[t]
    dy, w = _ints(3, rows, K).to(dt), _ints(4, K, cols).to(dt)  # dx = dy w
    op = _B().Dense(w, max_M=rows)
    assert op.kernel(rows, 1) == kernel
    dx = _empty(rows, cols, dtype=dt)
    op.backward(dy, dx, dx=dx, workspace=_ws(op.workspace_bytes(rows, train=True)))
    assert torch.equal(dx, (dy.double() @ w.double()).float().to(dt))
    dy, x = _ints(5, K, rows).to(dt), _ints(6, K, cols).to(dt)  # dw = dy^T x
    op = _B().Dense(_ints(7, rows, cols).to(dt), max_M=K)
    assert op.kernel(K, 2) == kernel
    dw = _empty(rows, cols, dtype=dt)
    op.backward(dy, x, dw=dw, workspace=_ws(op.workspace_bytes(K, train=True)))
    assert torch.equal(dw, (dy.double().t() @ x.double()).float().to(dt))


GATED = [(700, 8200, 72, "256 x 256 tile"), (130, 6200, 4104, "256 x 256 tile"), (2050, 2050, 72, "256 x 192 tile"),
         (1030, 2050, 72, "128 x 128 tile"), (100, 8200, 2056, "128 x 128 tile"), (130, 3100, 72, "64 x 64 tile"),
         (130, 1030, 4104, "64 x 64 tile"), (130, 40, 72, "64 x 64 tile, two groups of waves"),
         (130, 40, 4104, "64 x 64 tile, two groups of waves"), (333, 1159, 2056, "64 x 64 tile, two groups of waves"), (5, 40, 72, "16 x 16, K split over the waves"),
         (5, 2050, 72, "16 x 32, K split over the waves"), (20, 40, 72, "32 x 16, K split over the waves"),
         (20, 2050, 72, "32 x 32, K split over the waves"), (16, 5003, 1032, "16 x 16, K split over the waves")]


@pytest.mark.parametrize("t", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,cols,K,kernel", GATED)
def test_gated_kernels(rows, cols, K, kernel, t):
    dt = R.DT[t]
    x, w = _ints(8, rows, K).to(dt), _ints(9, 2 * cols, K).to(dt)
    op = _B().Gated(w, activation="relu", max_M=rows)
    assert op.kernel(rows) == kernel
    h, pre = _empty(rows, cols, dtype=dt), _empty(rows, 2 * cols, dtype=F32)
    op.forward(x, h, pre=pre, workspace=_ws(op.workspace_bytes(rows)))
    gu = x.double() @ w.double().t()
    assert torch.equal(pre, gu.float())
    assert torch.equal(h, (gu[:, :cols].clamp(min=0) * gu[:, cols:]).float().to(dt))


def test_every_kernel_is_here():
    names = {p[3] for p in PRODUCTS + WAVES}
    assert names == {p[3] for p in GATED} and len(names) == 9


def test_kernel_refuses():
    op = _B().Dense(torch.zeros(16, 64, dtype=BF, device="cuda"), max_M=10)
    for M, product in ((0, 0), (11, 0), (5, 3), (5, -1)):
        with pytest.raises(ValueError):
            op.kernel(M, product)


# ------------------------------------------------------------------ the run
class _Step:
    """A block and the head on top, trained from a teacher's alternatives: x -> gated ->
    down with the residual x -> head -> distillation, and all gradients back."""

    M, H, I, V, k, T = 70, 264, 200, 1003, 12, 2.0

    def __init__(self, seed=0):
        B = _B()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s, scale=1.0: (torch.randn(s, generator=gen, device="cuda") * scale).to(BF)
        M, H, I, V, k = self.M, self.H, self.I, self.V, self.k
        self.x, self.w13, self.w2 = n(M, H), n(2 * I, H, scale=H ** -0.5), n(H, I, scale=I ** -0.5)
        self.wh, self.bh = n(V, H, scale=3 * H ** -0.5), n(V)
        self.teacher = n(M, V, scale=3.0)
        self.gated, self.down = B.Gated(self.w13, max_M=M), B.Dense(self.w2, max_M=M)
        self.head = B.Dense(self.wh, bias=self.bh, max_M=M)
        self.scores = B.TokenScores(V, top_k=k, dtype=BF, max_M=M)
        self.distill = B.Distill(V, k, dtype=F32, grad_dtype=BF, temperature=self.T, max_M=M)
        self.weight = torch.full((M,), 1.0 / M, device="cuda")
        self.h, self.pre, self.y, self.z = _empty(M, I), _empty(M, 2 * I, dtype=F32), _empty(M, H), _empty(M, V, dtype=F32)
        self.t, self.ids = _empty(M, k, dtype=F32), _empty(M, k, dtype=I32)
        self.loss, self.dz = _empty(M, dtype=F32), _empty(M, V)
        self.dy, self.dwh, self.dbh, self.dh, self.dw2 = _empty(M, H), _empty(V, H), _empty(V), _empty(M, I), _empty(H, I)
        self.dx, self.dw13 = _empty(M, H), _empty(2 * I, H)
        self.ws = _ws(max(self.gated.workspace_bytes(M, True), self.down.workspace_bytes(M, True),
                          self.head.workspace_bytes(M, True), self.scores.workspace_bytes(M), self.distill.workspace_bytes(M)))
        self.outputs = ("h", "pre", "y", "z", "t", "ids", "loss", "dz", "dy", "dwh", "dbh", "dh", "dw2", "dx", "dw13")

    def run(self, stream=None):
        ws = dict(workspace=self.ws, stream=stream)
        self.scores.forward(self.teacher, None, None, top_logprobs=self.t, top_ids=self.ids, **ws)
        self.gated.forward(self.x, self.h, pre=self.pre, **ws)
        self.down.forward(self.h, self.y, residual=self.x, **ws)
        self.head.forward(self.y, self.z, **ws)
        self.distill.forward_backward(self.z, self.ids, self.t, self.weight, self.loss, self.dz, **ws)
        self.head.backward(self.dz, self.y, dx=self.dy, dw=self.dwh, dbias=self.dbh, **ws)
        self.down.backward(self.dy, self.h, dx=self.dh, dw=self.dw2, **ws)
        self.gated.backward(self.dh, self.x, self.pre, dx=self.dx, dw=self.dw13, **ws)

    def results(self):
        return {name: getattr(self, name).clone() for name in self.outputs}


def _f64(t):
    return t.double().cpu()


def test_training_step():
    """Every stage within its bound of the definition on what the stages before it gave."""
    s = _Step()
    s.run()
    top = R.scores(_f64(s.teacher), torch.zeros(s.M, dtype=I32), s.k)
    assert torch.equal(s.ids.cpu(), top["ids"])
    _within(s.t, *top["top"], "t")
    h, eh, pre, ep = R.gated(_f64(s.x), _f64(s.w13), "silu", "bf16", "fp32")
    _within(s.h, h, eh, "h")
    _within(s.pre, pre, ep, "pre")
    y, ey, _, _ = R.dense(_f64(s.h), _f64(s.w2), None, "none", _f64(s.x), "bf16", "bf16")
    _within(s.y, y, ey, "y")
    z, ez, _, _ = R.dense(_f64(s.y), _f64(s.wh), _f64(s.bh), "none", None, "bf16", "fp32")
    _within(s.z, z, ez, "z")
    loss, el, dz, edz = R.distill(_f64(s.z), s.ids.cpu(), _f64(s.t), _f64(s.weight), s.T)
    _within(s.loss, loss, el + R.U * loss.abs(), "loss")
    _within(s.dz, dz, edz * 1.01 + R.rounding("bf16", dz), "dz")
    for got, (want, bound) in zip((s.dy, s.dwh, s.dbh), R.dense_backward(_f64(s.dz), None, _f64(s.y), _f64(s.wh), "none", "bf16")):
        _within(got, want, bound, "head")
    for got, (want, bound) in zip((s.dh, s.dw2), R.dense_backward(_f64(s.dy), None, _f64(s.h), _f64(s.w2), "none", "bf16")):
        _within(got, want, bound, "down")
    for got, (want, bound) in zip((s.dx, s.dw13), R.gated_backward(_f64(s.dh), _f64(s.pre), _f64(s.x), _f64(s.w13), "silu", "bf16")):
        _within(got, want, bound, "gated")


def test_same_bits_again():
    s = _Step(1)
    s.run()
    first = s.results()
    for name in s.outputs:
        getattr(s, name).fill_(3)
    s.ws.fill_(0x7F)
    s.run()
    for name, v in s.results().items():
        assert torch.equal(v, first[name]), name


def test_captured_step():
    """A captured training step, replayed on changed inputs and weights with eager work
    and synchronizations between, gives the eager step's bits."""
    s, eager = _Step(2), _Step(2)
    s.run()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run(stream=torch.cuda.current_stream())
    for i in range(4):
        new = _Step(10 + i)
        for name in ("x", "w13", "w2", "wh", "bh", "teacher"):
            getattr(s, name).copy_(getattr(new, name))
            getattr(eager, name).copy_(getattr(new, name))
        s.ws.fill_(0xFF)
        graph.replay()
        eager.run()
        if i % 2:
            torch.cuda.synchronize()
        want = eager.results()
        for name, v in s.results().items():
            assert torch.equal(v, want[name]), (i, name)


def test_two_streams_with_workspaces_of_their_own():
    """Two steps at once on two streams, each on its own workspace and handles shared."""
    a, b = _Step(3), _Step(4)
    a.run()
    b.run()
    want = a.results(), b.results()
    b.gated, b.down = a.gated, a.down  # one handle, two callers
    b.w13.copy_(a.w13)
    b.w2.copy_(a.w2)
    b.run()
    want = want[0], b.results()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        a.run(stream=sa)
        b.run(stream=sb)
    torch.cuda.synchronize()
    for s, w in ((a, want[0]), (b, want[1])):
        for name, v in s.results().items():
            assert torch.equal(v, w[name]), name


def test_decode_step():
    """One to four tokens through the block and the head, their logits scored: each token
    as in a batch of its own bits (a row's sums do not depend on the others)."""
    s = _Step(5)
    tokens = torch.arange(4, dtype=I32, device="cuda")
    single = []
    for M in (4, 1, 2, 3):
        s.gated.forward(s.x, s.h, workspace=s.ws, M=M)
        s.down.forward(s.h, s.y, residual=s.x, workspace=s.ws, M=M)
        s.head.forward(s.y, s.z, workspace=s.ws, M=M)
        lp, ent = _empty(4, dtype=F32), _empty(4, dtype=F32)
        sc = _B().TokenScores(s.V, top_k=5, dtype=F32, max_M=4)
        top, ids = _empty(4, 5, dtype=F32), _empty(4, 5, dtype=I32)
        sc.forward(s.z, tokens, lp, entropy=ent, top_logprobs=top, top_ids=ids, workspace=s.ws, M=M)
        want = R.scores(_f64(s.z[:M]), tokens[:M].cpu(), 5)
        assert torch.equal(ids[:M].cpu(), want["ids"])
        _within(lp[:M], *want["logprobs"])
        _within(ent[:M], *want["entropy"])
        _within(top[:M], *want["top"])
        single.append((s.z[:M].clone(), lp[:M].clone()))
    for z, lp in single[1:]:
        assert torch.equal(z, single[0][0][:len(z)]) and torch.equal(lp, single[0][1][:len(lp)])


# ------------------------------------------------------------------ far rows, large sizes
def test_rows_past_four_gib():
    """Row distances that put rows past 2^32 bytes, in every matrix that takes them."""
    B = _B()
    M, N, K = 3, 24, 64
    far = 1 << 30
    x, w, res = _ints(1, M, K).to(BF), _ints(2, N, K).to(BF), _ints(3, M, N).to(BF)
    buf = torch.zeros((M - 1) * far + 4096, dtype=BF, device="cuda")
    other = torch.zeros_like(buf)  # (interleaved rows of one buffer count as an overlap)
    view = lambda cols, off, of=buf: of.as_strided((M, cols), (far, 1), off)
    op = B.Dense(w, max_M=M)
    y, dx = view(N, 0), view(K, 1024)
    y.copy_(res)
    op.forward(x, y, residual=y)
    want = (x.double() @ w.double().t() + res.double()).to(BF)
    assert torch.equal(y, want)
    dy = view(N, 2048, other)
    dy.copy_(res)
    op.backward(dy, x, dx=dx, workspace=_ws(op.workspace_bytes(M, train=True)))
    assert torch.equal(dx, (res.double() @ w.double()).to(BF))
    # logits and their gradient
    V = 1000
    z = view(V, 3000)
    gen = torch.Generator().manual_seed(1)
    zc = torch.randn(M, V, generator=gen).to(BF)
    z.copy_(zc)
    sc, lp = B.TokenScores(V, dtype=BF, max_M=M), _empty(M, dtype=F32)
    tokens = torch.tensor([5, 0, 999], dtype=I32)
    sc.forward(z, tokens.cuda(), lp, workspace=_ws(sc.workspace_bytes(M)))
    _within(lp, *R.scores(zc.double(), tokens, 0)["logprobs"])
    ids, t = torch.tensor([[1], [999], [7]], dtype=I32), torch.zeros(M, 1)
    di, loss, weight = B.Distill(V, 1, dtype=BF, max_M=M), _empty(M, dtype=F32), torch.ones(M)
    di.forward_backward(z, ids.cuda(), t.cuda(), weight.cuda(), loss, z, workspace=_ws(di.workspace_bytes(M)))
    want = R.distill(zc.double(), ids, t.double(), weight.double(), 1.0)
    _within(z, want[2], want[3] * 1.01 + R.rounding("bf16", want[2]))


def test_operand_rows_far_apart():
    """x at the largest row distance: tiles of rows reach 2^31 bytes, all rows past 2^32."""
    M, N, K, far = 700, 40, 72, 1 << 22
    buf = torch.zeros((M - 1) * far + K, dtype=BF, device="cuda")
    x = buf.as_strided((M, K), (far, 1))
    xc, w, dy = _ints(1, M, K).to(BF), _ints(2, N, K).to(BF), _ints(3, M, N).to(BF)
    x.copy_(xc)
    op = _B().Dense(w, max_M=M)
    ws = _ws(op.workspace_bytes(M, train=True))
    y, dw = _empty(M, N), _empty(N, K)
    for m in (M, 16, 100):
        op.forward(x, y, workspace=ws, M=m)
        assert torch.equal(y[:m], (xc[:m].double() @ w.double().t()).to(BF))
    op.backward(dy, x, dw=dw, workspace=ws)
    assert torch.equal(dw, (dy.double().t() @ xc.double()).float().to(BF))
    with pytest.raises(_B().MoeError):
        op.forward(torch.empty_strided((2, K), (far + 8, 1), dtype=BF, device="cuda"), y)


def test_weights_past_four_gib():
    """A weight of more than 2^32 bytes: forward, both gradients."""
    N, K = 300008, 8192
    w = _ints(1, N, K).to(BF)
    op = _B().Dense(w, max_M=200)
    for M in (2, 40, 200):
        x, dy = _ints(2, M, K).to(BF), _ints(3, M, N).to(BF)
        y, dx, dw = _empty(M, N, dtype=F32), _empty(M, K), _empty(N, K)
        ws = _ws(op.workspace_bytes(M, train=True))
        op.forward(x, y, workspace=ws)
        op.backward(dy, x, dx=dx, dw=dw, workspace=ws)
        total = torch.zeros(M, K, dtype=torch.float64, device="cuda")
        for a in range(0, N, 50000):
            part = w[a:a + 50000].double()
            assert torch.equal(y[:, a:a + 50000], (x.double() @ part.t()).float())
            total += dy[:, a:a + 50000].double() @ part
            assert torch.equal(dw[a:a + 50000], (dy[:, a:a + 50000].double().t() @ x.double()).float().to(BF))
        assert torch.equal(dx, total.float().to(BF))
        del dw, ws


def test_refused_on_the_device():
    """Overlaps, short workspaces, misaligned operands: refused before anything runs."""
    B = _B()
    w = torch.zeros(24, 64, dtype=BF, device="cuda")
    op = B.Dense(w, activation="silu", max_M=300)
    x, y = torch.zeros(300, 64, dtype=BF, device="cuda"), torch.zeros(300, 24, dtype=BF, device="cuda")
    ws = _ws(op.workspace_bytes(300, train=True))
    big = torch.zeros(301, 64, dtype=BF, device="cuda")

    def refused(status, f):
        with pytest.raises(B.MoeError) as e:
            f()
        assert e.value.status == status

    refused(B.MOE_ERR_INVALID_ARG, lambda: op.forward(big[:300], big[1:, :24], workspace=ws))  # y over x
    refused(B.MOE_ERR_INVALID_ARG, lambda: op.forward(x, y, pre=y, workspace=ws))
    refused(B.MOE_ERR_INVALID_ARG, lambda: op.forward(x, y[1:], residual=y[:-1], workspace=ws, M=299))
    refused(B.MOE_ERR_INVALID_ARG, lambda: op.forward(big.view(-1)[4:4 + 300 * 64].view(300, 64), y, workspace=ws))
    refused(B.MOE_ERR_INVALID_ARG, lambda: op.forward(torch.zeros(300, 68, dtype=BF, device="cuda")[:, :64], y, workspace=ws))
    refused(B.MOE_ERR_INVALID_ARG, lambda: op.backward(y, x, dw=w, pre=y.clone(), workspace=ws))  # over the weights
    refused(B.MOE_ERR_INVALID_ARG, lambda: op.backward(y, x, pre=y.clone(), workspace=ws))  # nothing asked for
    refused(B.MOE_ERR_WORKSPACE, lambda: op.backward(y, x, dx=x.clone(), pre=y.clone(), workspace=ws[:-256]))
    refused(B.MOE_ERR_WORKSPACE, lambda: op.backward(y, x, dx=x.clone(), pre=y.clone()))
    refused(B.MOE_ERR_WORKSPACE, lambda: op.backward(y, x, dx=x.clone(), pre=y.clone(), workspace=_ws(ws.numel() + 16)[16:]))
    sc = B.TokenScores(400000, top_k=3, dtype=BF, max_M=4)
    z = torch.zeros(4, 400000, dtype=BF, device="cuda")
    top, ids = torch.zeros(4, 3, device="cuda"), torch.zeros(4, 3, dtype=I32, device="cuda")
    refused(B.MOE_ERR_WORKSPACE, lambda: sc.forward(z, None, None, top_logprobs=top, top_ids=ids))
    refused(B.MOE_ERR_INVALID_ARG, lambda: sc.forward(z, None, None, top_logprobs=top, top_ids=top.view(I32), workspace=_ws(sc.workspace_bytes(4))))
    di = B.Distill(100, 2, dtype=BF, max_M=4)
    zz, wt, loss = torch.zeros(5, 100, dtype=BF, device="cuda"), torch.ones(4, device="cuda"), torch.zeros(4, device="cuda")
    i2, t2 = torch.zeros(4, 2, dtype=I32, device="cuda"), torch.zeros(4, 2, device="cuda")
    wd = _ws(di.workspace_bytes(4))
    refused(B.MOE_ERR_INVALID_ARG, lambda: di.forward_backward(zz[:4], i2, t2, wt, loss, zz[1:], workspace=wd))  # half in place
    refused(B.MOE_ERR_INVALID_ARG, lambda: di.forward_backward(zz[:4], i2, t2, loss, loss, zz[:4], workspace=wd))
    assert (z == 0).all() and (y == 0).all() and (zz == 0).all()
