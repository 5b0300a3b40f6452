"""Every kernel of the operators beside the call: sizes that the choosing rules
give to each of them (asserted through the library on a device of 256 CUs), at
ragged edges, strides and addresses, against exact or 64-bit results."""

import numpy as np
import pytest

import ops_ref as R
from test_gpu_layer import Layer
from test_gpu_linear import _case, _dt, _expect, _f64, _linear
from test_gpu_router import _case as _router_case, _check as _router_check, _run as _router_run

pytestmark = pytest.mark.gpu


def _is(name, handle, M):
    import torch

    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert handle.kernel(M) == name


def _rows(n):
    return "rows, 1 K-step a wave" if n == 1 else f"rows, {n} K-steps a wave"


MID = "{} x {}, K split over the waves".format
TILE = "{} x {} tile".format

# rows: the first of a pair fits the CUs, the second has more tiles than workgroups
FEW_BF16 = [(16, 50, 992, 1), (5, 12400, 352, 1), (7, 60, 2016, 2), (3, 8300, 1056, 2), (2, 70, 2976, 3),
            (16, 4201, 2400, 3), (9, 40, 4000, 4), (4, 4203, 4064, 4), (16, 33, 5120, 5), (1, 4300, 4992, 5),
            (12, 48, 6144, 6), (15, 4202, 6112, 6)]
FEW_FP16 = [c for c in FEW_BF16 if c[3] <= 3] + [(11, 20000, 416, 1), (2, 9000, 1984, 2)]
LINEAR = ([("bf16", M, N, K, _rows(S)) for M, N, K, S in FEW_BF16]
          + [("fp16", M, N, K, _rows(S)) for M, N, K, S in FEW_FP16]
          + [("bf16", 16, 100, 8192, MID(16, 16)), ("bf16", 3, 41, 6176, MID(16, 16)),
             ("bf16", 13, 4210, 6400, MID(16, 32)), ("bf16", 16, 4111, 6176, MID(16, 32)),
             ("fp16", 16, 100, 4000, MID(16, 16)), ("fp16", 5, 4215, 3200, MID(16, 32))]
          + [(xt, M, N, K, name) for xt in ("bf16", "fp16") for M, N, K, name in (
              (17, 48, 160, MID(32, 16)), (31, 301, 1440, MID(32, 16)),
              (17, 5000, 96, MID(32, 32)), (40, 4999, 288, MID(32, 32)))]
          + [("bf16", 33, 12300, 160, TILE(64, 128)), ("bf16", 300, 2605, 544, TILE(64, 128)),
             ("bf16", 65, 16500, 96, TILE(128, 128)), ("bf16", 300, 7001, 352, TILE(128, 128)),
             ("bf16", 65, 33000, 160, TILE(128, 256)), ("bf16", 385, 10001, 1056, TILE(128, 256)),
             ("fp16", 33, 16500, 160, TILE(64, 128)), ("fp16", 300, 4001, 544, TILE(64, 128)),
             ("fp16", 65, 24600, 96, TILE(128, 128)), ("fp16", 300, 7001, 352, TILE(128, 128)),
             ("fp16", 65, 33000, 160, TILE(128, 256)), ("fp16", 385, 10001, 544, TILE(128, 256))])


def _exact(rng, M, N, K, xt, yt):
    """Whole halves and quarters, sums exact in binary32, inside fp16 where y is."""
    d = _case(rng, M, N, K, xt, yt, bias=True, residual=True, integers=True)
    if yt == "fp16":
        d["scales"] -= np.uint8(6)
    y, mag = _expect(d)
    assert mag.max() < 2.0 ** 22
    return d, y


@pytest.mark.parametrize("xt,M,N,K,name", LINEAR)
def test_linear_kernels_exact_sums_in_place(xt, M, N, K, name):
    """Bias, and the residual in place, both types of y."""
    import torch

    for yt in (xt, "fp32"):
        d, y = _exact(np.random.default_rng([M, N, K]), M, N, K, xt, yt)
        lin = _linear(d, max_M=M)
        _is(name, lin, M)
        out = d["residual"].cuda()
        lin.forward(d["x"].cuda(), out, residual=out)
        assert torch.equal(out.cpu(), torch.from_numpy(y).float().to(_dt(yt)))


TILES = [("bf16", 300, 2600, TILE(64, 128)), ("bf16", 300, 7000, TILE(128, 128)), ("bf16", 385, 10000, TILE(128, 256)),
         ("fp16", 300, 4000, TILE(64, 128)), ("fp16", 300, 7000, TILE(128, 128)), ("fp16", 385, 10000, TILE(128, 256))]


@pytest.mark.parametrize("xt,M,N,name", TILES)
@pytest.mark.parametrize("wide", [False, True])
def test_tile_epilogues(xt, M, N, name, wide):
    """16-byte pieces, groups of four and single columns (by address), with and
    without bias and residual, in place and not; bytes between and behind the rows stay."""
    import torch

    K, yt = 160, "fp32" if wide else xt
    d, _ = _exact(np.random.default_rng([M, N, 3]), M, N, K, xt, yt)
    x, ld = d["x"].cuda(), N + 24
    for bias, residual in ((True, True), (True, False), (False, True), (False, False)):
        e = dict(d, bias=d["bias"] if bias else None, residual=d["residual"] if residual else None)
        want = torch.from_numpy(_expect(e)[0]).float().to(_dt(yt)).cuda()
        lin = _linear(e, max_M=M + 4)
        _is(name, lin, M)
        for start in (0, 4, 1):
            buf = torch.full((start + (M + 2) * ld,), 3.0, dtype=_dt(yt), device="cuda")
            rows = buf[start:].view(M + 2, ld)
            res = None
            if residual and start != 4:  # in place
                res = rows[:, :N]
                res[:M] = d["residual"].cuda()
            elif residual:
                res = d["residual"].cuda()
            lin.forward(x, rows[:, :N], residual=res, M=M)
            assert torch.equal(rows[:M, :N], want)
            assert bool((rows[:, N:] == 3.0).all()) and bool((buf[:start] == 3.0).all())
            assert bool((rows[M:] == 3.0).all())


@pytest.mark.parametrize("xt,M,N,name", TILES)
def test_tiles_random_and_non_finite_rows(xt, M, N, name):
    """Random values within the arithmetic's bound; a token of infinities and
    NaN, and a NaN scale, reach only their row and column."""
    import torch

    rng = np.random.default_rng([M, N, 5])
    d = _case(rng, M, N, 480, xt, "fp32", residual=True)
    lin = _linear(d, max_M=M)
    _is(name, lin, M)
    x, res = d["x"].cuda(), d["residual"].cuda()
    base = lin.forward(x, torch.empty_like(res), residual=res)
    y, mag = _expect(d)
    got = _f64(base.cpu())
    assert np.all(np.abs(got - y) <= R.sum_error(480) * mag + R.U32 * np.abs(y))
    rest = torch.arange(M, device="cuda") != M - 2
    for v in (float("nan"), float("inf")):
        bad = x.clone()
        bad[M - 2, 77] = v
        again = lin.forward(bad, torch.empty_like(res), residual=res)
        assert torch.equal(again[rest], base[rest])
        w = torch.from_numpy(R.weights(d["codes"][:, 32:48], d["scales"][:, 2:3])[:, 77 - 64]).cuda()
        odd = ~again[M - 2].isfinite()
        assert bool(odd[w != 0].all())
        if v > 0:  # an infinity: of the weight's sign, NaN where that is zero
            assert torch.equal(again[M - 2][w != 0], torch.where(w[w != 0] > 0, v, -v).float())
            assert bool(again[M - 2][w == 0].isnan().all())
    scales = d["scales"].copy()
    scales[N - 3, 4] = 255
    again = _linear(dict(d, scales=scales), max_M=M).forward(x, torch.empty_like(res), residual=res)
    cols = torch.arange(N, device="cuda") != N - 3
    assert torch.equal(again[:, cols], base[:, cols]) and bool(again[:, N - 3].isnan().all())


@pytest.mark.parametrize("xt,M,N,name", TILES)
def test_tiles_in_graphs_on_streams_and_far_rows(xt, M, N, name):
    import torch

    d, y = _exact(np.random.default_rng([M, N, 7]), M, N, 224, xt, "fp32")
    want = torch.from_numpy(y).float().cuda()
    lin = _linear(d, max_M=M)
    _is(name, lin, M)
    x, res = d["x"].cuda(), d["residual"].cuda()
    out, eager = torch.empty_like(res), torch.empty_like(res)
    lin.forward(x, out, residual=res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(x, out, residual=res)
    for _ in range(4):
        out.zero_()
        graph.replay()
        lin.forward(x, eager, residual=res)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for o in (out, eager):
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o in zip(streams, (out, eager)):
            lin.forward(x, o, residual=res, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(eager, want)
    far = (5 << 30) // (2 * (M - 1)) // 8 * 8  # elements: the last row of x 5 GiB behind the first, of y 10
    xf = torch.empty(far * (M - 1) + 256, dtype=x.dtype, device="cuda").as_strided(x.shape, (far, 1))
    yf = torch.empty(far * (M - 1) + N, dtype=res.dtype, device="cuda").as_strided(res.shape, (far, 1))
    xf.copy_(x)
    yf.copy_(res)
    lin.forward(xf, yf, residual=yf)
    assert torch.equal(yf, want)


ROUTER = [(1, 30, 520, "1 token"), (3, 300, 264, "4 tokens"), (8, 65, 1032, "8 tokens"), (9, 256, 6144, "16 tokens"),
          (40, 161, 2056, MID(16, 16)), (900, 250, 328, MID(16, 16)), (1024, 256, 520, MID(32, 32)),
          (993, 250, 328, MID(32, 32)), (2100, 255, 264, TILE(64, 64)), (1100, 500, 136, TILE(64, 64))]


@pytest.mark.parametrize("M,E,H,name", ROUTER)
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "bf16"), ("fp16", "fp32")])
def test_router_kernels(M, E, H, name, xt, wt):
    """Contiguous, then with rows 5 GiB apart in all, logits behind M left alone."""
    import torch
    from quantized_moe_expert_route_amd.binding import Router

    x, w = _router_case(M, E, H, xt, wt, seed=3)
    r = Router(w.cuda(), x_dtype=x.dtype)
    _is(name, r, M)
    base = _router_run(x, w)
    _router_check(base, x, w)
    far = (5 << 30) // (2 * max(M - 1, 1)) // 8 * 8
    xf = torch.empty(far * (M - 1) + H, dtype=x.dtype, device="cuda").as_strided((M, H), (far, 1))
    xf.copy_(x)
    out = torch.full((M + 3, E), 5.0, device="cuda")
    r.forward(xf, out, M=M)
    assert np.array_equal(out[:M].cpu().double().numpy(), base) and bool((out[M:] == 5.0).all())


@pytest.mark.parametrize("M,H,E,I,k", [
    # down: columns a workgroup by I
    (5, 5632, 20, 128, 4), (9, 7680, 18, 256, 5), (16, 5120, 30, 384, 6), (11, 3584, 16, 512, 8),
    # gate/up: K-steps a wave, more than 256 experts, one and two tokens a wave
    (4, 2048, 257, 128, 3), (16, 2560, 270, 128, 4), (3, 5120, 260, 128, 8), (10, 6144, 258, 128, 8),
    (13, 7168, 300, 128, 2), (8, 4096, 300, 128, 16),
    # one to four passes of five tokens an expert, all on few experts
    (16, 1024, 16, 256, 16), (16, 1024, 4, 256, 3), (11, 1024, 3, 256, 2), (6, 1024, 2, 256, 1)])
def test_layer_kernels(M, H, E, I, k):
    d = Layer(M, H, E, I, k, wt="fp32" if M % 2 else "bf16", alike=0.3, seed=4)
    d.check(d.call())


def test_kernel_names_and_bad_counts():
    d = _case(np.random.default_rng(1), 4, 32, 64, "bf16", "bf16")
    lin = _linear(d, max_M=40)
    assert lin.kernel(1) and lin.kernel(40)
    for M in (0, -1, 41):
        with pytest.raises(ValueError):
            lin.kernel(M)
    lin.close()
    with pytest.raises(ValueError):
        lin.kernel(1)


@pytest.mark.parametrize("xt,M,N,K", [(xt, M, N, K) for xt in ("bf16", "fp16")
                                      for M, N, K in ((4, 50, 352), (16, 100, 8192), (20, 300, 352), (300, 2600, 160),
                                                      (300, 7000, 160), (385, 10000, 160))])
def test_linear_subnormal_x(xt, M, N, K):
    """Subnormal numbers of x's type keep their value in every kernel."""
    import torch

    d = _case(np.random.default_rng([M, N, K, 9]), M, N, K, xt, "fp32", integers=True)
    unit = 2.0 ** -24 if xt == "fp16" else 2.0 ** -133
    d["x"] = (d["x"].double() * unit).to(_dt(xt))
    assert np.count_nonzero(_f64(d["x"])) > M * K // 2
    if xt == "bf16":
        d["scales"] += np.uint8(100)
    y, _ = _expect(d)
    lin = _linear(d)
    out = torch.empty(M, N, device="cuda")
    lin.forward(d["x"].cuda(), out)
    assert np.array_equal(_f64(out.cpu()), y)


@pytest.mark.parametrize("M,E,H", [(4, 50, 264), (16, 50, 264), (40, 50, 264), (1024, 256, 136), (1100, 500, 136)])
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "bf16"), ("fp16", "fp32")])
def test_router_subnormal_x(M, E, H, xt, wt):
    import torch

    g = torch.Generator().manual_seed(M + E)
    unit = 2.0 ** -24 if xt == "fp16" else 2.0 ** -133
    x = (torch.randint(-3, 4, (M, H), generator=g).double() * unit).to(_dt(xt))
    w = torch.randint(-9, 10, (E, H), generator=g).to(_dt(wt)) * 2.0 ** 60
    want = x.double().numpy() @ w.double().numpy().T
    assert np.array_equal(_router_run(x, w), want)
