"""MXFP4 linear layer on the GPU against its 64-bit definition: bitwise on
inputs whose sums are representable, within the arithmetic's bound on random
ones."""

import numpy as np
import pytest

import ops_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": "bfloat16", "fp16": "float16", "fp32": "float32"}


def _dt(name):
    import torch

    return getattr(torch, DT[name])


def _case(rng, M, N, K, xt, yt, bias=False, residual=False, integers=False):
    import torch

    if integers:
        # multiples of 1/2 of magnitude <= 3 * 6 * K: binary32 sums are exact in any order
        x = torch.from_numpy(rng.integers(-3, 4, (M, K)).astype(np.float32))
        codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
        scales = rng.integers(126, 129, (N, K // 32), dtype=np.uint8)
        extra = lambda *s: torch.from_numpy(rng.integers(-9, 10, s).astype(np.float32))
    else:
        x = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32))
        codes, scales = R.random_weights(rng, N, K)
        extra = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    return dict(x=x.to(_dt(xt)), codes=codes, scales=scales, bias=extra(N).to(_dt(xt)) if bias else None,
                residual=extra(M, N).to(_dt(yt)) if residual else None, xt=xt, yt=yt)


def _f64(t):
    return None if t is None else t.double().numpy()


def _linear(d, max_M=1 << 20):
    import torch
    from quantized_moe_expert_route_amd.binding import Linear

    cu = lambda a: None if a is None else (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).cuda()
    return Linear(cu(d["codes"]), cu(d["scales"]), bias=cu(d["bias"]), x_dtype=_dt(d["xt"]), max_M=max_M)


def _run(d, lin=None):
    import torch

    lin = lin or _linear(d)
    out = torch.full((d["x"].shape[0], lin.N), float("nan"), dtype=_dt(d["yt"]), device="cuda")
    res = None if d["residual"] is None else d["residual"].cuda()
    lin.forward(d["x"].cuda(), out, residual=res)
    torch.cuda.synchronize()
    return out.cpu()


def _expect(d):
    return R.linear(_f64(d["x"]), d["codes"], d["scales"], _f64(d["bias"]), _f64(d["residual"]))


def _check(got, d):
    y, mag = _expect(d)
    err = np.abs(_f64(got) - y)
    tol = (R.sum_error(d["x"].shape[1]) * mag) * (1 + R.half_step(d["yt"])) + R.half_step(d["yt"]) * np.abs(y)
    tol += 2.0 ** -25 if d["yt"] == "fp16" else 0.0  # half a subnormal step
    assert not np.isnan(_f64(got)).any()
    bad = np.argwhere(err > tol)
    assert len(bad) == 0, (len(bad), bad[:4].tolist(), float((err / tol).max()))


SIZES = [(1, 16, 32), (1, 1, 32), (2, 17, 160), (3, 5, 1024), (16, 64, 2048), (15, 33, 1056), (7, 130, 6144),
         (16, 40, 8192), (1, 24, 8224), (5, 48, 16384), (16, 16, 65536), (17, 50, 512), (31, 96, 4128),
         (33, 257, 1440), (64, 48, 2048), (65, 300, 672), (130, 70, 96), (257, 520, 1280), (300, 1543, 480)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
def test_exact_sums_are_bitwise(M, N, K, xt, yt):
    rng = np.random.default_rng([M, N, K])
    d = _case(rng, M, N, K, xt, yt, bias=(M + N) % 2 == 0, residual=(N + K // 32) % 2 == 0, integers=True)
    if yt == "fp16":  # keep the sums inside fp16's range
        d["scales"] -= np.uint8(6)
    y, mag = _expect(d)
    assert mag.max() < 2.0 ** 22
    import torch

    want = torch.from_numpy(y).float().to(_dt(yt))  # y is exact in binary32: one rounding
    assert torch.equal(_run(d), want)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("xt,yt,bias,residual", [("bf16", "bf16", True, True), ("fp16", "fp32", False, True),
                                                ("bf16", "fp32", True, False), ("fp16", "fp16", False, False)])
def test_random_within_the_bound(M, N, K, xt, yt, bias, residual):
    rng = np.random.default_rng([M, N, K, 1])
    d = _case(rng, M, N, K, xt, yt, bias, residual)
    _check(_run(d), d)


def test_large_weights_and_many_tiles():
    """More tiles than workgroups, at the widths the repository's workloads have."""
    rng = np.random.default_rng(5)
    for M, N in ((4, 20000), (16, 9000), (100, 12300)):
        d = _case(rng, M, N, 6144 if M < 100 else 512, "bf16", "bf16")
        _check(_run(d), d)


def test_one_handle_many_row_counts():
    """One handle serves every row count up to its bound; rows past M are left as they were."""
    import torch

    rng = np.random.default_rng(7)
    d = _case(rng, 300, 200, 1440, "bf16", "bf16")
    lin = _linear(d, max_M=300)
    y, mag = _expect(d)
    x = d["x"].cuda()
    for M in (0, 1, 2, 16, 17, 32, 33, 48, 64, 65, 127, 128, 129, 255, 300):
        out = torch.full((300, 200), 7.0, dtype=torch.bfloat16, device="cuda")
        lin.forward(x, out, M=M)
        got = _f64(out.cpu())
        assert np.all(got[M:] == 7.0)
        tol = R.sum_error(1440) * mag[:M] * 1.01 + R.half_step("bf16") * np.abs(y[:M])
        assert np.all(np.abs(got[:M] - y[:M]) <= tol)
    with pytest.raises(ValueError):
        lin.forward(torch.zeros(301, 1440, dtype=torch.bfloat16, device="cuda"), out)


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_strided_rows_and_in_place_residual(M):
    import torch

    rng = np.random.default_rng(M)
    N, K = 83, 352
    for xt, yt in (("bf16", "bf16"), ("fp16", "fp32")):
        d = _case(rng, M, N, K, xt, yt, residual=True)
        y, mag = _expect(d)
        xw = torch.full((M, K + 40), float("nan"), dtype=_dt(xt), device="cuda")
        xw[:, 8:K + 8] = d["x"].cuda()
        yw = torch.full((M, N + 13), 3.0, dtype=_dt(yt), device="cuda")
        yw[:, 5:N + 5] = d["residual"].cuda()
        view = yw[:, 5:N + 5]
        _linear(d).forward(xw[:, 8:K + 8], view, residual=view)
        got = yw.cpu()
        assert torch.all(got[:, :5] == 3.0) and torch.all(got[:, N + 5:] == 3.0)
        tol = R.sum_error(K) * mag * 1.01 + R.half_step(yt) * np.abs(y)
        assert np.all(np.abs(_f64(got[:, 5:N + 5]) - y) <= tol)


@pytest.mark.parametrize("M", [3, 50, 140])
@pytest.mark.parametrize("xt", ["bf16", "fp16"])
def test_extreme_scales(M, xt):
    """Scales from 2^-127 to 2^125 (x small and large to match), and rows
    whose blocks lie 2^40 apart."""
    import torch

    rng = np.random.default_rng(9)
    N, K = 48, 256
    d = _case(rng, M, N, K, xt, "fp32", integers=True)
    d["scales"][:16] = 252
    d["scales"][16:32] = rng.choice([90, 130], (16, K // 32))
    d["scales"][32:40] = 20
    d["x"] = (d["x"].float() * 2.0 ** -12).to(_dt(xt))
    y, mag = _expect(d)
    got = _f64(_run(d))
    with np.errstate(over="ignore"):
        want = y.astype(np.float32).astype(np.float64)
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    assert np.all(np.abs(got - y) <= R.sum_error(K) * mag)
    d["scales"][:] = 1  # 2^-126: the sums are binary32 subnormals
    d["scales"][::2] = 0
    y, _ = _expect(d)
    assert np.all(np.abs(_f64(_run(d)) - y) <= 2.0 ** -140)


@pytest.mark.parametrize("M", [2, 40, 140])
@pytest.mark.parametrize("xt", ["bf16", "fp16"])
def test_non_finite_values_stay_in_their_row_and_column(M, xt):
    """A NaN or infinity in one row of x, and a NaN scale in one row of w,
    reach only that row and column of y."""
    import torch

    rng = np.random.default_rng(11)
    N, K = 40, 320
    d = _case(rng, M, N, K, xt, "fp32")
    y, mag = _expect(d)
    base = _f64(_run(d))
    for v in (float("nan"), float("inf")):
        e = dict(d, x=d["x"].clone())
        e["x"][1, 77] = v
        got = _f64(_run(e))
        rest = np.arange(M) != 1
        assert np.array_equal(got[rest], base[rest])
        w = R.weights(d["codes"], d["scales"])[:, 77]
        assert np.all(~np.isfinite(got[1][w != 0]))
    e = dict(d, scales=d["scales"].copy())
    e["scales"][13, 4] = 255
    got = _f64(_run(e))
    assert np.all(np.isnan(got[:, 13]))
    rest = np.arange(N) != 13
    assert np.array_equal(got[:, rest], base[:, rest])


@pytest.mark.parametrize("M,N,K", [(4, 300, 1024), (40, 300, 1024), (300, 520, 1280)])
def test_graph_replays_streams_and_repeats_are_bitwise(M, N, K):
    import torch

    rng = np.random.default_rng(13)
    d = _case(rng, M, N, K, "bf16", "bf16", residual=True)
    lin = _linear(d)
    x, res = d["x"].cuda(), d["residual"].cuda()
    want = _run(d, lin)
    out, eager = torch.empty_like(res), torch.empty_like(res)
    lin.forward(x, out, residual=res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.forward(x, out, residual=res)
    for i in range(4):
        out.zero_()
        graph.replay()
        lin.forward(x, eager, residual=res)
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want) and torch.equal(eager.cpu(), want)
    # two streams at once on one handle
    outs = [torch.empty_like(res) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs):
            lin.forward(x, o, residual=res, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs)


def test_refusals_on_the_device():
    import torch
    from quantized_moe_expert_route_amd import binding as B

    rng = np.random.default_rng(15)
    d = _case(rng, 4, 32, 64, "bf16", "bf16")
    lin = _linear(d, max_M=4)
    buf = torch.zeros(4 * 64 + 4 * 32, dtype=torch.bfloat16, device="cuda")
    x, y = buf[:256].view(4, 64), buf[256:].view(4, 32)
    lin.forward(x, y)
    for xx, yy, rr in ((x, buf[128:256].view(4, 32), None),           # y over x
                       (buf[4:260].view(4, 64), torch.zeros(4, 32, dtype=torch.bfloat16, device="cuda"), None),  # misaligned x
                       (x, y, buf[240:368].view(4, 32))):             # residual over part of y
        with pytest.raises(B.MoeError) as e:
            lin.forward(xx, yy, residual=rr)
        assert e.value.status == B.MOE_ERR_INVALID_ARG
    strided = torch.zeros(4, 68, dtype=torch.bfloat16, device="cuda")[:, :64]
    with pytest.raises(B.MoeError):
        lin.forward(strided, y)  # rows not 16-byte aligned
    with pytest.raises(ValueError):
        lin.forward(x.cpu(), y)


@pytest.mark.parametrize("M", [20, 140, 300])
@pytest.mark.parametrize("xt,yt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
def test_whole_pieces_in_place(M, xt, yt):
    """Widths and strides whose pieces of 16 bytes are whole (N 264: in a row's
    last tile only some are), bias and the residual in place, the columns
    between the rows untouched; then the same from an address that allows
    groups of four, and one that allows single elements only."""
    import torch

    rng = np.random.default_rng([M, 17])
    N, K = 264, 160
    d = _case(rng, M, N, K, xt, yt, bias=True, residual=True)
    lin = _linear(d)
    y, mag = _expect(d)
    tol = R.sum_error(K) * mag * 1.01 + R.half_step(yt) * np.abs(y) + (2.0 ** -25 if yt == "fp16" else 0.0)
    got = []
    for start in (0, 4, 1):
        buf = torch.full((M * 280 + 8,), 3.0, dtype=_dt(yt), device="cuda")
        rows = buf[start:start + M * 280].view(M, 280)
        rows[:, :N] = d["residual"].cuda()
        lin.forward(d["x"].cuda(), rows[:, :N], residual=rows[:, :N])
        assert bool((rows[:, N:] == 3.0).all()) and bool((buf[:start] == 3.0).all())
        got.append(rows[:, :N].cpu())
        assert np.all(np.abs(_f64(got[-1]) - y) <= tol)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("M", [3, 20, 130])
def test_rows_more_than_32_bits_apart(M):
    import torch

    rng = np.random.default_rng([M, 19])
    N, K = 48, 160
    d = _case(rng, M, N, K, "bf16", "bf16", residual=True)
    far = (5 << 30) // (2 * (M - 1)) // 8 * 8  # elements between rows: the last 5 GiB behind the first
    big = torch.empty(far * (M - 1) + 512, dtype=torch.bfloat16, device="cuda")
    x, y = (big[at:].as_strided((M, c), (far, 1)) for at, c in ((0, K), (256, N)))
    with pytest.raises(Exception):  # the rows lie between each other: refused as overlapping
        _linear(d).forward(x, y)
    x.copy_(d["x"])
    res = d["residual"].cuda()
    out = torch.empty_like(res)
    _linear(d).forward(x, out, residual=res)
    _check(out.cpu(), d)
    x = d["x"].cuda()
    y.copy_(d["residual"])
    _linear(d).forward(x, y, residual=y)
    _check(y.cpu(), d)


def test_most_rows_and_widest():
    """The largest row count (2^20) and width (2^24) a call may have, exact sums."""
    import torch

    rng = np.random.default_rng(23)
    d = _case(rng, 1 << 20, 8, 32, "bf16", "fp32", integers=True)
    assert torch.equal(_run(d), torch.from_numpy(_expect(d)[0]).float())
    codes = torch.randint(0, 256, (1 << 24, 16), dtype=torch.uint8, device="cuda")
    scales = torch.full((1 << 24, 1), 127, dtype=torch.uint8, device="cuda")
    from quantized_moe_expert_route_amd.binding import Linear

    lin = Linear(codes, scales)
    at = torch.from_numpy(np.r_[0:40, (1 << 24) - 40:1 << 24, rng.integers(0, 1 << 24, 200)]).cuda()
    for M in (1, 20):
        x = torch.from_numpy(rng.integers(-3, 4, (M, 32)).astype(np.float32)).bfloat16()
        out = torch.empty(M, 1 << 24, dtype=torch.float32, device="cuda")
        lin.forward(x.cuda(), out)
        want = R.linear(_f64(x), codes[at].cpu().numpy(), scales[at].cpu().numpy())[0]
        assert np.array_equal(_f64(out[:, at].cpu()), want)


@pytest.mark.parametrize("M,N,K", [(3, 48, 160), (16, 48, 8192), (20, 48, 160), (20, 5000, 160), (40, 16500, 160),
                                   (129, 24600, 160), (65, 33000, 160)])
@pytest.mark.parametrize("xt", ["bf16", "fp16"])
def test_scales_above_bf16_make_their_row_nan(M, N, K, xt):
    """Scale bytes 253 and 254 (no binary32 weight quantizes to them, and bf16
    does not hold all of their weights) are NaN as 255 is, in every kernel:
    their rows of w, and no other, have NaN results. 252 is a number."""
    rng = np.random.default_rng([M, N, K, 31])
    d = _case(rng, M, N, K, xt, "fp32")
    base = _run(d)
    rows = {5: 253, 17: 254, 30: 255, N - 1: 254}
    d["scales"] = d["scales"].copy()
    for n, v in rows.items():
        d["scales"][n, int(rng.integers(0, K // 32))] = v
    got = _run(d)
    nan = np.zeros(N, dtype=bool)
    nan[list(rows)] = True
    assert bool(got[:, nan].isnan().all())
    assert np.array_equal(got[:, ~nan].numpy(), base[:, ~nan].numpy())
    d["scales"][list(rows)] = 252
    d["x"] = (d["x"].float() * 2.0 ** -12).to(_dt(xt))
    assert bool(_run(d).isfinite().all())


@pytest.mark.parametrize("xt,M,N,K", [("bf16", 300, 2600, 160), ("bf16", 140, 8000, 224), ("bf16", 256, 6144, 96),
                                      ("fp16", 300, 4000, 160), ("fp16", 140, 8192, 96)])
def test_narrow_tiles_with_whole_pieces(xt, M, N, K):
    """64 x 128 tiles whose rows of 16-bit y are whole 16-byte pieces: only half
    of a wave's lanes move a piece of a tile's 16 rows, between writes of the
    sums by all of them."""
    import torch

    for extra in (False, True):
        d = _case(np.random.default_rng([M, N, K, 41]), M, N, K, xt, xt, bias=extra, residual=extra, integers=True)
        if xt == "fp16":
            d["scales"] -= np.uint8(6)
        y, mag = _expect(d)
        assert mag.max() < 2.0 ** 22
        assert torch.equal(_run(d), torch.from_numpy(y).float().to(_dt(xt)))
