"""Router projection on the GPU against 64-bit sums."""

import numpy as np
import pytest

import ops_ref as R

pytestmark = pytest.mark.gpu


def _case(M, E, H, xt, wt, seed=0):
    import torch

    g = torch.Generator().manual_seed(seed + 7 * M + 11 * E + H)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
    return torch.randn(M, H, generator=g).to(dt[xt]), (torch.randn(E, H, generator=g) / H ** 0.5).to(dt[wt])


def _run(x, w, **kw):
    import torch
    from quantized_moe_expert_route_amd.binding import Router

    r = Router(w.cuda(), x_dtype=x.dtype)
    out = torch.full((x.shape[0], w.shape[0]), float("nan"), device="cuda")
    r.forward(x.cuda(), out, **kw)
    return out.cpu().double().numpy()


def _check(got, x, w):
    xd, wd = x.double().numpy(), w.double().numpy()
    y, mag = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    H = x.shape[1]
    # up to 16 tokens the sums are float64 (H roundings of at most the magnitudes' sum), one rounding at the end
    err = H * 2.0 ** -52 * mag if x.shape[0] <= 16 else R.sum_error(H) * mag
    tol = R.U32 * np.abs(y) * (1 + 1e-6) + err
    assert not np.isnan(got).any()
    assert np.all(np.abs(got - y) <= tol), float((np.abs(got - y) / tol).max())


@pytest.mark.parametrize("M,E,H", [(1, 1, 8), (1, 256, 6144), (2, 3, 40), (4, 256, 6144), (5, 161, 2056),
                                   (13, 60, 2560), (16, 384, 7168), (16, 1024, 512), (17, 64, 1024), (31, 7, 264),
                                   (64, 256, 6144), (65, 129, 2056), (200, 40, 1000), (257, 300, 512),
                                   (1000, 161, 264)])
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "bf16"), ("fp16", "fp32")])
def test_logits(M, E, H, xt, wt):
    x, w = _case(M, E, H, xt, wt)
    _check(_run(x, w), x, w)


def test_strided_rows_and_rows_past_M():
    import torch
    from quantized_moe_expert_route_amd.binding import Router

    for M in (3, 40, 150):
        x, w = _case(M, 33, 520, "bf16", "fp32")
        wide = torch.full((M, 600), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, 16:536] = x.cuda()
        out = torch.full((M + 2, 33), 5.0, device="cuda")
        Router(w.cuda()).forward(wide[:, 16:536], out, M=M)
        got = out.cpu().double().numpy()
        assert np.all(got[M:] == 5.0)
        _check(got[:M], x, w)


def test_values_across_the_range():
    """Large and tiny weights beside each other (fp32 holds more than 16 bits
    can), infinities and NaN in one token only."""
    import torch

    for M in (4, 40):
        x, w = _case(M, 24, 256, "bf16", "fp32")
        w[:, ::3] *= 2.0 ** 60
        w[:, 1::3] *= 2.0 ** -60
        _check(_run(x, w), x, w)
        base = _run(x, w)
        x[2, 9] = float("nan")
        got = _run(x, w)
        rest = np.arange(M) != 2
        assert np.all(np.isnan(got[2])) and np.array_equal(got[rest], base[rest])


@pytest.mark.parametrize("M", [4, 16, 40, 300])
def test_graph_replay_and_repeats(M):
    import torch
    from quantized_moe_expert_route_amd.binding import Router

    x, w = _case(M, 160, 1024, "bf16", "bf16")
    want = _run(x, w)
    r, xg = Router(w.cuda()), x.cuda()
    out, eager = torch.empty(M, 160, device="cuda"), torch.empty(M, 160, device="cuda")
    r.forward(xg, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.forward(xg, out)
    for _ in range(4):
        out.zero_()
        graph.replay()
        r.forward(xg, eager)
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().double().numpy(), want)
        assert np.array_equal(eager.cpu().double().numpy(), want)


def test_feeds_the_routed_call():
    """x -> logits -> moe_forward: the call picks the experts of the 64-bit logits."""
    import torch
    from quantized_moe_expert_route_amd import binding as B

    rng = np.random.default_rng(3)
    for M in (4, 40):
        H, E, I, k = 512, 24, 128, 3
        x, rw = _case(M, E, H, "bf16", "fp32", seed=5)
        w13, s13 = R.random_weights(rng, E, 2 * I, H)
        w2, s2 = R.random_weights(rng, E, H, I)
        cu = lambda a: torch.from_numpy(a).cuda()
        plan = B.Plan(M, H, E, I, k)
        wp, sp = B.pack_w13(cu(w13), cu(s13))
        logits = torch.empty(M, E, device="cuda")
        out = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
        router = B.Router(rw.cuda())
        plan.forward(x.cuda(), router.forward(x.cuda(), logits), wp, sp, cu(w2), cu(s2), out)
        ids = plan.view("topk_ids", torch.int32, (M, k)).cpu().numpy()
        want, _ = R.route((x.double().numpy() @ rw.double().numpy().T).astype(np.float32), k, 2.5)
        assert np.array_equal(ids, want)
        assert torch.isfinite(out.float()).all()


def test_rows_more_than_32_bits_apart_and_most_rows():
    import torch
    from quantized_moe_expert_route_amd.binding import Router

    for M, E in ((3, 40), (40, 40), (600, 300)):  # each of the three kernels
        x, w = _case(M, E, 264, "bf16", "bf16")
        far = (5 << 30) // (2 * (M - 1)) // 8 * 8
        big = torch.empty(far * (M - 1) + 512, dtype=torch.bfloat16, device="cuda").as_strided((M, 264), (far, 1))
        big.copy_(x)
        out = torch.full((M, E), float("nan"), device="cuda")
        Router(w.cuda()).forward(big, out)
        _check(out.cpu().double().numpy(), x, w)
    x, w = _case(1 << 20, 3, 8, "fp16", "fp32")
    _check(_run(x, w), x, w)
    x, w = _case(20, 5, 65536, "bf16", "fp32")
    _check(_run(x, w), x, w)
    _check(_run(x[:9], w), x[:9], w)


def test_wide_tiles_of_every_type_and_non_finite_tokens():
    """64 x 64 tiles, ragged in all three sizes; a NaN token stays alone."""
    for xt, wt in (("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "bf16"), ("fp16", "fp32")):
        x, w = _case(1100, 500, 328, xt, wt)
        base = _run(x, w)
        _check(base, x, w)
        x[77, 100] = float("nan")
        x[1099, 5] = float("inf")
        got = _run(x, w)
        rest = ~np.isin(np.arange(1100), (77, 1099))
        assert np.array_equal(got[rest], base[rest]) and np.all(np.isnan(got[77])) and not np.isfinite(got[1099]).any()


def test_one_handle_on_two_streams():
    import torch
    from quantized_moe_expert_route_amd.binding import Router

    xs = [_case(M, 96, 1024, "bf16", "bf16")[0].cuda() for M in (9, 500)]
    r = Router(_case(9, 96, 1024, "bf16", "bf16")[1].cuda())
    want = [r.forward(x, torch.empty(x.shape[0], 96, device="cuda")).clone() for x in xs]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(8):
        for x, o, s in zip(xs, outs, streams):
            r.forward(x, o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def _row_checks(got, x, w, rows, cols):
    """`got` of token rows and expert columns against 64-bit sums: the same
    infinities and NaN (a sum at a time: no library's way through zeros)."""
    xd, wd = x.double().numpy(), w.double().numpy()
    with np.errstate(all="ignore"):
        for m in rows:
            for e in cols:
                want = float(np.add.reduce(xd[m] * wd[e]))
                assert np.isnan(got[m, e]) == np.isnan(want) and (np.isfinite(want) or np.isnan(want)
                                                                  or got[m, e] == want), (m, e, got[m, e], want)
                if np.isfinite(want):
                    assert np.isfinite(got[m, e])


@pytest.mark.parametrize("M,E,H", [(9, 40, 264), (40, 40, 264), (1024, 256, 328), (1100, 500, 328)])
@pytest.mark.parametrize("xt,wt", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "bf16"), ("fp16", "fp32")])
def test_infinities_and_nan_as_in_64_bits(M, E, H, xt, wt):
    """Infinities in x and in w, met by weights and values that some of their
    16-bit parts are zero of, and NaN of every payload, in each kernel."""
    import torch

    x, w = _case(M, E, H, xt, wt)
    base = _run(x, w)
    w[3] = torch.where(w[3] < 0, -0.5, 0.5).to(w.dtype)  # exact in 8 bits: the lower parts are zero
    x[2], x[5] = 1.0, -2.0
    clean = [m for m in range(M) if m not in (1, 2, 5, 6, M - 1)]
    x[1, 17] = float("inf")
    x[6, 100], x[6, 200] = float("inf"), float("-inf")
    x[M - 1, H - 1] = float("-inf")
    w[7, 30] = float("inf")
    w[9, 31] = float("-inf")
    w[11, 17] = 0.0  # meets x[1]'s infinity
    if wt == "fp32":
        w.view(torch.int32)[13, 5] = 0x7F800001  # a NaN by its low bits alone
        w.view(torch.int32)[14, 6] = -1
    else:
        w[13, 5] = float("nan")
    got = _run(x, w)
    _row_checks(got, x, w, (0, 1, 2, 5, 6, M // 2, M - 1), range(min(E, 40)))
    cols = [e for e in range(E) if e not in (3, 7, 9, 11, 13, 14)]
    assert np.array_equal(got[np.ix_(clean, cols)], base[np.ix_(clean, cols)])


@pytest.mark.parametrize("M,E", [(9, 40), (40, 40), (1024, 256), (1100, 500)])
def test_partial_sums_above_binary32(M, E):
    """Products of up to 2^126 whose partial sums pass binary32's range and
    whose sum does not."""
    import torch

    x, w = _case(M, E, 264, "bf16", "bf16")
    x[4] = 2.0 ** 126
    w[6, :159], w[6, 159:263], w[6, 263] = 1.0, -1.0, -55.0
    xd, wd = x.double().numpy(), w.double().numpy()
    want = float(xd[4] @ wd[6])
    assert want == 0.0
    got = _run(x, w)
    assert got[4, 6] == want
