"""The few-token MoE layer on the GPU against its 64-bit definition."""

import numpy as np
import pytest

import ops_ref as R

pytestmark = pytest.mark.gpu


class Layer:
    """Inputs of one shape (numpy float64 beside the device tensors), a plan, a router."""

    def __init__(self, M, H, E, I, k, wt="bf16", alike=0.0, seed=0, max_M=None):
        import torch
        from quantized_moe_expert_route_amd import binding as B

        rng = np.random.default_rng([seed, M, H, E, I, k])
        self.M, self.H, self.E, self.I, self.k = M, H, E, I, k
        base = rng.standard_normal((1, H))
        x = np.sqrt(alike) * base + np.sqrt(1 - alike) * rng.standard_normal((M, H))
        self.x = torch.from_numpy(x.astype(np.float32)).bfloat16()
        self.rw = torch.from_numpy((rng.standard_normal((E, H)) / H ** 0.5).astype(np.float32))
        self.rw = self.rw.bfloat16() if wt == "bf16" else self.rw
        self.w13, self.s13 = R.random_weights(rng, E, 2 * I, H, lo=118, hi=121)
        self.w2, self.s2 = R.random_weights(rng, E, H, I, lo=118, hi=121)
        cu = lambda a: torch.from_numpy(a).cuda()
        self.plan = B.Plan(M if max_M is None else max_M, H, E, I, k)
        self.g13 = B.pack_w13(cu(self.w13), cu(self.s13))
        self.g2 = (cu(self.w2), cu(self.s2))
        self.router = B.Router(self.rw.cuda())

    def call(self, x=None, out=None, **kw):
        import torch

        x = self.x.cuda() if x is None else x
        if out is None:
            out = torch.full((x.shape[0], self.H), float("nan"), dtype=torch.bfloat16, device="cuda")
        return self.plan.layer(x, self.router, *self.g13, *self.g2, out, **kw)

    def reference(self, x=None):
        x = self.x if x is None else x
        return R.layer(x.double().numpy(), self.rw.double().numpy(), self.w13, self.s13, self.w2, self.s2, self.k, 2.5)

    def check(self, got, x=None):
        import torch

        M = got.shape[0]
        out, err, ids, wt = self.reference(x)
        g = got.cpu().double().numpy()
        assert np.array_equal(self.plan.view("topk_ids", torch.int32, (M, self.k)).cpu().numpy(), ids)
        w = self.plan.view("topk_w", torch.float32, (M, self.k)).cpu().double().numpy()
        assert np.all(np.abs(w - wt) <= (self.k + 4) * 2 * R.U32 * wt)
        tol = err * (1 + R.half_step("bf16")) + R.half_step("bf16") * np.abs(out)
        assert not np.isnan(g).any()
        bad = np.abs(g - out) > tol
        assert not bad.any(), (int(bad.sum()), float((np.abs(g - out) / tol).max()))


SHAPES = [(1, 512, 1, 128, 1), (1, 512, 16, 128, 2), (4, 512, 16, 128, 2), (3, 1024, 7, 256, 7), (13, 2560, 60, 384, 6),
          (16, 512, 300, 512, 16), (16, 1536, 40, 256, 8), (7, 4096, 33, 128, 5), (5, 8192, 12, 512, 3),
          (16, 6144, 20, 256, 8), (2, 7168, 9, 384, 4), (9, 512, 1024, 128, 8)]


@pytest.mark.parametrize("M,H,E,I,k", SHAPES)
@pytest.mark.parametrize("wt,alike", [("bf16", 0.0), ("fp32", 0.9)])
def test_layer(M, H, E, I, k, wt, alike):
    d = Layer(M, H, E, I, k, wt, alike)
    d.check(d.call())


def test_same_experts_and_all_experts():
    """Every token on the same experts (identical tokens), and every expert picked by all."""
    d = Layer(16, 512, 32, 128, 4, alike=1.0)
    got = d.call()
    d.check(got)
    assert bool((got == got[0]).all())
    d = Layer(16, 512, 16, 128, 16)
    d.check(d.call())


def test_ties_go_to_the_lower_expert():
    import torch

    d = Layer(6, 512, 24, 128, 5)
    d.rw[12:] = d.rw[:12]  # every logit twice
    from quantized_moe_expert_route_amd.binding import Router

    d.router = Router(d.rw.cuda())
    d.check(d.call())
    d.rw.zero_()  # all logits equal: experts 0..k-1
    d.router = Router(d.rw.cuda())
    d.check(d.call())
    assert torch.equal(d.plan.view("topk_ids", torch.int32, (6, 5)).cpu(), torch.arange(5, dtype=torch.int32).repeat(6, 1))


def test_fewer_tokens_than_the_plan_and_rows_behind_them():
    import torch

    d = Layer(16, 1024, 30, 256, 4, max_M=40)
    whole = d.call()
    d.check(whole)
    x = d.x.cuda()
    for M in (0, 1, 2, 7, 15, 16):
        out = torch.full((16, 1024), 9.0, dtype=torch.bfloat16, device="cuda")
        d.call(x=x, out=out, M=M)
        assert bool((out[M:] == 9.0).all())
        if M:
            d.check(out[:M], d.x[:M])
            # a token's result does not depend on the tokens beside it beyond the order of its experts' sums
            assert torch.allclose(out[:M].float(), whole[:M].float(), rtol=2.0 ** -7, atol=1e-3)


def test_calls_of_all_kinds_on_one_plan():
    """Layer calls between calls of moe_forward, at changing sizes, on one workspace: both keep their results."""
    import torch

    d = Layer(16, 512, 24, 128, 3, max_M=64)
    rng = np.random.default_rng(1)
    x64 = torch.from_numpy(rng.standard_normal((64, 512)).astype(np.float32)).bfloat16().cuda()
    logits = d.router.forward(x64, torch.empty(64, 24, device="cuda"))

    def forward(M):
        out = torch.empty((M, 512), dtype=torch.bfloat16, device="cuda")
        d.plan.forward(x64, logits, *d.g13, *d.g2, out, M=M)
        return out

    want = {M: forward(M).clone() for M in (3, 16, 40, 64)}
    layer = {M: d.call(x=d.x.cuda()[:M]).clone() for M in (1, 4, 16)}
    d.check(d.call())
    for _ in range(3):
        for M, L in ((3, 16), (40, 1), (64, 4), (16, 16)):
            assert torch.equal(forward(M), want[M])
            assert torch.equal(d.call(x=d.x.cuda()[:L]), layer[L])


def test_changing_inputs_one_workspace():
    import torch

    d = Layer(16, 512, 40, 128, 6)
    for i in range(12):
        rng = np.random.default_rng(100 + i)
        M = int(rng.integers(1, 17))
        x = torch.from_numpy(rng.standard_normal((M, 512)).astype(np.float32)).bfloat16()
        d.check(d.call(x=x.cuda()), x)


@pytest.mark.parametrize("M", [1, 4, 16])
def test_graph_replays_equal_eager(M):
    import torch

    d = Layer(M, 1536, 40, 256, 8)
    x = d.x.cuda()
    want = d.call().clone()
    out = torch.empty_like(want)
    d.call(x=x, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.call(x=x, out=out)
    for i in range(5):
        out.zero_()
        graph.replay()
        eager = d.call(x=x)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)
    d.check(out)


def test_two_plans_on_two_streams():
    import torch

    a, b = Layer(4, 6144, 24, 256, 8, seed=1), Layer(16, 2048, 60, 384, 4, seed=2)
    want = [p.call().clone() for p in (a, b)]
    xs = [p.x.cuda() for p in (a, b)]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, x, o, s in zip((a, b), xs, outs, streams):
            p.call(x=x, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_non_finite_tokens_and_experts_stay_apart():
    """A token of infinities or NaN leaves the other tokens' results; weights
    that overflow in one expert reach only the tokens that picked it."""
    import torch

    d = Layer(6, 512, 12, 128, 2)
    base = d.call().clone()
    ids = d.reference()[2]
    for v in (float("nan"), float("inf")):
        x = d.x.clone()
        x[3] = v
        got = d.call(x=x.cuda())
        rest = [t for t in range(6) if t != 3]
        assert torch.equal(got[rest], base[rest])
    e = int(ids[0, 0])
    hit = np.any(ids == e, 1)
    assert not hit.all()
    s2 = d.s2.copy()
    s2[e] = 254
    out = torch.empty_like(base)
    d.plan.layer(d.x.cuda(), d.router, *d.g13, d.g2[0], torch.from_numpy(s2).cuda(), out)
    assert torch.equal(out[torch.from_numpy(~hit).cuda()], base[torch.from_numpy(~hit).cuda()])


def test_decode_step_through_all_operators():
    """A decode step: projection with the residual, the layer, an output head
    in fp32, each on the one before; the router's own call gives the layer's routing."""
    import torch
    from quantized_moe_expert_route_amd import binding as B

    rng = np.random.default_rng(21)
    d = Layer(8, 1024, 40, 256, 4, wt="fp32")
    co, so = R.random_weights(rng, 1024, 512, lo=119, hi=121)
    ch, sh = R.random_weights(rng, 3001, 1024, lo=118, hi=120)
    cu = lambda a: torch.from_numpy(a).cuda()
    attn = torch.from_numpy(rng.standard_normal((8, 512)).astype(np.float32)).bfloat16()
    x = d.x.cuda()
    B.Linear(cu(co), cu(so)).forward(attn.cuda(), x, residual=x)  # x += attn Wo^T
    y, mag = R.linear(attn.double().numpy(), co, so, residual=d.x.double().numpy())
    x1 = x.cpu()
    assert np.all(np.abs(x1.double().numpy() - y) <= R.sum_error(512) * mag * 1.01 + R.half_step("bf16") * np.abs(y))
    moe = d.call(x=x)
    d.check(moe, x1)
    logits = d.router.forward(x, torch.empty(8, 40, device="cuda"))
    assert np.array_equal(R.route(logits.cpu().numpy(), 4, 2.5)[0], d.reference(x1)[2])
    head = torch.empty(8, 3001, device="cuda")
    B.Linear(cu(ch), cu(sh)).forward(moe, head)
    y, mag = R.linear(moe.cpu().double().numpy(), ch, sh)
    assert np.all(np.abs(head.cpu().double().numpy() - y) <= R.sum_error(1024) * mag + R.U32 * np.abs(y))


def test_refusals_on_the_device():
    import torch
    from quantized_moe_expert_route_amd import binding as B

    d = Layer(4, 512, 8, 128, 2, max_M=20)
    out = torch.empty(17, 512, dtype=torch.bfloat16, device="cuda")

    def status(**kw):
        with pytest.raises(B.MoeError) as e:
            d.call(**kw)
        return e.value.status

    assert status(x=torch.zeros_like(out), out=out) == B.MOE_ERR_UNSUPPORTED  # 17 tokens
    x = d.x.cuda()
    assert status(x=x, out=x) == B.MOE_ERR_INVALID_ARG                       # in place
    d.plan.set_mid_format(B.MID_MXFP4)
    assert status() == B.MOE_ERR_UNSUPPORTED
    d.plan.set_mid_format(B.MID_E4M3)
    d.plan.set_weight_layout(0)
    assert status() == B.MOE_ERR_UNSUPPORTED
    d.plan.set_weight_layout(B.LAYOUT_W13_PACKED)
    d.plan.set_shared_slot(True)
    assert status() == B.MOE_ERR_UNSUPPORTED
    d.plan.set_shared_slot(False)
    keep = d.router
    d.router = B.Router(torch.zeros(8, 1024, dtype=torch.bfloat16, device="cuda"))  # other H
    assert status() == B.MOE_ERR_INVALID_ARG
    d.router = B.Router(d.rw.cuda(), x_dtype=torch.float16)
    assert status() == B.MOE_ERR_INVALID_ARG
    d.router = keep
    d.check(d.call())
    wide = B.Plan(4, 8704, 2, 128, 1)
    with pytest.raises(B.MoeError) as e:
        wide.layer(torch.zeros(4, 8704, dtype=torch.bfloat16, device="cuda"),
                   B.Router(torch.zeros(2, 8704, dtype=torch.bfloat16, device="cuda")),
                   torch.zeros(2 * 128 * 8704, dtype=torch.uint8, device="cuda"),
                   torch.zeros(2 * 128 * 544, dtype=torch.uint8, device="cuda"),
                   torch.zeros(2 * 64 * 8704, dtype=torch.uint8, device="cuda"),
                   torch.zeros(2 * 4 * 8704, dtype=torch.uint8, device="cuda"),
                   torch.zeros(4, 8704, dtype=torch.bfloat16, device="cuda"))
    assert e.value.status == B.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("M,H,E,I,k", [(16, 8192, 20, 512, 16), (9, 3584, 300, 256, 7), (12, 8192, 260, 128, 4),
                                       (16, 7168, 64, 384, 9), (6, 4608, 130, 512, 10)])
def test_widest_and_slots_shared_by_both_halves(M, H, E, I, k):
    """The widest hidden and expert sizes, K-steps that do not divide by the
    waves, and experts that tokens of both halves of the batch picked."""
    d = Layer(M, H, E, I, k, alike=0.5)
    d.check(d.call())


def test_two_graphs_share_a_plan():
    """Two captured calls of different sizes on one plan's workspace, replayed
    in turn with eager calls between them."""
    import torch

    d = Layer(16, 1024, 40, 256, 4)
    x = d.x.cuda()
    sizes = (3, 16)
    want = [d.call(x=x[:M]).clone() for M in sizes]
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    for M, o in zip(sizes, outs):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.call(x=x[:M], out=o)
        graphs.append(g)
    for i in range(4):
        for o in outs:
            o.zero_()
        for g in graphs[::1 if i % 2 else -1]:
            g.replay()
            d.call(x=x[:7])
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_inputs_inside_the_workspace_are_refused():
    import torch
    from quantized_moe_expert_route_amd import binding as B

    d = Layer(4, 512, 8, 128, 2)
    inside = d.plan.workspace.view(torch.bfloat16)[:4 * 512].view(4, 512)
    for kw in (dict(x=inside), dict(out=inside)):
        with pytest.raises(B.MoeError) as e:
            d.call(**kw)
        assert e.value.status == B.MOE_ERR_INVALID_ARG


def test_every_logit_nan():
    """Routing of a batch whose logits are all NaN (also the NaN of all ones)
    stays inside the expert list; the next call is as before."""
    import torch
    from quantized_moe_expert_route_amd.binding import Router

    for E in (8, 70, 300):
        d = Layer(16, 512, E, 128, 5)
        want = d.call().clone()
        keep = d.router
        for bits in (-1, 0x7FC00000):
            d.router = Router(torch.full((E, 512), bits, dtype=torch.int32, device="cuda").view(torch.float32))
            d.call()
            ids = d.plan.view("topk_ids", torch.int32, (16, 5))
            assert int(ids.min()) >= 0 and int(ids.max()) < E
        d.router = keep
        assert torch.equal(d.call(), want)


@pytest.mark.parametrize("M,E,H,I", [(1, 1, 512, 128), (4, 1, 512, 256), (6, 2, 1024, 384), (16, 1, 512, 512),
                                     (13, 3, 4608, 256)])
def test_h_keeps_32_bits(M, E, H, I):
    """Sums that cancel: every product and sum is a multiple of 1/4 below 2^22
    (exact in binary32), and a row of W2 takes one h from another near to it, so
    that an h held in fewer bits shows in the output's 8. Also more tokens on one
    expert than one pass of the down product takes."""
    import torch
    from quantized_moe_expert_route_amd import binding as B

    rng = np.random.default_rng([M, E, H, I, 29])
    mags = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    x = rng.integers(1, 5, (M, H)).astype(np.float64)
    keep = 512  # the other columns of W13 are zero
    gate, up = rng.choice([2, 4, 5, 6], (E, I, H)), rng.choice([2, 4, 5, 6, 10, 12, 13, 14], (E, I, H))
    w13 = np.concatenate([gate, up], 1)
    w13[:, :, keep:] = 0
    value = lambda c: np.where(c >= 8, -mags[c & 7], mags[c & 7])
    rw = np.zeros((E, H))
    rw[:, :8] = rng.integers(0, 5, (E, 8))  # scores above 1/2: the one slot's weight is exactly 1
    picks = np.argmax(x @ rw.T, 1)  # ties go to the lower expert
    h = np.stack([value(w13[picks[t]]) @ x[t] for t in range(M)])
    h = h[:, :I] * h[:, I:]  # SiLU is its argument where that is above 104
    assert (value(w13[:, :I]) @ x.T).min() > 104 and np.abs(h).max() < 2 ** 22
    w2 = np.zeros((E, H, I), dtype=np.int64)
    for e in range(E):
        t = np.flatnonzero(picks == e)
        order = np.argsort(h[t[0]] if len(t) else rng.random(I))
        for n in range(H):  # n: neighbours of the expert's tokens in turn
            if len(t):
                order = np.argsort(h[t[n % len(t)]])
            i = int(rng.integers(0, I - 1))
            w2[e, n, order[i]], w2[e, n, order[i + 1]] = 2, 10  # 1 and -1
    pack = lambda c: (c[..., ::2] | (c[..., 1::2] << 4)).astype(np.uint8)
    cu = lambda a: torch.from_numpy(a).cuda()
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")
    plan = B.Plan(M, H, E, I, 1, routed_scaling=1.0)
    out = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    plan.layer(torch.from_numpy(x).bfloat16().cuda(), B.Router(torch.from_numpy(rw).bfloat16().cuda()),
               *B.pack_w13(cu(pack(w13)), one(E, 2 * I, H // 32)), cu(pack(w2)), one(E, H, I // 32), out)
    want = np.stack([value(w2[picks[t]]) @ h[t] for t in range(M)])
    assert np.abs(want).max() < 2 ** 22
    assert torch.equal(out.cpu(), torch.from_numpy(want).float().bfloat16())


@pytest.mark.parametrize("M", [1, 16])
def test_stage_and_call_events(M):
    """Events set on the plan are recorded by a layer call too, not left with
    an earlier call's times."""
    import torch
    from quantized_moe_expert_route_amd import binding as B

    d = Layer(M, 1024, 24, 256, 4)
    d.call()
    n = len(B.stage_names())
    ev = B.HipEvents(2 * n + 2)
    s = torch.cuda.current_stream()
    try:
        for _ in range(2):
            d.plan.set_stage_events(ev.handles[:2 * n])
            ev.record(2 * n, s)
            want = d.call()
            ev.record(2 * n + 1, s)
            torch.cuda.synchronize()
            used = [i for i, name in enumerate(B.stage_names()) if name in ("route", "gate_up", "down")]
            for i in range(n):
                assert ev.elapsed_ms(2 * n, 2 * i) >= 0 and ev.elapsed_ms(2 * i + 1, 2 * n + 1) >= 0
                assert ev.elapsed_ms(2 * i, 2 * i + 1) > 0 if i in used else ev.elapsed_ms(2 * i, 2 * i + 1) >= 0
            for a, b in zip(used, used[1:]):  # in order
                assert ev.elapsed_ms(2 * a + 1, 2 * b) >= 0
            d.check(want)
            d.plan.set_call_events(*ev.handles[:2])
            ev.record(2 * n, s)
            d.call()
            ev.record(2 * n + 1, s)
            torch.cuda.synchronize()
            assert ev.elapsed_ms(2 * n, 0) >= 0 and ev.elapsed_ms(0, 1) > 0 and ev.elapsed_ms(1, 2 * n + 1) >= 0
        d.plan.set_call_events(None, None)
        d.check(d.call())
    finally:
        d.plan.set_call_events(None, None)
        ev.close()
