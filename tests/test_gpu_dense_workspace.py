"""Workspaces of the 16-bit layers: what backward calls that read dy as it is need, and the
head's calls one after another on one workspace."""

import pytest
import torch

from test_gpu_dense import _ints, _nan, _ws

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _dense(N, K, **kw):
    from quantized_moe_expert_route_amd.binding import Dense

    gen = torch.Generator().manual_seed(N)
    return Dense(_ints(gen, N, K).to(BF).cuda(), **kw), gen


@pytest.mark.parametrize("M", [1, 40, 513, 2048])
def test_dy_as_it_is(M):
    """Without dz and dbias the head's backward needs the split sums alone, and gives the same
    bits; calls that read dy otherwise, or want dbias, ask for the rest."""
    from quantized_moe_expert_route_amd import binding as B

    N, K = 4096, 264
    op, gen = _dense(N, K)
    x, dy = _ints(gen, M, K).to(BF).cuda(), _ints(gen, M, N).to(BF).cuda()
    full, plain = op.workspace_bytes(M, train=True), op.workspace_bytes(M, train=True, plain=True)
    assert plain <= full - 2 * M * N and op.workspace_bytes(M) <= plain
    got = []
    for n in (full, plain):
        dx, dw = _nan((M, K), BF), _nan((N, K), BF)
        op.backward(dy, x, dx=dx, dw=dw, workspace=_ws(n))
        got.append((dx, dw))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.equal(got[1][0], (dy.double() @ op.w.double()).float().to(BF))
    assert torch.equal(got[1][1], (dy.double().t() @ x.double()).float().to(BF))
    alone = _nan((M, K), BF)
    op.backward(dy, None, dx=alone, workspace=_ws(plain))
    assert torch.equal(alone, got[0][0])
    wide = torch.zeros(M + 1, N + 4, dtype=BF, device="cuda")
    wide[:M, :N] = dy
    for bad in (dict(dbias=_nan((N,), BF)), dict(dy=wide[:M, 1:N + 1])):
        if plain == full:
            continue
        with pytest.raises(B.MoeError) as e:
            op.backward(**{**dict(dy=dy, x=x, dx=dx, dw=dw, workspace=_ws(plain)), **bad})
        assert e.value.status == B.MOE_ERR_WORKSPACE


def test_plain_where_dz_is_needed():
    """With an activation, or N not a multiple of 8, `plain` saves nothing."""
    for N, act in ((4096, "silu"), (4095, "none")):
        op, _ = _dense(N, 64, activation=act)
        assert op.workspace_bytes(300, train=True, plain=True) == op.workspace_bytes(300, train=True)


def test_head_step_on_one_workspace():
    """Forward, scores, distillation and backward of a head, one after another."""
    from quantized_moe_expert_route_amd import binding as B

    M, V, H, k = 16, 70001, 64, 8
    gen = torch.Generator().manual_seed(1)
    w = (torch.randn(V, H, generator=gen) / 8).to(BF).cuda()
    x = torch.randn(M, H, generator=gen).to(BF).cuda()
    head = B.Dense(w)
    logits = torch.empty(M, V, device="cuda")
    scores = B.TokenScores(V, top_k=k, dtype=logits.dtype)
    distill = B.Distill(V, k=k, dtype=logits.dtype, grad_dtype=x.dtype, temperature=2.0)
    ws = _ws(max(head.workspace_bytes(M, train=True, plain=True), scores.workspace_bytes(M), distill.workspace_bytes(M)))
    head.forward(x, logits, workspace=ws)
    tokens = torch.randint(0, V, (M,), generator=gen).int().cuda()
    logprobs, entropy, loss = (torch.empty(M, device="cuda") for _ in range(3))
    top, ids = torch.empty(M, k, device="cuda"), torch.empty(M, k, dtype=torch.int32, device="cuda")
    scores.forward(logits, tokens, logprobs, entropy=entropy, top_logprobs=top, top_ids=ids, workspace=ws)
    dlogits, dx, dw = torch.empty(M, V, dtype=BF, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    weight = torch.full((M,), 1.0 / M, device="cuda")
    distill.forward_backward(logits, ids, top, weight, loss, dlogits, workspace=ws)
    head.backward(dlogits, x, dx=dx, dw=dw, workspace=ws)
    z = x.double() @ w.double().t()
    lq = torch.log_softmax(z, 1)
    assert (logprobs.double() - lq.gather(1, tokens[:, None].long())[:, 0]).abs().max() < 1e-4
    assert (top.double() - lq.topk(k, 1)[0]).abs().max() < 1e-4
    want = dlogits.double() @ w.double()
    # sums of 70001 exact products in 32 bits, at worst a half step each, and one rounding
    assert ((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 70001 * 2.0 ** -24 * (dlogits.double().abs() @ w.double().abs())).all()
    assert torch.isfinite(loss).all() and not dw.isnan().any()
