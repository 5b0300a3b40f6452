"""Host-side checks of the layers in 16 bits and of the operators on the head's
logits: every refusal comes before any device work. No GPU."""

import ctypes

import pytest
import torch

from quantized_moe_expert_route_amd import binding as B

A, A2, A3 = 0x10000, 0x20000000, 0x40000000  # host addresses, never dereferenced: every case fails first
BAD, NOT, DEV, WS = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_DEVICE, B.MOE_ERR_WORKSPACE


def _create(name, *args):
    h = ctypes.c_void_p()
    st = getattr(B.lib(), name)(*args, ctypes.byref(h))
    assert not h.value
    return st


@pytest.mark.parametrize("change,status", [
    (dict(N=0), BAD), (dict(K=-8), BAD), (dict(mm=-1), BAD), (dict(t=B.FP32), BAD), (dict(t=9), BAD),
    (dict(w=None), BAD), (dict(w=A + 8), BAD), (dict(bias=A2 + 1), BAD), (dict(act=-1), BAD), (dict(act=5), BAD),
    (dict(K=60), NOT), (dict(K=65544), NOT), (dict(N=(1 << 22) + 1), NOT), (dict(mm=(1 << 20) + 1), NOT), (dict(), DEV),
])
def test_dense_create(change, status):
    a = dict(N=16, K=64, t=B.BF16, w=A, bias=None, act=0, mm=16)
    a.update(change)
    assert _create("moe_dense_create", *a.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(I=0), BAD), (dict(H=0), BAD), (dict(mm=-1), BAD), (dict(t=B.FP32), BAD), (dict(w=None), BAD),
    (dict(w=A + 2), BAD), (dict(act=0), BAD), (dict(act=5), BAD), (dict(H=68), NOT), (dict(H=1 << 17), NOT),
    (dict(I=(1 << 21) + 1), NOT), (dict(I=1 << 62), NOT), (dict(mm=1 << 21), NOT), (dict(), DEV),
])
def test_gated_create(change, status):
    a = dict(I=16, H=64, t=B.FP16, w=A, act=2, mm=16)
    a.update(change)
    assert _create("moe_gated_create", *a.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(V=0), BAD), (dict(k=-1), BAD), (dict(k=101), NOT), (dict(k=65), NOT), (dict(V=10, k=11), BAD), (dict(t=3), BAD),
    (dict(mm=-1), BAD), (dict(V=(1 << 24) + 1), NOT), (dict(mm=(1 << 20) + 1), NOT),
])
def test_scores_create(change, status):
    a = dict(V=100, k=8, t=B.FP32, mm=16)
    a.update(change)
    assert _create("moe_scores_create", *a.values()) == status


@pytest.mark.parametrize("change,status", [
    (dict(V=0), BAD), (dict(k=0), BAD), (dict(k=65), NOT), (dict(t=-1), BAD), (dict(gt=B.FP32), BAD), (dict(gt=4), BAD),
    (dict(T=0.0), BAD), (dict(T=-1.0), BAD), (dict(T=float("inf")), BAD), (dict(T=float("nan")), BAD), (dict(T=1e-39), BAD),
    (dict(mm=-1), BAD), (dict(V=1 << 25), NOT), (dict(mm=1 << 21), NOT),
])
def test_distill_create(change, status):
    a = dict(V=100, k=8, t=B.BF16, gt=B.FP16, T=1.0, mm=16)
    a.update(change)
    assert _create("moe_distill_create", *a.values()) == status


def test_null_handles():
    L = B.lib()
    n = ctypes.c_size_t()
    assert L.moe_dense_create(16, 64, 0, A, None, 0, 1, None) == BAD
    assert L.moe_gated_create(16, 64, 0, A, 2, 1, None) == BAD
    assert L.moe_scores_create(16, 1, 0, 1, None) == BAD
    assert L.moe_distill_create(16, 1, 0, 0, 1.0, 1, None) == BAD
    for f in (L.moe_dense_destroy, L.moe_gated_destroy, L.moe_scores_destroy, L.moe_distill_destroy):
        f(None)
    assert L.moe_dense_workspace_bytes(None, 1, 0, ctypes.byref(n)) == BAD
    assert L.moe_gated_workspace_bytes(None, 1, 0, ctypes.byref(n)) == BAD
    assert L.moe_scores_workspace_bytes(None, 1, ctypes.byref(n)) == BAD
    assert L.moe_distill_workspace_bytes(None, 1, ctypes.byref(n)) == BAD
    assert L.moe_dense_forward(None, 1, A, 64, None, 0, A2, 16, 0, None, 0, 0, None, 0, None) == BAD
    assert L.moe_dense_backward(None, 1, A, 16, None, 0, 0, A2, 64, A3, 64, None, None, None, 0, None) == BAD
    assert L.moe_gated_forward(None, 1, A, 64, A2, 16, None, 0, None, 0, None) == BAD
    assert L.moe_gated_backward(None, 1, A, 16, A2, 0, A3, 64, None, 0, A, None, 0, None) == BAD
    assert L.moe_scores_forward(None, 1, A, 16, A2, A3, None, None, None, None, None, 0, None) == BAD
    assert L.moe_distill_forward(None, 1, A, 16, A2, A3, A, None, None, 0, None) == BAD
    assert L.moe_distill_backward(None, 1, A, 16, A2, A3, A, A, A, 16, None) == BAD
    assert L.moe_distill_forward_backward(None, 1, A, 16, A2, A3, A, A, A, 16, None, 0, None) == BAD


def _bare(cls, **attrs):
    h = cls.__new__(cls)
    h._h = None
    for key, v in attrs.items():
        setattr(h, key, v)
    return h


CPU = torch.device("cpu")
BF = torch.bfloat16


def test_binding_refuses_bad_tensors_dense():
    """The binding checks every tensor before the library sees its pointer."""
    op = _bare(B.Dense, device=CPU, max_M=4, N=24, K=64, dtype=BF, activation="silu", _code=B.BF16, bias=None)
    x, y, w = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 24, dtype=BF), torch.zeros(24, 64, dtype=BF)
    base = dict(x=x, out=y, residual=y, pre=y)
    for bad in (dict(x=x.float()), dict(x=x[:, :32]), dict(x=torch.zeros(64, 4, dtype=BF).t()), dict(x=None), dict(x=x[:0], M=1),
                dict(x=torch.zeros(5, 64, dtype=BF)), dict(out=y.half()), dict(out=y[:2]), dict(residual=y.float()),
                dict(residual=y[:, :20]), dict(pre=y.double()), dict(pre=y[:3]), dict(M=-1), dict(M=5),
                dict(workspace=torch.zeros(8)), dict(workspace=torch.zeros(16, dtype=torch.uint8)[::2])):
        with pytest.raises((ValueError, TypeError, AttributeError)):
            op.forward(**{**base, **bad})
    base = dict(dy=y, x=x, dx=x, dw=w, dbias=y[0], pre=y)
    for bad in (dict(dy=y.float()), dict(dy=y[:, :8]), dict(x=x[:2]), dict(dx=x.half()), dict(dw=w[:20]), dict(pre=None),
                dict(dw=torch.zeros(24, 128, dtype=BF)[:, :64]), dict(dbias=y[0, :20]), dict(dbias=y[0].float()),
                dict(dbias=torch.zeros(48, dtype=BF)[::2]), dict(M=9)):
        with pytest.raises((ValueError, TypeError)):
            op.backward(**{**base, **bad})


def test_binding_refuses_bad_tensors_gated():
    op = _bare(B.Gated, device=CPU, max_M=4, I=12, H=64, dtype=BF, _code=B.BF16)
    x, h, pre, w = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 12, dtype=BF), torch.zeros(4, 24, dtype=BF), torch.zeros(24, 64, dtype=BF)
    for bad in (dict(x=x.half()), dict(out=h[:, :8]), dict(pre=pre[:, :12]), dict(pre=torch.zeros(4, 48, dtype=BF)[:, :24]),
                dict(pre=pre[:3]), dict(M=5), dict(workspace=x)):
        with pytest.raises(ValueError):
            op.forward(**{**dict(x=x, out=h, pre=pre), **bad})
    for bad in (dict(dh=pre), dict(x=x[:1]), dict(dx=x[:, :32]), dict(dw=w.half()), dict(dw=w[:12]), dict(pre=h), dict(M=-1)):
        with pytest.raises(ValueError):
            op.backward(**{**dict(dh=h, x=x, pre=pre, dx=x, dw=w), **bad})
    with pytest.raises(ValueError):
        B.Gated(torch.zeros(3, 64, dtype=BF))
    with pytest.raises(ValueError):
        B.Gated(w, activation="swish")
    with pytest.raises(ValueError):
        B.Dense(w.float())
    with pytest.raises(ValueError):
        B.Dense(w, bias=torch.zeros(24))


def test_binding_refuses_bad_tensors_head():
    f32, i32 = torch.float32, torch.int32
    op = _bare(B.TokenScores, device=CPU, max_M=4, V=50, top_k=3, dtype=f32, _fp32=f32, _i32=i32)
    z, v, n = torch.zeros(4, 50), torch.zeros(4), torch.zeros(4, dtype=i32)
    top, ids = torch.zeros(4, 3), torch.zeros(4, 3, dtype=i32)
    base = dict(logits=z, tokens=n, logprobs=v, entropy=v, lse=v, top_logprobs=top, top_ids=ids)
    for bad in (dict(logits=z.half()), dict(logits=z[:, :40]), dict(tokens=n.long()), dict(tokens=n[:3]), dict(logprobs=v[:2]),
                dict(entropy=v.double()), dict(lse=torch.zeros(8)[::2]), dict(top_logprobs=None), dict(top_ids=ids.long()),
                dict(top_ids=torch.zeros(4, 4, dtype=i32)[:, :3]), dict(M=5)):
        with pytest.raises(ValueError):
            op.forward(**{**base, **bad})
    op = _bare(B.Distill, device=CPU, max_M=4, V=50, k=3, dtype=BF, grad_dtype=BF, _fp32=f32, _i32=i32)
    zb = z.to(BF)
    base = dict(logits=zb, ids=ids, t=top, weight=v, loss=v, grad=zb)
    for bad in (dict(logits=z), dict(ids=ids.long()), dict(ids=ids[:, :2]), dict(t=top.double()), dict(t=top[:3]),
                dict(weight=v[:3]), dict(loss=n), dict(grad=z), dict(grad=zb[:, :49]), dict(M=-1)):
        with pytest.raises(ValueError):
            op.forward_backward(**{**base, **bad})
    for bad in (dict(lse=v[:1]), dict(lse=v.half()), dict(weight=v.half())):
        with pytest.raises(ValueError):
            op.backward(**{**dict(logits=zb, ids=ids, t=top, lse=v, weight=v, grad=zb), **bad})
    with pytest.raises(ValueError):
        op.forward(zb, ids, top, v, lse=v.double())
