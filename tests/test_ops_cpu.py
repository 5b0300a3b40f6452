"""Host-side checks of the operators beside the routed-MoE call: every refusal
comes before any device work, and the 64-bit references of their GPU tests
agree with brute force. No GPU."""

import ctypes

import numpy as np
import pytest
import torch

import ops_ref as R
from oracle import moe as O
from quantized_moe_expert_route_amd import binding as B

A, A2, A3 = 0x10000, 0x2000000, 0x4000000  # host addresses, never dereferenced: every case fails first


def _router_create(E=8, H=64, xt=B.BF16, w=A, wt=B.BF16, mm=16):
    h = ctypes.c_void_p()
    st = B.lib().moe_router_create(E, H, xt, w, wt, mm, ctypes.byref(h))
    assert not h.value
    return st


@pytest.mark.parametrize("change,status", [
    (dict(w=None), B.MOE_ERR_INVALID_ARG),
    (dict(w=A + 8), B.MOE_ERR_INVALID_ARG),
    (dict(E=0), B.MOE_ERR_INVALID_ARG),
    (dict(H=-8), B.MOE_ERR_INVALID_ARG),
    (dict(mm=-1), B.MOE_ERR_INVALID_ARG),
    (dict(xt=B.FP32), B.MOE_ERR_INVALID_ARG),
    (dict(wt=B.FP16), B.MOE_ERR_INVALID_ARG),
    (dict(xt=7), B.MOE_ERR_INVALID_ARG),
    (dict(E=1025), B.MOE_ERR_UNSUPPORTED),
    (dict(H=60), B.MOE_ERR_UNSUPPORTED),
    (dict(H=65544), B.MOE_ERR_UNSUPPORTED),
    (dict(mm=(1 << 20) + 1), B.MOE_ERR_UNSUPPORTED),
    (dict(), B.MOE_ERR_DEVICE),  # a host address
])
def test_router_refusals(change, status):
    assert _router_create(**change) == status


def test_null_handles():
    L = B.lib()
    assert L.moe_router_create(8, 64, B.BF16, A, B.BF16, 16, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_router_forward(None, 1, A, 64, A2, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_linear_create(16, 32, B.BF16, A, A2, None, 16, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_linear_forward(None, 1, A, 32, None, 0, A2, 16, B.BF16, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_layer_forward(None, None, 1, A, A, A, A, A, A2, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_router_kernel(None, 1) is None and L.moe_linear_kernel(None, 1) is None
    L.moe_router_destroy(None)
    L.moe_linear_destroy(None)


def _pack_bytes(N, K):
    w, s = ctypes.c_size_t(), ctypes.c_size_t()
    st = B.lib().moe_linear_pack_bytes(N, K, ctypes.byref(w), ctypes.byref(s))
    return st, w.value, s.value


def test_linear_pack_bytes():
    assert _pack_bytes(16, 128) == (B.MOE_OK, 1024, 64)
    assert _pack_bytes(17, 160) == (B.MOE_OK, 4 * 1024, 4 * 64)  # padded to whole 16 x 128 pieces
    assert _pack_bytes(0, 32)[0] == B.MOE_ERR_INVALID_ARG
    assert _pack_bytes(4, 0)[0] == B.MOE_ERR_INVALID_ARG
    assert _pack_bytes(4, 48)[0] == B.MOE_ERR_UNSUPPORTED
    assert _pack_bytes(4, 65568)[0] == B.MOE_ERR_UNSUPPORTED
    assert _pack_bytes((1 << 24) + 1, 32)[0] == B.MOE_ERR_UNSUPPORTED
    assert B.lib().moe_linear_pack_bytes(16, 128, None, None) == B.MOE_ERR_INVALID_ARG


def test_pack_linear_refusals():
    L = B.lib()
    b, c, d = 0x200000, 0x400000, 0x600000
    assert L.moe_pack_linear(None, b, 16, 128, c, d, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_pack_linear(A, b, 16, 128, None, d, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_pack_linear(A + 4, b, 16, 128, c, d, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_pack_linear(A, b, 16, 128, A + 512, d, None) == B.MOE_ERR_INVALID_ARG  # over the input
    assert L.moe_pack_linear(A, b, 16, 128, c, c + 16, None) == B.MOE_ERR_INVALID_ARG   # over each other
    assert L.moe_pack_linear(A, b, 16, 100, c, d, None) == B.MOE_ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert L.moe_pack_linear(A, b, 16, 128, c, d, None) == B.MOE_ERR_DEVICE


@pytest.mark.parametrize("change,status", [
    (dict(N=0), B.MOE_ERR_INVALID_ARG),
    (dict(K=40), B.MOE_ERR_UNSUPPORTED),
    (dict(xt=B.FP32), B.MOE_ERR_INVALID_ARG),
    (dict(w=None), B.MOE_ERR_INVALID_ARG),
    (dict(s=A2 + 4), B.MOE_ERR_INVALID_ARG),
    (dict(bias=A3 + 2), B.MOE_ERR_INVALID_ARG),
    (dict(mm=-1), B.MOE_ERR_INVALID_ARG),
    (dict(mm=1 << 21), B.MOE_ERR_UNSUPPORTED),
    (dict(), B.MOE_ERR_DEVICE),
])
def test_linear_refusals(change, status):
    a = dict(N=16, K=128, xt=B.BF16, w=A, s=A2, bias=None, mm=16, **{})
    a.update(change)
    h = ctypes.c_void_p()
    st = B.lib().moe_linear_create(a["N"], a["K"], a["xt"], a["w"], a["s"], a["bias"], a["mm"], ctypes.byref(h))
    assert st == status and not h.value


def _bare(cls, **attrs):
    h = cls.__new__(cls)
    h._h = None
    for key, v in attrs.items():
        setattr(h, key, v)
    return h


def test_binding_refuses_bad_tensors():
    """The binding checks every tensor before the library sees its pointer
    (objects without a device handle: the checks come first)."""
    cpu = torch.device("cpu")
    lin = _bare(B.Linear, device=cpu, max_M=4, N=24, K=64, x_dtype=torch.bfloat16, bias=None, _fp32=torch.float32)
    x, y = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 24, dtype=torch.bfloat16)
    for bad in (dict(x=x.float()), dict(x=x[:, :32]), dict(x=torch.zeros(64, 4, dtype=torch.bfloat16).t()),
                dict(x=torch.zeros(5, 64, dtype=torch.bfloat16)), dict(out=y.half()), dict(out=y[:2]),
                dict(out=y[:, :23]), dict(residual=y.float()), dict(residual=y[:1]),
                dict(out=y.float(), residual=y), dict(M=5), dict(x=x[:1].expand(4, 64))):
        with pytest.raises(ValueError):
            lin.forward(**dict(dict(x=x, out=y), **bad))
    with pytest.raises(TypeError):
        lin.forward(x, None)
    rt = _bare(B.Router, device=cpu, max_M=4, E=8, H=64, x_dtype=torch.bfloat16, _fp32=torch.float32)
    lg = torch.zeros(4, 8)
    for bad in (dict(x=x.half()), dict(logits=lg.double()), dict(logits=torch.zeros(4, 16)[:, :8]),
                dict(logits=lg[:3]), dict(x=x[:, ::2]), dict(M=-1)):
        with pytest.raises(ValueError):
            rt.forward(**dict(dict(x=x, logits=lg), **bad))
    for bad in (dict(w=torch.zeros(4, 30, dtype=torch.uint8)), dict(w=torch.zeros(4, 32, dtype=torch.int8)),
                dict(s=torch.zeros(4, 1, dtype=torch.uint8)), dict(bias=torch.zeros(4))):
        with pytest.raises(ValueError):
            B.Linear(**dict(dict(w=torch.zeros(4, 32, dtype=torch.uint8), s=torch.zeros(4, 2, dtype=torch.uint8)),
                            **bad))
    with pytest.raises(ValueError):
        B.Router(torch.zeros(4, 64, dtype=torch.bfloat16).t())
    with pytest.raises(ValueError):
        B.Router(torch.zeros(4, 64, dtype=torch.float64))


def test_layer_binding_refuses_bad_tensors():
    M, H, E, I = 4, 512, 16, 128
    p = B.Plan.__new__(B.Plan)
    p._h = ctypes.c_void_p()
    p.shape = B.moe_shape(M, H, E, I, 2, 2.5, 0)
    p.device = torch.device("cpu")
    rt = _bare(B.Router, device=p.device, max_M=4, E=E, H=H, x_dtype=torch.bfloat16)
    u8 = lambda n: torch.zeros(n, dtype=torch.uint8)
    good = dict(x=torch.zeros((M, H), dtype=torch.bfloat16), router=rt, w13=u8(E * I * H), s13=u8(E * I * H // 16),
                w2=u8(E * H * I // 2), s2=u8(E * H * I // 32), out=torch.zeros((M, H), dtype=torch.bfloat16))
    for bad in (dict(x=torch.zeros((M, H))), dict(x=torch.zeros((M + 1, H), dtype=torch.bfloat16)), dict(M=-1),
                dict(w13=u8(E * I * H - 1)), dict(s2=u8(E * H * 16)), dict(out=torch.zeros((M - 1, H), dtype=torch.int16))):
        with pytest.raises(ValueError):
            p.layer(**dict(good, **bad))
    with pytest.raises(TypeError):
        p.layer(**dict(good, router=torch.zeros(E, H)))


def test_workspace_of_the_layer_is_behind_the_call():
    """The layer's regions add little, and nothing in front of the call's."""
    b = B.shape_workspace_bytes(4, 6144, 256, 256, 8)
    assert b % 256 == 0 and b < 2 << 20
    big = B.shape_workspace_bytes(4096, 6144, 256, 512, 8)
    assert big < 4096 * 8 * 6144 * 4 * 1.5  # at most 16 tokens' worth for a large plan


def test_reference_weights_and_linear():
    rng = np.random.default_rng(0)
    codes, scales = R.random_weights(rng, 3, 64)
    W = R.weights(codes, scales)
    mags = [0, .5, 1, 1.5, 2, 3, 4, 6]
    for n in range(3):
        for k in range(64):
            c = (int(codes[n, k // 2]) >> (4 * (k % 2))) & 15
            assert W[n, k] == (-1) ** (c >> 3) * mags[c & 7] * 2.0 ** (int(scales[n, k // 32]) - 127)
    x = rng.standard_normal((2, 64))
    y, mag = R.linear(x, codes, scales, bias=np.ones(3))
    for m in range(2):
        for n in range(3):
            s = sum(x[m, k] * W[n, k] for k in range(64)) + 1
            assert abs(y[m, n] - s) < 1e-12 * mag[m, n]


def test_reference_layer_against_the_dense_definition():
    rng = np.random.default_rng(1)
    M, H, E, I, k = 3, 64, 6, 32, 2
    x, rw = rng.standard_normal((M, H)), rng.standard_normal((E, H)) / 8
    w13, s13 = R.random_weights(rng, E, 2 * I, H)
    w2, s2 = R.random_weights(rng, E, H, I)
    out, err, ids, wt = R.layer(x, rw, w13, s13, w2, s2, k, 2.5)
    logits = (x @ rw.T).astype(np.float32)
    o_ids, o_w = O.route(logits, k, 2.5)
    assert np.array_equal(ids, o_ids) and np.allclose(wt, o_w, rtol=1e-6)
    dense = np.zeros((M, H))
    for e in range(E):  # every expert over every token, masked
        gu = x @ R.weights(w13[e], s13[e]).T
        y = (gu[:, :I] / (1 + np.exp(-gu[:, :I])) * gu[:, I:]) @ R.weights(w2[e], s2[e]).T
        dense += y * (wt * (ids == e)).sum(1)[:, None]
    assert np.allclose(out, dense, rtol=1e-12, atol=1e-12)
    assert np.all(err > 0) and np.median(err / np.abs(out)) < 2e-2


@pytest.mark.parametrize("kw,nbytes", [
    (dict(M=4, H=6144, E=256, I=256, top_k=8, shared_I=256), 4208640),
    (dict(M=4096, H=6144, E=256, I=512, top_k=8, shared_I=512), 1102433536),
    (dict(M=64, H=16384, E=64, I=128, top_k=4), 17579264),
    (dict(M=0, H=512, E=16, I=128, top_k=2), 1024),
])
def test_plans_without_the_layer_pay_nothing_for_it(kw, nbytes):
    """Shapes that moe_layer_forward refuses need the workspace they needed
    before it was there."""
    assert B.shape_workspace_bytes(**kw) == nbytes
