"""An error that a caller's earlier HIP call left behind is not a call's own:
every entry point that launches returns ok after it."""

import ctypes

import numpy as np
import pytest

import ops_ref as R

pytestmark = pytest.mark.gpu


def test_calls_after_a_failed_call_of_the_caller():
    import torch
    from quantized_moe_expert_route_amd import binding as B

    M, H, E, I, k, N = 4, 512, 16, 128, 2, 96
    rng = np.random.default_rng(37)
    cu = lambda a: torch.from_numpy(a).cuda()
    w13, s13 = (cu(a) for a in R.random_weights(rng, E, 2 * I, H))
    w2, s2 = (cu(a) for a in R.random_weights(rng, E, H, I))
    x = cu(rng.standard_normal((M, H)).astype(np.float32)).bfloat16()
    router = B.Router(cu(rng.standard_normal((E, H)).astype(np.float32)))
    lin = B.Linear(*(cu(a) for a in R.random_weights(rng, N, H)))
    plan = B.Plan(M, H, E, I, k)
    timed = B.Plan(M, H, E, I, k)  # launches with events around them
    ev = B.HipEvents(2)
    timed.set_call_events(*ev.handles)
    packed = B.pack_w13(w13, s13)
    packed2 = B.pack_w2(w2, s2)
    bf16 = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    logits, y, out, out2, out3 = torch.empty(M, E, device="cuda"), bf16(M, N), bf16(M, H), bf16(M, H), bf16(M, H)
    calls = {
        "pack_w13": lambda: B.pack_w13(w13, s13, out=packed),
        "pack_w2": lambda: B.pack_w2(w2, s2, out=packed2),
        "router": lambda: router.forward(x, logits),
        "linear": lambda: lin.forward(x, y),
        "layer": lambda: plan.layer(x, router, *packed, w2, s2, out),
        "forward": lambda: plan.forward(x, logits, *packed, w2, s2, out2),
        "noalloc": lambda: plan.forward_noalloc(x, logits, *packed, w2, s2, out3),
        "timed": lambda: timed.forward(x, logits, *packed, w2, s2, out3),
    }
    for f in calls.values():
        f()
    torch.cuda.synchronize()
    want = [t.clone() for t in (logits, y, out, out2)]
    for t in (logits, y, out, out2):
        t.zero_()
    torch.cuda.synchronize()
    hip = ctypes.CDLL("libamdhip64.so")
    failed = []
    for name, f in calls.items():
        assert hip.hipSetDevice(1 << 20) != 0
        try:
            f()
        except B.MoeError as e:
            failed.append((name, e.status))
        hip.hipGetLastError()  # (clears it for torch)
    torch.cuda.synchronize()
    ev.close()
    assert not failed
    for t, w in zip((logits, y, out, out2), want):
        assert torch.equal(t, w)
