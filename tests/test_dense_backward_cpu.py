"""Backward calls without x, which only dw reads."""

import pytest
import torch

from quantized_moe_expert_route_amd import binding as B
from test_dense_head_cpu import BF, CPU, _bare


@pytest.mark.parametrize("cls", [B.Dense, B.Gated])
def test_x_is_read_for_dw_alone(cls):
    """Without dw the call reaches the library (which refuses the missing handle); with it
    the binding asks for x."""
    sizes = dict(N=24, K=64, activation="silu", bias=None) if cls is B.Dense else dict(I=24, H=64)
    op = _bare(cls, device=CPU, max_M=4, dtype=BF, _code=B.BF16, **sizes)
    dy, dx = torch.zeros(4, 24, dtype=BF), torch.zeros(4, 64, dtype=BF)
    pre = dy if cls is B.Dense else torch.zeros(4, 48, dtype=BF)
    dw = torch.zeros(24 if cls is B.Dense else 48, 64, dtype=BF)
    with pytest.raises(B.MoeError) as e:
        op.backward(dy, None, pre=pre, dx=dx, stream=_Stream)
    assert e.value.status == B.MOE_ERR_INVALID_ARG
    for x in (None, dx.float(), dx[:2]):
        with pytest.raises((TypeError, ValueError)):
            op.backward(dy, x, pre=pre, dx=dx, dw=dw, stream=_Stream)
    with pytest.raises(ValueError):
        op.backward(dy, dx[:2], pre=pre, dx=dx, stream=_Stream)


class _Stream:
    cuda_stream = 0


def test_kernel_names_refuse_a_missing_handle():
    L = B.lib()
    assert L.moe_scores_kernel(None, 1) is None and L.moe_distill_kernel(None, 1, 0) is None
    for cls in (B.TokenScores, B.Distill):
        with pytest.raises(ValueError):
            _bare(cls, device=CPU, max_M=4).kernel(1)
