"""The codes of refused linear attention and group norm calls: a bad argument is not an unsupported one."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from util import cuda_device

pytestmark = pytest.mark.gpu

INVALID, UNSUPPORTED = gdr.GDR_ERR_INVALID_ARG, gdr.GDR_ERR_UNSUPPORTED


def code(call, *args, **kw):
    with pytest.raises(gdr.GdrError) as e:
        call(*args, **kw)
    return e.value.code


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hk,Hv,D,scale,want", [(1, 2, 64, float("nan"), INVALID), (2, 3, 64, 1.0, INVALID), (0, 2, 64, 1.0, INVALID),
                                                (1, 2, 96, 1.0, UNSUPPORTED)])
def test_linear(Hk, Hv, D, scale, want, dtype):
    dev = cuda_device()
    q, v = torch.zeros(1, 4, Hk, D, dtype=dtype, device=dev), torch.zeros(1, 4, Hv, D, dtype=dtype, device=dev)
    g = torch.zeros(Hv, device=dev)
    assert code(gdr.linear_fwd, q, q, v, g, scale=scale) == want
    assert code(gdr.linear_fwd, q, q, v, g, scale=scale, save_states=True) == want
    assert code(gdr.linear_bwd, q, q, v, g, None, v, scale=scale) == want
    assert code(gdr.linear_decode_step, *(t[:, 0].contiguous() for t in (q, q, v)), g,
                torch.zeros(1, Hv, D, D, device=dev), scale=scale) == want


@pytest.mark.parametrize("C,eps,want", [(64, 0.0, INVALID), (64, float("nan"), INVALID), (8193, 1e-5, UNSUPPORTED)])
def test_norm(C, eps, want):
    x = torch.zeros(3, C, device=cuda_device())
    assert code(gdr.group_norm_fwd, x, 1, eps=eps) == want
    assert code(gdr.group_norm_bwd, x, 1, None, None, None, x, eps=eps) == want
