"""Calls that write a tensor of the caller's in place say so to autograd: a graph that saved the tensor
refuses its backward instead of using the new values."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from gated_delta_rule_31_gb300.autograd import group_norm, linear_attention
from util import cuda_device

pytestmark = pytest.mark.gpu


def randn(*s, dtype=torch.float32):
    return torch.randn(*s, device=cuda_device()).to(dtype)


def step_inputs(B=2, H=2, D=64):
    return randn(B, H, D), randn(B, H, D), randn(B, H, D)


def refuses(result):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        result.sum().backward()


def delta_step(state, out=None):
    q, k, v = step_inputs()
    g, beta = -torch.rand(2, 2, device=q.device), torch.rand(2, 2, device=q.device)
    return gdr.decode_step(q, k, v, g, beta, state, out=out)


def linear_step(state, out=None):
    return gdr.linear_decode_step(*step_inputs(), torch.full((2,), -0.1, device=state.device), state, out=out)


@pytest.mark.parametrize("step", [delta_step, linear_step])
def test_steps(step):
    state = randn(2, 2, 64, 64)
    q = randn(2, 9, 2, 64).requires_grad_()
    k, v = randn(2, 9, 2, 64), randn(2, 9, 2, 64)
    g = torch.full((2,), -0.1, device=q.device)
    before = state._version
    o, _ = linear_attention(q, k, v, g, state)
    step(state)
    assert state._version > before
    refuses(o)

    out = randn(2, 2, 64)
    w = randn(64).requires_grad_()
    y = group_norm(out.view(4, 64), 1, w)
    assert step(state, out=out) is out
    refuses(y)


@pytest.mark.parametrize("which", ["x", "gate"])
def test_norm(which):
    d = dict(x=randn(6, 128), gate=randn(6, 128))
    w = randn(128).requires_grad_()
    y = group_norm(d["x"], 2, w, gate=d["gate"], activation="silu")
    assert gdr.group_norm_fwd(d["x"], 2, gate=d["gate"], activation="silu", out=d[which]) is d[which]
    refuses(y)


@pytest.mark.parametrize("step", [delta_step, linear_step])
def test_out_is_checked(step):
    state = randn(2, 2, 64, 64)
    want = state.clone()
    for out in (randn(2, 2, 32), randn(1, 2, 64), randn(2, 2, 64, dtype=torch.bfloat16), randn(2, 2, 64, 2)[..., 0], torch.zeros(2, 2, 64)):
        with pytest.raises(ValueError, match="out"):
            step(state, out=out)
    assert torch.equal(state, want)


def test_inference_tensors():
    """Tensors made in inference mode have no version to raise, inside it or outside."""
    with torch.inference_mode():
        state, x = randn(2, 2, 64, 64), randn(6, 128)
        delta_step(state, out=randn(2, 2, 64))
        linear_step(state, out=randn(2, 2, 64))
        gdr.group_norm_fwd(x, 2, out=x)
    delta_step(state)
    linear_step(state)
    gdr.group_norm_fwd(x, 2, out=x)
    assert torch.isfinite(state).all() and torch.isfinite(x).all()
