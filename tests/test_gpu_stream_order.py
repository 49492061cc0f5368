"""Calls in a row on one stream, each taking the one before it as input, give what they give when the
stream is waited for after every call. Decode steps start while the kernel before them ends, so nothing
of theirs may be read before that kernel, and those before it, are complete."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from util import cuda_device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
B, H, D = 24, 8, 128  # 192 (batch, head) pairs: the CTAs of several steps fit the GPU at once


def inputs(dtype, seed):
    dev = cuda_device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *s, to=dtype: torch.randn(*s, generator=gen, device=dev).to(to)  # noqa: E731
    f32 = torch.float32
    return dict(q=randn(B, H, D), k=randn(B, H, D), v=randn(B, H, D), decay=-torch.rand(H, generator=gen, device=dev),
                g=-torch.rand(B, H, generator=gen, device=dev), beta=torch.rand(B, H, generator=gen, device=dev),
                linear=randn(B, H, D, D, to=f32), delta=randn(B, H, D, D, to=f32),
                prompt=[randn(B, 40, H, D) for _ in range(3)])


def delta(x, q, k=None, v=None):
    return gdr.decode_step(q, x["k"] if k is None else k, x["v"] if v is None else v, x["g"], x["beta"], x["delta"])


def linear(x, q, k=None):
    return gdr.linear_decode_step(q, x["k"] if k is None else k, x["v"], x["decay"], x["linear"])


def steps_in_turn(x, wait):
    a = wait(linear(x, x["q"]))
    b = wait(delta(x, a))
    c = wait(linear(x, b))
    return a, b, c, wait(delta(x, c, v=a))


def two_linear_steps_then_delta(x, wait):
    a = wait(linear(x, x["q"]))
    b = wait(linear(x, a))
    return a, b, wait(delta(x, a, k=b))


def delta_steps(x, wait):
    """One step's result is an input of the next, and of the one after it."""
    a = wait(delta(x, x["q"]))
    b = wait(delta(x, x["q"], v=a))
    c = wait(delta(x, a, k=b))
    return a, b, c, wait(delta(x, c, k=b))


def prompt_then_step(x, wait):
    q, k, v = x["prompt"]
    o, state = gdr.linear_fwd(q, k, v, x["decay"], x["linear"])
    last = o.view(B * 40 * H * D)[-B * H * D:].view(B, H, D)
    wait(o)
    a = wait(delta(x, last))
    return o, a, wait(gdr.linear_decode_step(a, last, x["v"], x["decay"], state)), state


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("chain", [steps_in_turn, two_linear_steps_then_delta, delta_steps, prompt_then_step])
def test_chained_calls(chain, dtype):
    def waited(t):
        torch.cuda.synchronize()
        return t

    def done(x, out):
        return [t.clone() for t in (*out, x["linear"], x["delta"])]

    x = inputs(TYPES[dtype], 1)
    want = done(x, chain(x, waited))
    assert all(torch.isfinite(t.float()).all() for t in want)
    x = inputs(TYPES[dtype], 1)
    torch.cuda.synchronize()
    got = done(x, chain(x, lambda t: t))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # The same launches in a graph, with no host time between them, and what they read changed before each
    # replay, so that a value read too early is an older one.
    x = inputs(TYPES[dtype], 1)
    start = {n: x[n].clone() for n in ("q", "linear", "delta")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(x, lambda t: t)
    for t in out:
        t.zero_()
    for i in range(10):
        for n, t in start.items():
            x[n].copy_(t)
        if i % 2:
            x["q"].neg_()
        graph.replay()
        if i % 2 == 0:
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, done(x, out))), i
