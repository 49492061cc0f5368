"""The group norm on tensors that start off the 16-byte grid, and in place: the same values as anywhere else.

Bounds as for aligned tensors: one rounding to bf16 (2^-9), or fp32 sums of up to 64 roundings in a row
and an activation good to a few units (128 x 2^-24). The fp32 sums of dw and db have the latter in both."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from linear_ref import group_norm, rel
from util import cuda_device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {"bf16": 1.1 * 2.0 ** -9, "fp32": 128 * 2.0 ** -24}
SHAPES = [(4, 32), (32, 128), (1, 4096), (8, 33), (4, 6), (6, 99), (2, 2047), (1, 5001)]


def make(rows, C, dtype):
    gen = torch.Generator().manual_seed(C)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=(2 * randn(rows, C) + 0.5).to(dtype), gate=randn(rows, C).to(dtype), dy=randn(rows, C).to(dtype),
                weight=1 + 0.3 * randn(C), bias=0.3 * randn(C))


def placed(t, offset, dev):
    """A contiguous copy that starts `offset` values into its memory."""
    return torch.empty(t.numel() + offset, dtype=t.dtype, device=dev)[offset:].view(t.shape).copy_(t)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offsets", [(1, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 3, 0, 0), (2, 2, 2, 2, 2), (4, 4, 4, 4, 4), (0, 0, 0, 1, 3)])
@pytest.mark.parametrize("groups,D", SHAPES)
def test_offsets(groups, D, offsets, dtype):
    dev = cuda_device()
    d = make(21, groups * D, TYPES[dtype])
    leaf = {n: d[n].double().requires_grad_() for n in ("x", "gate", "weight", "bias")}
    ref = group_norm(leaf["x"], groups, leaf["weight"], leaf["bias"], leaf["gate"], "silu")
    want = dict(zip(leaf, torch.autograd.grad(ref, list(leaf.values()), d["dy"].double())))
    x, gate, dy, weight, bias = (placed(d[n], k, dev) for n, k in zip(("x", "gate", "dy", "weight", "bias"), offsets))
    out = placed(d["x"], offsets[0], dev)
    y = gdr.group_norm_fwd(x, groups, weight, bias, gate, activation="silu", out=out)
    assert rel(y, ref) <= TOL[dtype]
    got = gdr.group_norm_bwd(x, groups, weight, bias, gate, dy, activation="silu")
    for n in leaf:
        assert rel(got["d" + n], want[n]) <= (TOL[dtype] if n in ("x", "gate") else TOL["fp32"]), n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("groups,D", SHAPES + [(8, 257), (2, 4100)])
def test_in_place(groups, D, gated, dtype):
    """Onto x and onto the gate; groups that start inside a vector are read and written beside their neighbours."""
    dev = cuda_device()
    d = {n: t.to(dev) for n, t in make(1300, groups * D, TYPES[dtype]).items()}
    gate = d["gate"] if gated else None
    args = d["weight"], d["bias"]
    want = gdr.group_norm_fwd(d["x"], groups, *args, gate, activation="silu")
    y = d["x"].clone()
    assert gdr.group_norm_fwd(y, groups, *args, gate, activation="silu", out=y) is y and torch.equal(y, want)
    if gated:
        y = gate.clone()
        assert gdr.group_norm_fwd(d["x"], groups, *args, y, activation="silu", out=y) is y and torch.equal(y, want)
