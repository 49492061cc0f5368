"""Infinite gates and weights in the group norm's backward: sums over rows that are infinite (or zero) by the
formula stay so, whatever the number of rows that the lanes of a block share."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from util import cuda_device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SHAPES = [(4, 64), (1, 4096), (4, 33), (3, 99), (1, 8191)]  # whole vectors, wide groups, groups inside vectors, single values
AT = 5


def make(rows, C, dtype):
    gen = torch.Generator().manual_seed(rows)
    x, gate = (torch.randn(rows, C, generator=gen).to(dtype) for _ in range(2))
    return x, gate, 1 + 0.3 * torch.rand(C, generator=gen), 0.3 * torch.randn(C, generator=gen)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [3, 700, 5001])
@pytest.mark.parametrize("groups,D", SHAPES)
def test_infinite_gates(groups, D, rows, dtype):
    """silu(inf) = inf, so with dy = 1 db is inf, and with dy the sign of the normalised value dw is."""
    dev = cuda_device()
    x, gate, w, b = make(rows, groups * D, TYPES[dtype])
    gate[:, AT] = float("inf")
    t = x.double().view(rows, groups, D)
    dy = (t - t.mean(-1, keepdim=True)).view(rows, -1).sign().to(x.dtype)  # no value of these equals its mean
    assert dy[:, AT].all()
    args = [t.to(dev) for t in (w, b, gate)]
    got = gdr.group_norm_bwd(x.to(dev), groups, *args, dy.to(dev), activation="silu")
    assert got["dweight"][AT] == float("inf")
    assert torch.isfinite(got["dweight"][:AT]).all() and torch.isfinite(got["dbias"][:AT]).all()
    got = gdr.group_norm_bwd(x.to(dev), groups, *args, torch.ones_like(x).to(dev), activation="silu")
    assert got["dbias"][AT] == float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("groups,D", SHAPES)
def test_infinite_weights(groups, D, rows, dtype):
    """Without a gate n = inf times a value, where the sigmoid has no slope: nothing reaches dw and db."""
    dev = cuda_device()
    x, _, w, b = make(rows, groups * D, TYPES[dtype])
    w[AT] = float("inf")
    got = gdr.group_norm_bwd(x.to(dev), groups, w.to(dev), b.to(dev), None, torch.ones_like(x).to(dev), activation="sigmoid")
    assert got["dweight"][AT] == 0 and got["dbias"][AT] == 0
