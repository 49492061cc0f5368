"""The per-token group norm on the GPU against its definition in 64 bits, gradients by automatic
differentiation of that definition.

Bounds, on ||x - ref|| / ||ref||: bf16 results are computed in fp32 and rounded once (2^-9; fp32 error
below 2^-16 beside it). fp32 results: statistics over D and sums over the rows in fp32, taken as
sums of up to 64 roundings in a row, and an activation good to a few units: 128 x 2^-24. Constant rows: x - mean
is the rounding of x, at most 2^-24 |x| (times 1/sqrt(eps))."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from linear_ref import group_norm, rel
from util import cuda_device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {"bf16": 1.1 * 2.0 ** -9, "fp32": 128 * 2.0 ** -24}


def make(rows, C, dtype, gate, affine, seed=0, mean=0.5):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    d = dict(x=(randn(rows, C) * 2 + mean).to(dtype), dy=randn(rows, C).to(dtype))
    d["gate"] = (randn(rows, C) * 2).to(dtype) if gate else None
    d["weight"] = 1 + 0.3 * randn(C) if affine else None
    d["bias"] = 0.3 * randn(C) if affine else None
    return d


def check(d, groups, dev, dtype, **kw):
    names = [n for n in ("x", "gate", "weight", "bias") if d[n] is not None]
    leaf = {n: d[n].double().requires_grad_() for n in names}
    ref = group_norm(leaf["x"], groups, leaf.get("weight"), leaf.get("bias"), leaf.get("gate"), **kw)
    grads = dict(zip(names, torch.autograd.grad(ref, [leaf[n] for n in names], d["dy"].double(), materialize_grads=True)))
    x = {n: t.to(dev) if t is not None else None for n, t in d.items()}
    y = gdr.group_norm_fwd(x["x"], groups, x["weight"], x["bias"], x["gate"], **kw)
    assert y.dtype == d["x"].dtype and rel(y, ref) <= TOL[dtype]
    got = gdr.group_norm_bwd(x["x"], groups, x["weight"], x["bias"], x["gate"], x["dy"], **kw)
    for n in names:
        assert rel(got["d" + n], grads[n]) <= (TOL[dtype] if n in ("x", "gate") else TOL["fp32"]), n
    return y, got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("groups,D", [(1, 8), (3, 1), (2, 7), (5, 24), (32, 64), (32, 128), (3, 100), (4, 256), (6, 99), (2, 264),
                                      (2, 600), (1, 1024), (1, 1030), (1, 4096), (2, 2047), (1, 8192), (1, 8191)])
def test_group_sizes(groups, D, dtype):
    if D == 1:  # one value is its own mean: the root-mean-square form alone has something to say
        check(make(33, groups, TYPES[dtype], True, True), groups, cuda_device(), dtype, activation="silu", center=False)
    else:
        check(make(33, groups * D, TYPES[dtype], True, True, seed=D), groups, cuda_device(), dtype, activation="silu")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("activation", ["none", "silu", "sigmoid"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("center", [False, True])
def test_forms(activation, gate, affine, center, dtype):
    check(make(50, 4 * 64, TYPES[dtype], gate, affine, seed=1), 4, cuda_device(), dtype, activation=activation,
          center=center, eps=1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 2, 607, 608, 609, 5001])
def test_rows(rows, dtype):
    check(make(rows, 5 * 40, TYPES[dtype], True, True, seed=rows), 5, cuda_device(), dtype, activation="silu")


def test_no_rows():
    dev = cuda_device()
    x, w = torch.empty(0, 64, device=dev), torch.ones(64, device=dev)
    assert gdr.group_norm_fwd(x, 2, w, w).shape == (0, 64)
    gr = gdr.group_norm_bwd(x, 2, w, w, None, x)
    assert not gr["dweight"].any() and not gr["dbias"].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_constant_and_zero_rows(dtype):
    dev = cuda_device()
    x = torch.zeros(4, 2 * 64, dtype=TYPES[dtype])
    x[1], x[2], x[3, :64] = 3.0, -0.7, 1e4
    b = torch.randn(128, generator=torch.Generator().manual_seed(0))
    y = gdr.group_norm_fwd(x.to(dev), 2, None, b.to(dev))
    want = b.expand(4, 128).to(TYPES[dtype]).float()
    assert torch.allclose(y.float().cpu(), want, rtol=2.0 ** -8, atol=1e4 * 2.0 ** -22 / 1e-5 ** 0.5)
    assert torch.equal(y[0].float().cpu(), want[0])
    gr = gdr.group_norm_bwd(x.to(dev), 2, None, b.to(dev), None, torch.ones_like(x).to(dev))
    assert torch.isfinite(gr["dx"].float()).all()
    assert torch.equal(gr["dbias"].cpu(), torch.full((128,), 4.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_gates_and_offsets(dtype):
    d = make(20, 128, TYPES[dtype], True, True, mean=30.0)
    d["gate"] = d["gate"] * 60
    check(d, 2, cuda_device(), dtype, activation="silu")
    check(d, 2, cuda_device(), dtype, activation="sigmoid")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [1, 3, 8])
def test_unaligned_tensors(offset, dtype):
    """Contiguous slices that start off the 16-byte grid give the same values."""
    dev = cuda_device()
    d = make(9, 4 * 32, TYPES[dtype], True, True, seed=2)
    want, _ = check(d, 4, dev, dtype, activation="silu")
    x = torch.empty(9 * 128 + offset, dtype=TYPES[dtype], device=dev)[offset:].view(9, 128)
    x.copy_(d["x"])
    y = gdr.group_norm_fwd(x, 4, d["weight"].to(dev), d["bias"].to(dev), d["gate"].to(dev), activation="silu")
    assert rel(y, want) <= TOL[dtype]
    gr = gdr.group_norm_bwd(x, 4, d["weight"].to(dev), d["bias"].to(dev), d["gate"].to(dev), d["dy"].to(dev), activation="silu")
    assert torch.isfinite(gr["dweight"]).all()


def test_in_place_and_leading_dims():
    dev = cuda_device()
    d = make(30, 128, torch.bfloat16, True, False)
    x, z = d["x"].to(dev).view(2, 15, 2, 64).view(2, 15, 128), d["gate"].to(dev).view(2, 15, 128)
    want = gdr.group_norm_fwd(x, 2, gate=z, activation="silu")
    got = gdr.group_norm_fwd(x.clone(), 2, gate=z, activation="silu", out=None)
    assert torch.equal(want, got)
    y = x.clone()
    assert gdr.group_norm_fwd(y, 2, gate=z, activation="silu", out=y) is y and torch.equal(y, want)


def test_repeats_bitwise_on_another_stream():
    dev = cuda_device()
    d = {n: t.to(dev) for n, t in make(3000, 512, torch.bfloat16, True, True).items()}
    args = (d["x"], 4, d["weight"], d["bias"], d["gate"], d["dy"])
    want = gdr.group_norm_bwd(*args, activation="silu")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gdr.group_norm_bwd(*args, activation="silu")
    side.synchronize()
    assert all(torch.equal(want[n], got[n]) for n in want)


def test_autograd_and_differences():
    from gated_delta_rule_31_gb300.autograd import group_norm as op

    dev = cuda_device()
    d = make(12, 96, torch.float32, True, True)
    leaf = {n: d[n].to(dev).requires_grad_() for n in ("x", "weight", "bias", "gate")}
    y = op(leaf["x"], 3, leaf["weight"], leaf["bias"], leaf["gate"], activation="silu")
    got = torch.autograd.grad(y, list(leaf.values()), d["dy"].to(dev))

    def loss(**kw):
        e = {n: t.double() for n, t in {**d, **kw}.items()}
        return float((group_norm(e["x"], 3, e["weight"], e["bias"], e["gate"], "silu") * e["dy"]).sum())

    for n, g in zip(leaf, got):
        u = torch.randn(d[n].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
        eps = 1e-5
        num = (loss(**{n: d[n].double() + eps * u}) - loss(**{n: d[n].double() - eps * u})) / (2 * eps)
        # differences: eps^2 times third derivatives of order one, and 1e-16 / eps of the loss
        assert abs(float((g.cpu().double() * u).sum()) - num) <= 1e-5 * float(g.cpu().double().norm() * u.norm()), n


def test_more_than_two_to_the_31_values():
    dev = cuda_device()
    rows, C = 2 ** 31 // 4096 + 40, 4096
    x = torch.empty(rows, C, dtype=torch.bfloat16, device=dev).normal_(generator=torch.Generator(device=dev).manual_seed(0))
    y = gdr.group_norm_fwd(x, 32, gate=x, activation="silu")
    last = x[-8:].cpu().double()
    assert rel(y[-8:], group_norm(last, 32, gate=last, activation="silu")) <= TOL["bf16"]
    gr = gdr.group_norm_bwd(x, 32, None, None, None, y, activation="silu")
    leaf = last.clone().requires_grad_()
    (want,) = torch.autograd.grad(group_norm(leaf, 32, activation="silu"), leaf, y[-8:].cpu().double())
    assert rel(gr["dx"][-8:], want) <= TOL["bf16"]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("groups,D", [(8, 1), (8, 33), (4, 6), (12, 10), (4, 514), (2, 1500), (8, 257), (8, 1025), (2, 4100), (8, 8191),
                                      (4, 33), (12, 301), (4, 2051)])
def test_groups_that_start_inside_a_vector(groups, D, dtype):
    """Rows start on 16 bytes, groups between: the results, and a group whose neighbour holds NaN. (Not the
    gradients of single values: x / sqrt(x^2 + eps) leaves dx = g r (1 - h^2), a difference of equals that
    loses x^2 / eps times fp32's precision.)"""
    dev = cuda_device()
    kw = dict(activation="silu", center=D > 1)
    d = make(19, groups * D, TYPES[dtype], True, True, seed=D)
    x = {n: t.to(dev) for n, t in d.items()}
    if D > 1:
        y, got = check(d, groups, dev, dtype, **kw)
    else:
        y = gdr.group_norm_fwd(x["x"], groups, x["weight"], x["bias"], x["gate"], **kw)
        assert rel(y, group_norm(*(d[n].double() if n else groups for n in ("x", "", "weight", "bias", "gate")), **kw)) <= TOL[dtype]
        got = gdr.group_norm_bwd(x["x"], groups, x["weight"], x["bias"], x["gate"], x["dy"], **kw)
    bad = slice(D, 2 * D)
    for n in ("x", "gate", "dy"):
        x[n][3, bad] = float("nan")
    y2 = gdr.group_norm_fwd(x["x"], groups, x["weight"], x["bias"], x["gate"], **kw)
    got2 = gdr.group_norm_bwd(x["x"], groups, x["weight"], x["bias"], x["gate"], x["dy"], **kw)
    here = torch.zeros(19, groups * D, dtype=torch.bool, device=dev)
    here[3, bad] = True
    for a, b in ((y2, y), (got2["dx"], got["dx"]), (got2["dgate"], got["dgate"])):
        assert a[here].isnan().all() and torch.equal(a[~here], b[~here])
    for n in ("dweight", "dbias"):
        assert got2[n][bad].isnan().all()
        assert torch.equal(got2[n][:D], got[n][:D]) and torch.equal(got2[n][2 * D:], got[n][2 * D:])
