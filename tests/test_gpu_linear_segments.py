"""Linear attention in bf16 over several segments (and in fp32 beside it): the state handed from one segment to
the next, forwards and in reverse, against the recurrence in 64 bits.

Bounds as for one segment, on ||x - ref|| / ||ref|| for each head: bf16 results round the weights in
a chunk, the state and the result once to bf16 each (up to 2^-9 each), so 3 x 2^-9. What is returned in
fp32 is a sum of fp32 products in fp32: 256 x 2^-24."""
import ctypes

import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from linear_ref import linear, make, rel_heads
from util import cuda_device, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
FP32 = 256 * 2.0 ** -24
TOL = {"bf16": 3 * 2.0 ** -9, "fp32": FP32}


def segments(B, T, Hk, Hv, Dk, Dv, dtype):
    p = gdr.LinearProblem(B, T, Hk, Hv, Dk, Dv, {"bf16": 1, "fp32": 0}[dtype], 1.0)
    return (gdr.lib().gdr_linear_fwd_workspace(ctypes.byref(p)) - 256) // (4 * B * Hv * Dk * Dv)


def check(shape, dtype, **kw):
    assert segments(*shape, dtype) > 1
    d = make(*shape, TYPES[dtype], **kw)
    ref = linear(**d)
    x = to_dev(d, cuda_device())
    args = x["q"], x["k"], x["v"], x["g"], x["h0"]
    o, ht, states = gdr.linear_fwd(*args, lengths=x["lengths"], save_states=True)
    gr = gdr.linear_bwd(*args, x["do"], x["dht"], lengths=x["lengths"])
    assert rel_heads(o, ref["o"], 2) <= TOL[dtype]
    assert rel_heads(ht, ref["ht"], 1) <= FP32
    for n in ("dq", "dk", "dv"):
        assert rel_heads(gr[n], ref[n], 2) <= TOL[dtype], n
    assert rel_heads(gr["dh0"], ref["dh0"], 1) <= FP32
    if d["lengths"] is not None:
        for b, n in enumerate(d["lengths"].tolist()):
            for t in (o, gr["dq"], gr["dk"], gr["dv"]):
                assert not t[b, n:].any()
    # Results that are not asked for change none of the others, and the kept states stand for those formed again.
    plain, none = gdr.linear_fwd(*args, lengths=x["lengths"], output_final_state=False)
    assert none is None and torch.equal(plain, o)
    for kw in (dict(need_dh0=False), dict(states=states), dict(states=states, need_dh0=False)):
        again = gdr.linear_bwd(*args, x["do"], x["dht"], lengths=x["lengths"], **kw)
        assert all(torch.equal(gr[n], again[n]) for n in ("dq", "dk", "dv"))
        assert again["dh0"] is None if "need_dh0" in kw else torch.equal(gr["dh0"], again["dh0"])
    return d, x, o, ht, gr


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("g", [0.0, -1e-4, -0.01, None])
def test_decays(g, dtype):
    """No decay, where the first segment's tokens weigh as much as the last's; slow ones; and a range over the heads."""
    check((1, 2100, 2, 4, 64, 64), dtype, g=g, seed=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hk,Hv,Dk,Dv", [(1, 1, 128, 128), (1, 3, 128, 32), (2, 4, 32, 128), (2, 2, 64, 128), (1, 2, 32, 32)])
def test_heads(Hk, Hv, Dk, Dv, dtype):
    check((1, 2305, Hk, Hv, Dk, Dv), dtype, g=-0.002, seed=Dk + Dv)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("g", [0.0, -1e-3])
def test_ragged_lengths(g, dtype):
    """Lengths at, before and after the segments' ends, in the first segment, and zero; NaN past them."""
    T = 2100
    shape = (6, T, 1, 2, 64, 32)
    block = {"bf16": 128, "fp32": 64}[dtype]
    nseg = segments(*shape, dtype)
    seg = -(-(-(-T // block)) // nseg) * block
    assert 0 < seg < T
    check(shape, dtype, g=g, seed=2, lengths=[T, 0, seg, seg + 1, seg - 1, 77])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_state_before_and_none_after(dtype):
    check((2, 2200, 1, 2, 64, 64), dtype, g=-1e-3, seed=3, initial=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeats_bitwise(dtype):
    """On another stream, and replayed from a graph."""
    d, x, o, ht, gr = check((1, 3333, 1, 2, 64, 64), dtype, g=-1e-3, seed=4)
    args = x["q"], x["k"], x["v"], x["g"], x["h0"]

    def both():
        o, ht = gdr.linear_fwd(*args)
        return [o, ht, *gdr.linear_bwd(*args, x["do"], x["dht"]).values()]

    want = [o, ht, *gr.values()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
