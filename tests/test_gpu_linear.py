"""Linear attention with a constant decay per head on the GPU against the recurrence in 64 bits.

Bounds, on ||x - ref|| / ||ref|| for each head. bf16 results: the intra-chunk weights, the state and
the result are each rounded once to bf16 (relative error up to 2^-9), so 3 x 2^-9. fp32 results:
sums of up to 256 terms in fp32, 256 x 2^-24; a state also carries the decays' own rounding, |g| T
2^-24 times a weight exp(-|g| T) whose product is below 2^-24."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from linear_ref import linear, make, rel, rel_heads
from util import cuda_device, to_dev

pytestmark = pytest.mark.gpu

BF16 = 3 * 2.0 ** -9
FP32 = 256 * 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {"bf16": BF16, "fp32": FP32}


def check(d, dtype, dev, scale=None):
    ref = linear(**d, scale=scale)
    x = to_dev(d, dev)
    o, ht = gdr.linear_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], scale=scale, lengths=x["lengths"])
    gr = gdr.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["h0"], x["do"], x["dht"], scale=scale, lengths=x["lengths"])
    assert o.dtype == d["v"].dtype and ht.dtype == torch.float32
    assert rel_heads(o, ref["o"], 2) <= TOL[dtype]
    assert rel_heads(ht, ref["ht"], 1) <= FP32
    for n in ("dq", "dk", "dv"):
        assert gr[n].dtype == d["q"].dtype
        assert rel_heads(gr[n], ref[n], 2) <= TOL[dtype], n
    assert rel_heads(gr["dh0"], ref["dh0"], 1) <= FP32
    return o, ht, gr


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300, 769])
def test_lengths_around_the_blocks(T, dtype):
    check(make(2, T, 2, 2, 128, 128, TYPES[dtype], seed=T), dtype, cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Dk", [32, 64, 128])
@pytest.mark.parametrize("Dv", [32, 64, 128])
def test_head_sizes(Dk, Dv, dtype):
    check(make(1, 200, 2, 4, Dk, Dv, TYPES[dtype], seed=Dk + Dv), dtype, cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("Hk,G", [(1, 1), (1, 2), (2, 3), (1, 5), (3, 4), (1, 8), (2, 16)])
def test_shared_heads(Hk, G, dtype):
    check(make(1, 150, Hk, Hk * G, 64, 128, TYPES[dtype], seed=G), dtype, cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
def test_ragged_lengths_and_what_lies_past_them(fill, dtype):
    n = [300, 0, 1, 128, 129, 64, 299]
    d = make(len(n), 300, 2, 4, 128, 64, TYPES[dtype], lengths=n, fill=fill, seed=3)
    o, _, gr = check(d, dtype, cuda_device())
    for b, m in enumerate(n):
        for x in (o, gr["dq"], gr["dk"], gr["dv"]):
            assert not x[b, m:].any()


def test_lengths_are_clamped():
    dev = cuda_device()
    d = make(3, 70, 1, 2, 64, 64, torch.bfloat16, seed=5)
    d["lengths"] = torch.tensor([-4, 70, 1000], dtype=torch.int32)
    check(d, "bf16", dev)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("g", [0.0, -1e-4, -0.7, -30.0, -2000.0, float("-inf")])
def test_decays(g, dtype):
    """From none to a state that each token replaces; a zero state times a dead decay stays zero."""
    check(make(1, 333, 1, 2, 64, 64, TYPES[dtype], g=g, seed=7), dtype, cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_initial_state_and_a_scale(dtype):
    check(make(2, 140, 2, 2, 64, 64, TYPES[dtype], initial=False, seed=8), dtype, cuda_device(), scale=-0.37)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_heads_need_no_segments(dtype):
    """Enough (batch, head) pairs to fill the GPU: one segment per sequence, every state carried through it."""
    check(make(40, 260, 4, 8, 32, 64, TYPES[dtype], seed=9, lengths=[260 - 6 * i for i in range(40)]), dtype,
          cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_tokens(dtype):
    dev = cuda_device()
    d = to_dev(make(2, 0, 1, 2, 64, 32, TYPES[dtype], seed=1), dev)
    o, ht = gdr.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"])
    assert o.shape == (2, 0, 2, 32) and torch.equal(ht, d["h0"])
    gr = gdr.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dht"])
    assert torch.equal(gr["dh0"], d["dht"]) and gr["dq"].numel() == 0
    assert not gdr.linear_fwd(d["q"], d["k"], d["v"], d["g"])[1].any()
    e = to_dev(make(0, 5, 1, 2, 64, 32, TYPES[dtype], seed=1), dev)
    assert gdr.linear_fwd(e["q"], e["k"], e["v"], e["g"], e["h0"])[0].shape == (0, 5, 2, 32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hk,Hv,Dk,Dv", [(1, 16, 32, 128, 128), (3, 1, 5, 64, 32), (64, 4, 8, 32, 128), (1, 1, 1, 128, 64),
                                           (200, 2, 2, 128, 128)])
def test_step(B, Hk, Hv, Dk, Dv, dtype):
    dev = cuda_device()
    d = make(B, 3, Hk, Hv, Dk, Dv, TYPES[dtype], seed=B)
    ref = linear(**d, grads=False)
    x = to_dev(d, dev)
    state = x["h0"].clone()
    os = [gdr.linear_decode_step(x["q"][:, t].contiguous(), x["k"][:, t].contiguous(), x["v"][:, t].contiguous(),
                                 x["g"], state) for t in range(3)]
    assert rel_heads(torch.stack(os, 1), ref["o"], 2) <= TOL[dtype]
    assert rel_heads(state, ref["ht"], 1) <= FP32


def test_prompt_then_steps_continue_one_sequence():
    dev = cuda_device()
    d = make(2, 140, 2, 4, 128, 128, torch.bfloat16, seed=2, lengths=[130, 77], fill=0.0)
    more = make(2, 4, 2, 4, 128, 128, torch.bfloat16, seed=3)
    x, y = to_dev(d, dev), to_dev(more, dev)
    _, state = gdr.linear_fwd(x["q"], x["k"], x["v"], x["g"], x["h0"], lengths=x["lengths"])
    for t in range(4):
        o = gdr.linear_decode_step(y["q"][:, t].contiguous(), y["k"][:, t].contiguous(), y["v"][:, t].contiguous(),
                                   x["g"], state)
    for b, n in enumerate([130, 77]):
        one = {m: torch.cat([d[m][b:b + 1, :n], more[m][b:b + 1]], 1) for m in ("q", "k", "v")}
        ref = linear(**one, g=d["g"], h0=d["h0"][b:b + 1], grads=False)
        assert rel(o[b], ref["o"][0, -1]) <= BF16
        assert rel(state[b], ref["ht"][0]) <= FP32


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeats_bitwise_on_another_stream(dtype):
    dev = cuda_device()
    d = to_dev(make(2, 400, 2, 6, 128, 64, TYPES[dtype], seed=4), dev)

    def both():
        o, ht = gdr.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"])
        return [o, ht, *gdr.linear_bwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["do"], d["dht"]).values()]

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = both()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_kept_states_give_the_same_gradients(dtype):
    dev = cuda_device()
    for n in (None, [500, 0, 129]):
        d = to_dev(make(3, 500, 2, 4, 64, 128, TYPES[dtype], seed=13, lengths=n), dev)
        args = d["q"], d["k"], d["v"], d["g"], d["h0"]
        o, ht = gdr.linear_fwd(*args, lengths=d["lengths"])
        o2, ht2, states = gdr.linear_fwd(*args, lengths=d["lengths"], save_states=True)
        assert torch.equal(o, o2) and torch.equal(ht, ht2)
        want = gdr.linear_bwd(*args, d["do"], d["dht"], lengths=d["lengths"])
        got = gdr.linear_bwd(*args, d["do"], d["dht"], lengths=d["lengths"], states=states)
        assert all(torch.equal(want[x], got[x]) for x in want)


def test_runs_in_a_captured_graph():
    dev = cuda_device()
    d = to_dev(make(1, 300, 2, 4, 128, 128, torch.bfloat16, seed=6), dev)
    want = gdr.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdr.linear_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"])
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_gradients_against_differences():
    """<do, o> + <dht, ht> changes along a random direction by the gradients' product with it: central
    differences of the 64-bit form, whose own error is about eps^2 of the change."""
    dev = cuda_device()
    d = make(1, 70, 1, 2, 32, 32, torch.float32, seed=11)
    x = to_dev(d, dev)
    gr = gdr.linear_bwd(x["q"], x["k"], x["v"], x["g"], x["h0"], x["do"], x["dht"])

    def loss(**kw):
        r = linear(**{**d, **kw}, grads=False)
        return float((r["o"] * d["do"].double()).sum() + (r["ht"] * d["dht"].double()).sum())

    for name, of in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("h0", "dh0")):
        u = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
        eps = 1e-4
        num = (loss(**{name: d[name].double() + eps * u}) - loss(**{name: d[name].double() - eps * u})) / (2 * eps)
        ana = float((gr[of].cpu().double() * u).sum())
        # the loss is linear in each argument: what is left is the gradient's fp32 error
        assert abs(ana - num) <= FP32 * float(gr[of].cpu().double().norm() * u.norm()) + 1e-6 * abs(num), name


def test_autograd():
    from gated_delta_rule_31_gb300.autograd import linear_attention

    dev = cuda_device()
    d = make(2, 90, 2, 4, 64, 64, torch.bfloat16, seed=12, lengths=[90, 33])
    ref = linear(**d)
    x = to_dev(d, dev)
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = linear_attention(*leaves[:3], x["g"], leaves[3], lengths=x["lengths"])
    grads = torch.autograd.grad((o, ht), leaves, (x["do"], x["dht"]))
    for g, leaf, n in zip(grads, leaves, ("dq", "dk", "dv", "dh0")):
        assert g.dtype == leaf.dtype
        assert rel(g, ref[n]) <= (FP32 if n == "dh0" else BF16), n
    (only_o,) = torch.autograd.grad(linear_attention(*leaves[:3], x["g"], leaves[3], lengths=x["lengths"])[0], leaves[2],
                                    x["do"])
    assert rel(only_o, linear(**{**d, "dht": None})["dv"]) <= BF16
    with pytest.raises(ValueError):
        linear_attention(*leaves[:3], x["g"].clone().requires_grad_())


def test_more_than_two_to_the_31_values():
    """Offsets past 32 bits: the last tokens of a sequence whose decay forgets all but the last hundred."""
    dev = cuda_device()
    T, H, D = 262400, 64, 128
    assert T * H * D > 2 ** 31
    gen = torch.Generator(device=dev).manual_seed(0)
    k, v, q = (torch.empty(1, T, h, D, dtype=torch.bfloat16, device=dev).normal_(generator=gen) for h in (1, H, 1))
    g = torch.full((H,), -1.0, device=dev)
    o, ht = gdr.linear_fwd(q, k, v, g)
    gr = gdr.linear_bwd(q, k, v, g, None, v)
    last = {n: x[:, -200:].cpu() for n, x in (("q", q), ("k", k), ("v", v), ("do", v))}
    ref = linear(**last, g=g.cpu())
    assert rel(o[:, -100:].cpu(), ref["o"][:, -100:]) <= BF16
    assert rel(ht, ref["ht"]) <= FP32
    for n in ("dq", "dk", "dv"):
        assert rel(gr[n][:, -100:].cpu(), ref[n][:, -100:]) <= BF16, n


@pytest.mark.parametrize("initial", [True, False])
def test_autograd_with_an_unused_result(initial):
    """A loss of ht alone, and one of o alone, without and with an initial state's gradient."""
    from gated_delta_rule_31_gb300.autograd import linear_attention

    d = make(1, 150, 1, 2, 64, 32, torch.bfloat16, seed=15, initial=initial)
    dht = torch.randn(1, 2, 32, 64, generator=torch.Generator().manual_seed(16))
    x = to_dev(d, cuda_device())
    names = ("q", "k", "v", "h0") if initial else ("q", "k", "v")
    leaves = [x[n].requires_grad_() for n in names]
    o, ht = linear_attention(*leaves[:3], x["g"], leaves[3] if initial else None)
    of_ht = torch.autograd.grad(ht, leaves, dht.to(ht.device), retain_graph=True)
    ref = linear(**{**d, "do": torch.zeros_like(d["do"]), "dht": dht})
    for g, n in zip(of_ht, names):
        assert rel(g, ref["d" + n]) <= (FP32 if n == "h0" else BF16), n
    of_o = torch.autograd.grad(o, leaves, x["do"])
    ref = linear(**{**d, "dht": None})
    for g, n in zip(of_o, names):
        assert rel(g, ref["d" + n]) <= (FP32 if n == "h0" else BF16), n
