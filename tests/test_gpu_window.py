"""Window attention on the GPU against its formulas in 64 bits.

Bounds, on ||x - ref|| / ||ref|| for each head. A bf16 rounding is off by at most 2^-8 of the value. o: the weights p
and the result, 2 roundings. dv: p and the result; dk and dq: the gradient of the scores and the result, 2 roundings.
Where the row sums of do o come from the rounded o, that is off by 2^-8 of those products' sizes as well. fp32: sums of up to 256 products and as many weights, 256 x 2^-24.
dq and dk are sums of p (do.v - delta) where the two terms may cancel, wholly where a query sees one token. Both are
fp32 sums of up to 128 products, each off by at most 128 x 2^-24 of its products' sizes: that much of the same sums of
sizes remains, whatever the difference is.
lse: a score of order one is a sum of 128 products, each step off by 2^-24 of partial sums below 16: 128 x 2^-20."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from attention_ref import attention, make
from gated_delta_rule_31_gb300.autograd import window_attention
from linear_ref import rel, rel_heads
from util import cuda_device, to_dev

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {"bf16": dict.fromkeys(("o", "dq", "dk", "dv"), 2 * 2.0 ** -8),
       "fp32": dict.fromkeys(("o", "dq", "dk", "dv"), 256 * 2.0 ** -24)}
LSE = 128 * 2.0 ** -20


def close(got, ref, n, dtype):
    rest = ref[n + "_size"] * 128 * 2.0 ** -24 if n + "_size" in ref else torch.zeros_like(ref[n])
    rest = rest + ref.pop(n + "_o", 0.0)
    x = got.detach().double().cpu()
    assert x.shape == ref[n].shape and torch.isfinite(x).all()
    for h in range(x.shape[2]):
        off, size = float((x[:, :, h] - ref[n][:, :, h]).norm()), float(ref[n][:, :, h].norm())
        assert off <= TOL[dtype][n] * size + float(rest[:, :, h].norm()), (n, h, off, size)


def check(d, dtype, dev, **kw):
    ref = attention(**d, **kw)
    x = to_dev(d, dev)
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=dev)
    o, lse, rest = gdr.window_attention_fwd(x["q"], x["k"], x["v"], lengths=x["lengths"], save_lse=True, workspace=ws, **kw)
    assert gdr.workspace_status(ws) == 0
    ws = torch.full((1 << 25,), 255, dtype=torch.uint8, device=dev)
    gr = gdr.window_attention_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], lengths=x["lengths"], rest=rest, workspace=ws, **kw)
    assert gdr.workspace_status(ws) == 0
    got = dict(o=o, **gr)
    if dtype == "bf16":  # without the rest the rounding of o enters
        assert rest.dtype == torch.bfloat16 and (rest.double().abs() <= 2.0 ** -8 * o.double().abs() + 2.0 ** -133).all()
        for n, y in gdr.window_attention_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], lengths=x["lengths"], **kw).items():
            ref[n + "_o"] = ref.get(n + "_size", torch.zeros_like(ref[n])) * 2.0 ** -8
            close(y, ref, n, dtype)
    else:
        assert rest is None
    for n, y in got.items():
        assert y.dtype == d["q"].dtype
        close(y, ref, n, dtype)
    lse, want = lse.double().cpu(), ref["lse"]
    assert torch.equal(torch.isinf(lse), torch.isinf(want)) and not torch.isnan(lse).any()
    there = torch.isfinite(want)
    assert not there.any() or float((lse - want)[there].abs().max()) <= LSE
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 127, 128, 129, 255, 257, 384, 385, 600])
def test_lengths_around_the_blocks(T, dtype):
    check(make(2, T, 4, 2, 128, TYPES[dtype], seed=T), dtype, cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 0), (5, 300), (63, 4), (64, 4), (65, 0), (100, 130), (127, 1), (128, 0),
                                          (128, 128), (129, 2), (200, 64), (256, 5), (1000, 7), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_and_sinks(window, sinks, dtype):
    check(make(1, 500, 2, 1, 64, TYPES[dtype], seed=window % 1000 + sinks % 1000), dtype, cuda_device(), window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("Hk,G", [(1, 1), (3, 1), (1, 2), (2, 3), (1, 5), (2, 4), (1, 8), (1, 16)])
def test_heads(Hk, G, D, dtype):
    check(make(2, 300, Hk * G, Hk, D, TYPES[dtype], seed=G), dtype, cuda_device(), window=150, sinks=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 2)])
def test_ragged_lengths_and_what_lies_past_them(window, sinks, fill, dtype):
    n = [300, 0, 1, 128, 129, 64, 299, 200]
    d = make(len(n), 300, 4, 2, 64, TYPES[dtype], lengths=n, fill=fill, seed=3)
    got = check(d, dtype, cuda_device(), window=window, sinks=sinks)
    for b, m in enumerate(n):
        for x in got.values():
            assert not x[b, m:].any()


def test_lengths_are_clamped():
    d = make(3, 70, 2, 1, 64, torch.bfloat16, seed=5)
    d["lengths"] = torch.tensor([-4, 70, 1000], dtype=torch.int32)
    check(d, "bf16", cuda_device())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-30, 0.01, 1.0])
def test_scales(scale, dtype):
    check(make(1, 200, 2, 2, 32, TYPES[dtype], seed=8, std=0.3), dtype, cuda_device(), scale=scale, window=90, sinks=1)


def test_scores_that_grow_and_fall_along_the_keys():
    """Scores of +-100, so that the running maximum moves far at every block: weights of one token, or of none, of a block."""
    dev = cuda_device()
    for up in (1, -1):
        d = make(1, 640, 2, 2, 64, torch.bfloat16, seed=6)
        ramp = torch.linspace(-100, 100, 640)[:, None] * up
        d["q"][...] = 0
        d["q"][..., 0] = 8.0  # times 64^-1/2: one
        d["k"][..., 0] = ramp.to(torch.bfloat16)
        ref = attention(**d)
        x = to_dev(d, dev)
        o, lse, _ = gdr.window_attention_fwd(x["q"], x["k"], x["v"], save_lse=True)
        assert rel_heads(o, ref["o"], 2) <= TOL["bf16"]["o"]
        assert float((lse.double().cpu() - ref["lse"]).abs().max()) <= 2.0 ** -16 * 100
        gr = gdr.window_attention_bwd(x["q"], x["k"], x["v"], o, lse, x["do"])
        assert rel_heads(gr["dv"], ref["dv"], 2) <= TOL["bf16"]["dv"]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_tokens(dtype):
    dev = cuda_device()
    for B, T in ((2, 0), (0, 5)):
        d = to_dev(make(B, T, 2, 1, 64, TYPES[dtype]), dev)
        o, lse, _ = gdr.window_attention_fwd(d["q"], d["k"], d["v"], save_lse=True)
        assert o.shape == d["q"].shape and lse.shape == (B, 2, T)
        assert gdr.window_attention_bwd(d["q"], d["k"], d["v"], o, lse, d["do"])["dk"].shape == d["k"].shape


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeats_bitwise_on_another_stream_and_in_a_graph(dtype):
    dev = cuda_device()
    d = to_dev(make(2, 500, 6, 2, 128, TYPES[dtype], seed=4, lengths=[500, 333], fill=0.0), dev)
    kw = dict(window=200, sinks=2, lengths=d["lengths"])

    def both():
        o, lse, rest = gdr.window_attention_fwd(d["q"], d["k"], d["v"], save_lse=True, **kw)
        return (o, lse, *gdr.window_attention_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], rest=rest, **kw).values())

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    for _ in range(2):
        graph.replay()
        for a, b, c in zip(first, second, third):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd(dtype):
    dev = cuda_device()
    d = make(2, 150, 4, 2, 64, TYPES[dtype], seed=9)
    ref = attention(**d, window=40, sinks=2)
    x = to_dev(d, dev)
    q, k, v = (x[n].requires_grad_() for n in ("q", "k", "v"))
    o = window_attention(q, k, v, window=40, sinks=2)
    (o.transpose(1, 2) * x["do"].transpose(1, 2)).sum().backward()  # a gradient in another layout
    for n, t in (("dq", q), ("dk", k), ("dv", v)):
        close(t.grad, ref, n, dtype)
    with torch.no_grad():
        assert torch.equal(window_attention(q, k, v, window=40, sinks=2), o)


def test_gradients_against_differences():
    """fp32: <do, o(x + e) - o(x - e)> / 2 against <grad, e>. The central difference is off by the third derivative,
    about e^2 = 1e-4 of the slope, and by the rounding of o, 2^-22 / 1e-2."""
    dev = cuda_device()
    d = to_dev(make(1, 100, 2, 1, 32, torch.float32, seed=2), dev)
    kw = dict(window=33, sinks=3)
    o, lse, _ = gdr.window_attention_fwd(d["q"], d["k"], d["v"], save_lse=True, **kw)
    gr = gdr.window_attention_bwd(d["q"], d["k"], d["v"], o, lse, d["do"], **kw)
    gen = torch.Generator(device=dev).manual_seed(1)
    for n in ("q", "k", "v"):
        e = 1e-2 * torch.randn(d[n].shape, generator=gen, device=dev)
        plus, minus = (gdr.window_attention_fwd(*(d[m] + (s * e if m == n else 0) for m in ("q", "k", "v")), **kw)[0] for s in (1, -1))
        slope = float((d["do"].double() * (plus.double() - minus.double())).sum()) / 2
        want = float((gr["d" + n].double() * e.double()).sum())
        assert abs(slope - want) <= 2e-3 * float(gr["d" + n].norm() * e.norm()), n


def test_a_long_sequence_in_parts():
    """Rows of a long sequence whose window is whole do not depend on where the sequence begins."""
    dev = cuda_device()
    gen = torch.Generator(device=dev).manual_seed(3)
    q, k, v = (torch.randn(1, 9000, h, 128, generator=gen, device=dev).bfloat16() for h in (4, 1, 1))
    o = gdr.window_attention_fwd(q, k, v, window=700)[0]
    part =  gdr.window_attention_fwd(*(x[:, 5120:7000].contiguous() for x in (q, k, v)), window=700)[0]
    assert rel(part[0, 700:], o[0, 5820:7000]) <= 2 * TOL["bf16"]["o"]


def test_refusals():
    dev = cuda_device()
    d = to_dev(make(2, 40, 4, 2, 64, torch.bfloat16), dev)
    q, k, v = d["q"], d["k"], d["v"]
    f = gdr.window_attention_fwd
    for bad in (lambda: f(q.cpu(), k, v), lambda: f(q, k[:, :30], v), lambda: f(q, k.float(), v), lambda: f(q.half(), k.half(), v.half()),
                lambda: f(q[:, :, ::2], k, v), lambda: f(q, k, v, window=-1), lambda: f(q, k, v, sinks=1.5),
                lambda: f(q, k, v, window=2 ** 31), lambda: f(q, k, v, lengths=torch.ones(3, dtype=torch.int32, device=dev)),
                lambda: f(q, k, v, lengths=torch.ones(2, device=dev)), lambda: f(q, k, v, out=torch.empty_like(k)),
                lambda: f(q, k, v, workspace=torch.empty(8, dtype=torch.uint8, device=dev)), lambda: f(q[0], k, v)):
        with pytest.raises(ValueError):
            bad()
    for kw, code in ((dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=-1.0), 1)):
        with pytest.raises(gdr.GdrError) as e:
            f(q, k, v, **kw)
        assert e.value.code == code
    with pytest.raises(gdr.GdrError) as e:  # three query heads for two key heads
        f(q[:, :, :3].contiguous(), k, v)
    assert e.value.code == 1
    w = torch.zeros(1, 8, 2, 48, device=dev)
    with pytest.raises(gdr.GdrError) as e:
        f(w, w, w)
    assert e.value.code == 2
    o, lse, _ = f(q, k, v, save_lse=True)
    for bad in (lambda: gdr.window_attention_bwd(q, k, v, o, lse[:, :2], d["do"]), lambda: gdr.window_attention_bwd(q, k, v, o, lse, d["do"].float())):
        with pytest.raises(ValueError):
            bad()


def test_a_saved_output_that_a_call_overwrites_is_noticed():
    dev = cuda_device()
    d = to_dev(make(1, 30, 2, 1, 64, torch.float32), dev)
    q = d["q"].requires_grad_()
    o = window_attention(q, d["k"], d["v"])
    y = (o * o).sum()
    gdr.window_attention_fwd(d["do"], d["k"], d["v"], out=o.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_long_sums_of_gradients_keep_their_precision():
    """fp32: a key that thousands of queries see. Its gradients, sums of as many terms of either sign, are off by at most
    256 x 2^-24 of what a sum of terms of one sign would be, as shorter ones are."""
    dev = cuda_device()
    d = make(1, 6000, 2, 1, 32, torch.float32, seed=1)
    ref = attention(**d, window=64, sinks=3)
    x = to_dev(d, dev)
    o, lse, _ = gdr.window_attention_fwd(x["q"], x["k"], x["v"], window=64, sinks=3, save_lse=True)
    gr = gdr.window_attention_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], window=64, sinks=3)
    for n in ("dq", "dk", "dv"):
        assert rel_heads(gr[n], ref[n], 2) <= TOL["fp32"][n]
    # the first tokens alone: 12000 terms each
    assert rel(gr["dv"][0, :3], ref["dv"][0, :3]) <= 32 * 2.0 ** -24 and rel(gr["dk"][0, :3], ref["dk"][0, :3]) <= 32 * 2.0 ** -24


def test_few_tokens_round_once():
    """bf16, up to 64 tokens: the weights enter to 2^-17, so each result is off by its own rounding, 2^-8 at most, alone."""
    dev = cuda_device()
    for T in (2, 3, 20, 64):
        d = make(4, T, 4, 2, 64, torch.bfloat16, seed=T)
        ref = attention(**d)
        x = to_dev(d, dev)
        o, lse, rest = gdr.window_attention_fwd(x["q"], x["k"], x["v"], save_lse=True)
        gr = gdr.window_attention_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], rest=rest)
        for n, y in dict(o=o, **gr).items():
            off = float((y.double().cpu() - ref[n]).norm() / ref[n].norm())
            # a rounding's error is spread evenly over its step: 1 / sqrt 3 of the most, with room for few values
            assert off <= 0.75 * 2.0 ** -8, (T, n, off)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_tensors_on_the_16_byte_grid_only(dtype):
    """Views that begin 16 bytes into their storage, and ones off the grid, which are refused."""
    dev = cuda_device()
    d = make(2, 130, 4, 2, 64, TYPES[dtype], seed=12)
    ref = attention(**d, window=50, sinks=1)
    step = 16 // TYPES[dtype].itemsize

    def view(x, by):
        flat = torch.empty(x.numel() + 64, dtype=x.dtype, device=dev)
        y = flat[by:by + x.numel()].view(x.shape)
        y.copy_(x)
        return y

    q, k, v, do = (view(d[n], step) for n in ("q", "k", "v", "do"))
    out = view(torch.zeros_like(d["q"]), 3 * step)
    o, lse, rest = gdr.window_attention_fwd(q, k, v, window=50, sinks=1, save_lse=True, out=out)
    assert o is out
    gr = gdr.window_attention_bwd(q, k, v, o, lse, do, window=50, sinks=1, rest=rest)
    for n, y in dict(o=o, **gr).items():
        close(y, ref, n, dtype)
    with pytest.raises(gdr.GdrError) as e:
        gdr.window_attention_fwd(view(d["q"], 1), k, v)
    assert e.value.code == 1


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_short_sequences(dtype):
    n = [(i * 7) % 6 for i in range(700)]
    check(make(700, 5, 3, 1, 32, TYPES[dtype], lengths=n, seed=13), dtype, cuda_device(), window=3, sinks=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_workspaces_of_earlier_calls_and_two_graphs(dtype):
    """Whatever a workspace holds; and two captured calls that share one, replayed one after the other."""
    dev = cuda_device()
    xs = [to_dev(make(1, 400, 4, 2, 64, TYPES[dtype], seed=s), dev) for s in (14, 15)]
    kw = dict(window=100, sinks=5)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device=dev)

    def both(x, w=None):
        o, lse, rest = gdr.window_attention_fwd(x["q"], x["k"], x["v"], save_lse=True, workspace=w, **kw)
        return (o, *gdr.window_attention_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], rest=rest, workspace=w, **kw).values())

    want = [both(x) for x in xs]
    graphs, got = [torch.cuda.CUDAGraph() for _ in xs], []
    for g, x in zip(graphs, xs):
        with torch.cuda.graph(g):
            got.append(both(x, ws))
    for order in ((0, 1), (1, 0)):
        for i in order:
            graphs[i].replay()
        for a, b in zip(got, want):
            assert all(torch.equal(u, w) for u, w in zip(a, b))


def test_lengths_that_change_between_replays():
    dev = cuda_device()
    d = to_dev(make(2, 300, 2, 1, 64, torch.bfloat16, seed=16), dev)
    n = torch.tensor([300, 10], dtype=torch.int32, device=dev)
    graph = torch.cuda.CUDAGraph()
    f = lambda: gdr.window_attention_fwd(d["q"], d["k"], d["v"], lengths=n, window=64)[0]  # noqa: E731
    f()
    with torch.cuda.graph(graph):
        o = f()
    for lengths in ([300, 10], [0, 300], [129, 1]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        graph.replay()
        assert torch.equal(o, f())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_values_that_are_none_are_not_hidden(dtype):
    """NaN in a query reaches its output, and that one alone; in a key every later query of its heads."""
    dev = cuda_device()
    d = make(1, 300, 4, 2, 64, TYPES[dtype], seed=17)
    ref = attention(**d)
    d["q"][0, 140, 3, 5] = float("nan")
    o = gdr.window_attention_fwd(*(d[n].to(dev) for n in "qkv"))[0]
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[0, 140, 3] = True
    assert torch.equal(o.isnan(), bad)
    close(o[:, :, :3], {"o": ref["o"][:, :, :3]}, "o", dtype)
    d["k"][0, 200, 0] = float("nan")
    o, lse, _ = gdr.window_attention_fwd(*(d[n].to(dev) for n in "qkv"), save_lse=True)
    assert o[0, 200:, :2].isnan().all() and lse[0, :2, 200:].isnan().all()
    close(o[:, :, 2:3], {"o": ref["o"][:, :, 2:3]}, "o", dtype)
