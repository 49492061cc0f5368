"""The softmax attention layer's operators together, as a model uses them: a prompt through window attention, its keys and
values appended to a paged cache, then tokens one by one; and calls in a row on one stream that feed one another."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from attention_ref import attention, turn
from gated_delta_rule_31_gb300.autograd import rotary, window_attention
from linear_ref import rel, rel_heads
from util import cuda_device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
# As window attention's own bounds (2 roundings of 2^-8, sums of 256 terms of 2^-24), with one rounding more each of the
# rotated queries and keys: scores of order one move by 2 x 2^-8 in all, and the weights with them.
TOL = {"bf16": 4 * 2.0 ** -8, "fp32": 256 * 2.0 ** -24}


def freqs(pairs, dev):
    return (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(dev)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks,sections", [(0, 0, None), (70, 3, None), (40, 0, (6, 6, 4))])
def test_prompts_then_tokens(window, sinks, sections, dtype):
    dev = cuda_device()
    B, T, more, Hq, Hk, D, page, R = 3, 150, 6, 6, 2, 64, 16, 16
    n = [150, 0, 77]
    gen = torch.Generator(device=dev).manual_seed(window)
    q, k, v = (torch.randn(B, T + more, h, D, generator=gen, device=dev).to(TYPES[dtype]) for h in (Hq, Hk, Hk))
    axes = len(sections) if sections else 1
    p = torch.stack([torch.arange(T + more, device=dev) + 1000, torch.arange(T + more, device=dev) // 9, torch.arange(T + more, device=dev) % 9][:axes], -1)
    p = p.to(torch.int32).expand(B, -1, -1).contiguous()
    f = freqs(R, dev)
    counts = torch.tensor(n, dtype=torch.int32, device=dev)
    per = -(-(T + more) // page)
    table = torch.randperm(B * per, generator=gen, device=dev).view(B, per).to(torch.int32)
    kc, vc = (torch.full((B * per, page, Hk, D), float("nan"), device=dev).to(TYPES[dtype]) for _ in range(2))
    kw = dict(inv_freq=f, sections=sections)

    def cut(x, a, b):
        return x[:, a:b].contiguous()

    rq, rk = (rotary(cut(x, 0, T), cut(p, 0, T), f, sections=sections) for x in (q, k))
    o = window_attention(rq, rk, cut(v, 0, T), window=window, sinks=sinks, lengths=counts)
    length = torch.zeros(B, dtype=torch.int32, device=dev)
    aq = gdr.kv_append(cut(k, 0, T), cut(v, 0, T), kc, vc, table, length, positions=cut(p, 0, T), counts=counts, q=cut(q, 0, T), **kw)
    for b in range(B):
        assert torch.equal(aq[b, :n[b]], rq[b, :n[b]]) and not aq[b, n[b]:].any()
    length += counts
    outs = []
    at = torch.arange(B, device=dev)
    for i in range(more):
        j = length.long()  # the next token of each sequence is the one that follows in its row
        tq, tk, tv = (x[at, j].contiguous() for x in (q, k, v))
        y = gdr.kv_append(tk, tv, kc, vc, table, length, positions=p[at, j].contiguous(), q=tq, **kw)
        length += 1
        outs.append(gdr.paged_decode_step(y, kc, vc, table, length, window=window, sinks=sinks))
    for b in range(B):
        m = n[b] + more
        one = [turn(x[b:b + 1, :m], p[b:b + 1, :m].cpu(), f.cpu(), sections) for x in (q, k)] + [v[b:b + 1, :m].double().cpu()]
        ref = attention(*one, window=window, sinks=sinks)["o"][0]
        assert not o[b, n[b]:].any()
        if n[b]:
            assert rel_heads(o[b, :n[b]], ref[:n[b]], 1) <= TOL[dtype]
        for i in range(more):
            assert rel(outs[i][b], ref[n[b] + i]) <= TOL[dtype]


def steps(x, wait):
    """Each call takes results of the ones before it: rotated queries, the cache, states, outputs."""
    out = []
    q, state = x["q"], x["state"].clone()
    kc, vc, n = x["kc"].clone(), x["vc"].clone(), x["n"].clone()
    for _ in range(6):
        y = wait(gdr.kv_append(q, x["v"], kc, vc, x["table"], n, inv_freq=x["f"], q=q))
        n = n + 1
        a = wait(gdr.paged_decode_step(y, kc, vc, x["table"], n, window=x["window"], sinks=2))
        b = wait(gdr.linear_decode_step(a, y, a, x["g"], state))
        q = wait(gdr.rotary(b, n, x["f"]))
        out += [y, a, b, q]
    return out + [kc, vc, state]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,window", [(2, 0), (30, 40)])
def test_calls_that_feed_one_another(B, window, dtype):
    """As they start while the call before them ends, nothing may be read before that one is complete."""
    dev = cuda_device()
    H, D, page = 8, 128, 16
    gen = torch.Generator(device=dev).manual_seed(B)
    r = lambda *s: torch.randn(*s, generator=gen, device=dev).to(TYPES[dtype])  # noqa: E731
    per = 6
    x = dict(q=r(B, H, D), v=r(B, H, D), kc=r(B * per, page, H, D), vc=r(B * per, page, H, D), f=freqs(32, dev), window=window,
             table=torch.randperm(B * per, generator=gen, device=dev).view(B, per).int(),
             n=torch.randint(1, 80, (B,), generator=gen, device=dev).int(), g=-torch.rand(H, generator=gen, device=dev),
             state=torch.randn(B, H, D, D, generator=gen, device=dev))

    def synced(t):
        torch.cuda.synchronize()
        return t

    want = steps(x, synced)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(x, lambda t: t), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(x, lambda t: t)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_training_step_of_a_layer_in_a_graph():
    """Rotation and attention with their gradients, captured."""
    dev = cuda_device()
    gen = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn(2, 100, 256, generator=gen, device=dev).bfloat16()
    w = [(torch.randn(256, h * 64, generator=gen, device=dev) / 16).bfloat16().requires_grad_() for h in (4, 2, 2)]
    p, f = torch.arange(100, dtype=torch.int32, device=dev).expand(2, -1).contiguous(), freqs(32, dev)

    def step():
        q, k, v = ((x @ m).view(2, 100, -1, 64) for m in w)
        o = window_attention(rotary(q, p, f), rotary(k, p, f), v, window=30, sinks=1)
        return torch.autograd.grad(o.float().square().sum(), w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            want = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
