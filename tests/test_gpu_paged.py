"""The decode step over a paged cache on the GPU against its formula in 64 bits.

Bounds, on ||x - ref|| / ||ref|| for each head. bf16: the weights and the result are rounded once each, 2 x 2^-8; fp32:
sums of up to 256 products and weights in a row (longer ones are cut), 256 x 2^-24."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from attention_ref import decode, make_cache, rows
from linear_ref import rel_heads
from util import cuda_device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {"bf16": 2 * 2.0 ** -8, "fp32": 256 * 2.0 ** -24}


def make(B, lengths, Hq, Hk, D, page, dtype, seed=0, fill=float("nan"), room=0):
    """q, caches, table, lengths; rows that hold no token hold `fill`."""
    gen = torch.Generator().manual_seed(seed)
    table, kc, vc = make_cache(B, max(lengths) + room, page, Hk, D, dtype, seed=seed, fill=fill)
    for b, n in enumerate(lengths):
        pg, r = rows(table, b, n, page)
        kc[pg, r], vc[pg, r] = (torch.randn(n, Hk, D, generator=gen).to(dtype) for _ in range(2))
    return torch.randn(B, Hq, D, generator=gen).to(dtype), kc, vc, table, torch.tensor(lengths, dtype=torch.int32)


def check(x, dtype, **kw):
    dev = cuda_device()
    ref = decode(*x, **kw)
    o = gdr.paged_decode_step(*(t.to(dev) for t in x), **kw)
    assert o.dtype == x[0].dtype and o.shape == x[0].shape
    assert rel_heads(o, ref, 1) <= TOL[dtype]
    for b in range(len(ref)):
        if not ref[b].any():
            assert not o[b].any()
    return o


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 129, 255, 1000, 5000])
def test_lengths(n, dtype):
    check(make(1, [n], 8, 2, 128, 16, TYPES[dtype], seed=n), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100, 256])
def test_pages(page, dtype):
    check(make(4, [300, 0, 1, 123], 4, 2, 64, page, TYPES[dtype], seed=page, room=70), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("Hk,G", [(1, 1), (5, 1), (2, 2), (1, 3), (2, 7), (1, 8), (1, 9), (2, 16), (1, 17), (1, 40)])
def test_heads(Hk, G, D, dtype):
    check(make(2, [200, 77], Hk * G, Hk, D, 16, TYPES[dtype], seed=G), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (10, 4), (16, 16), (63, 0), (64, 4), (65, 1), (100, 130), (1000, 3), (2 ** 31 - 1, 2 ** 31 - 1), (0, 5)])
def test_windows_and_sinks(window, sinks, dtype):
    check(make(5, [400, 64, 65, 3, 110], 4, 1, 64, 16, TYPES[dtype], seed=sinks % 100), dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_sequences(dtype):
    """More than the threads that sum up the lengths, most of them short, one long."""
    n = [(7 * i) % 50 for i in range(300)]
    n[150] = 3000
    check(make(300, n, 4, 2, 32, 8, TYPES[dtype], seed=1), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_enough_sequences_for_every_run(dtype):
    check(make(70, [130 + (37 * i) % 90 for i in range(70)], 16, 8, 64, 16, TYPES[dtype], seed=2), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 1), (63, 4), (200, 0), (130, 130)])
@pytest.mark.parametrize("D,Hq,Hk", [(32, 6, 2), (64, 16, 8), (128, 8, 4), (128, 18, 1)])
def test_more_walks_than_clusters_are_made_for(D, Hq, Hk, window, sinks, dtype):
    """Tiles of all sequences dealt out in runs: walks whole, cut once and cut into many parts, empty ones between them."""
    n = [(97 * i * i) % 400 for i in range(60)]
    n[7], n[8], n[59] = 1900, 0, 700
    x = make(60, n, Hq, Hk, D, 16, TYPES[dtype], seed=D + window)
    x[3][11, :2] = -1  # pages given back
    x[3][12] = 10 ** 6
    check(x, dtype, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Hq,Hk", [(1, 4, 1), (1, 8, 8), (3, 12, 12), (2, 72, 2)])
def test_long_sequences(B, Hq, Hk, dtype):
    check(make(B, [20000 + 777 * b for b in range(B)], Hq, Hk, 128, 64, TYPES[dtype], seed=B), dtype)


def test_a_table_with_more_room_than_tokens():
    """Short sequences in a table for long ones, over the sizes where clusters give way to runs."""
    for room in (100, 30000, 40000, 300000):
        q, kc, vc, table, n = make(2, [333, 65], 8, 2, 64, 16, torch.bfloat16, seed=room % 7)
        wide = torch.full((2, -(-room // 16)), 2 ** 31 - 1, dtype=torch.int32)
        wide[:, :table.shape[1]] = table[:, :wide.shape[1]]
        n = n.clamp(max=wide.shape[1] * 16)
        check((q, kc, vc, wide, n), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_pages_that_are_none(dtype):
    """Tokens on pages outside the cache are not seen: freed pages before the window, and others."""
    x = list(make(3, [200, 150, 90], 4, 2, 64, 16, TYPES[dtype], seed=4))
    t = x[3]
    t[0, :3] = -1
    t[1, 4] = 2 ** 30
    t[2, :] = -2 ** 31
    check(x, dtype)
    check(x, dtype, window=100, sinks=20)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_no_sequence_sees_anything(dtype):
    check(make(3, [0, 0, 0], 4, 2, 64, 16, TYPES[dtype]), dtype)
    dev = cuda_device()
    q = torch.randn(2, 4, 64, device=dev).to(TYPES[dtype])
    cache = torch.empty(0, 16, 2, 64, device=dev, dtype=TYPES[dtype])
    n = torch.tensor([5, 9], dtype=torch.int32, device=dev)
    for table in (torch.zeros(2, 3, dtype=torch.int32, device=dev), torch.zeros(2, 0, dtype=torch.int32, device=dev)):
        assert not gdr.paged_decode_step(q, cache, cache, table, n).any()
    e = torch.empty(0, 4, 64, device=dev, dtype=TYPES[dtype])
    assert gdr.paged_decode_step(e, cache, cache, torch.zeros(0, 3, dtype=torch.int32, device=dev), n[:0]).shape == (0, 4, 64)


def test_lengths_are_clamped():
    x = list(make(3, [48, 48, 48], 2, 1, 64, 16, torch.bfloat16, seed=5))
    x[4] = torch.tensor([-3, 10 ** 9, 2 ** 31 - 1], dtype=torch.int32)
    check(x, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_scores_that_grow_and_fall_along_the_keys(dtype):
    for up in (1, -1):
        q, kc, vc, table, n = make(1, [4000], 4, 1, 64, 16, TYPES[dtype], seed=6)
        q.zero_()
        q[..., 0] = 8.0
        pg, r = rows(table, 0, 4000, 16)
        kc[pg, r, :, 0] = (torch.linspace(-100, 100, 4000)[:, None] * up).to(TYPES[dtype])
        check((q, kc, vc, table, n), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_entries_that_share_pages_and_a_scale(dtype):
    q, kc, vc, table, n = make(4, [100] * 4, 4, 2, 64, 16, TYPES[dtype], seed=7)
    table[1:, :4] = table[0, :4]
    check((q, kc, vc, table, n), dtype, scale=0.3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_repeats_bitwise_on_another_stream_and_in_a_graph(dtype):
    dev = cuda_device()
    x = [t.to(dev) for t in make(3, [900, 30, 1], 8, 2, 128, 16, TYPES[dtype], seed=8, room=50)]
    first = gdr.paged_decode_step(*x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = gdr.paged_decode_step(*x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = gdr.paged_decode_step(*x)
    graph.replay()
    assert torch.equal(first, second) and torch.equal(first, third)
    x[4].add_(-1)  # the lengths are read on the device
    graph.replay()
    assert torch.equal(third, gdr.paged_decode_step(*x)) and not torch.equal(first, third)


@pytest.mark.parametrize("B", [1, 40])
def test_two_calls_at_once(B):
    """On two streams, each with its own workspace; and two graphs replayed at once."""
    dev = cuda_device()
    xs = [[t.to(dev) for t in make(B, [600 + 5 * b for b in range(B)], 8, 4, 128, 16, torch.bfloat16, seed=s)] for s in (1, 2)]
    want = [gdr.paged_decode_step(*x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    graphs, got = [torch.cuda.CUDAGraph() for _ in xs], [None, None]
    for i, x in enumerate(xs):
        with torch.cuda.graph(graphs[i]):
            for _ in range(5):
                got[i] = gdr.paged_decode_step(*x)
    torch.cuda.synchronize()
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(gdr.paged_decode_step(*xs[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[i]) for i in range(2) for a in outs[i])


def test_offsets_past_32_bits():
    """A cache of 2^31 elements and more: rows at its end."""
    dev = cuda_device()
    D, Hk, page = 128, 8, 64
    pages = (1 << 31) // (D * Hk * page) + 3
    q, kc, vc, table, n = make(1, [150], 8, Hk, D, page, torch.bfloat16, seed=9, fill=0.0)
    ref = decode(q, kc, vc, table, n)
    big = [torch.empty(pages, page, Hk, D, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    far = torch.arange(pages - 3, pages, device=dev)
    for b, c in zip(big, (kc, vc)):
        b[far] = c[table[0].long()].to(dev)
    o = gdr.paged_decode_step(q.to(dev), *big, far.to(torch.int32)[None], n.to(dev))
    assert rel_heads(o, ref, 1) <= TOL["bf16"]
    new = torch.randn(1, 1, Hk, D, device=dev).bfloat16()
    gdr.kv_append(new, new, *big, far.to(torch.int32)[None], n.to(dev))
    assert torch.equal(big[0][pages - 1, 150 - 128], new[0, 0]) and torch.equal(big[1][pages - 1, 150 - 128], new[0, 0])


def test_refusals():
    dev = cuda_device()
    q, kc, vc, table, n = (t.to(dev) for t in make(2, [20, 5], 4, 2, 64, 16, torch.bfloat16))
    f = gdr.paged_decode_step
    for bad in (lambda: f(q.cpu(), kc, vc, table, n), lambda: f(q, kc, vc[:1], table, n), lambda: f(q, kc.float(), vc.float(), table, n),
                lambda: f(q, kc, vc, table.long(), n), lambda: f(q, kc, vc, table, n.long()), lambda: f(q, kc, vc, table[:1], n),
                lambda: f(q, kc, vc, table, n, window=-1), lambda: f(q, kc, vc, table, n, out=q[:, :2]), lambda: f(q[0], kc, vc, table, n),
                lambda: f(q, kc, vc, table, n, workspace=torch.empty(8, dtype=torch.uint8, device=dev)), lambda: f(q, kc[0], vc, table, n),
                lambda: f(q, kc[..., :32].contiguous(), vc[..., :32].contiguous(), table, n)):
        with pytest.raises(ValueError):
            bad()
    for call, code in ((lambda: f(q, kc, vc, table, n, scale=float("inf")), 1), (lambda: f(q[:, :3].contiguous(), kc, vc, table, n), 1),
                       (lambda: f(q, kc, vc, table, n, scale=-0.1), 1)):
        with pytest.raises(gdr.GdrError) as e:
            call()
        assert e.value.code == code


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_caches_on_the_16_byte_grid_only(dtype):
    dev = cuda_device()
    q, kc, vc, table, n = make(2, [70, 33], 4, 2, 64, 16, TYPES[dtype], seed=10)
    ref = decode(q, kc, vc, table, n)
    step = 16 // TYPES[dtype].itemsize

    def view(x, by):
        flat = torch.empty(x.numel() + 64, dtype=x.dtype, device=dev)
        y = flat[by:by + x.numel()].view(x.shape)
        y.copy_(x)
        return y

    args = table.to(dev), n.to(dev)
    assert rel_heads(gdr.paged_decode_step(view(q, step), view(kc, step), view(vc, 3 * step), *args), ref, 1) <= TOL[dtype]
    for bad in ((1, 0, 0), (0, 1, 0), (0, 0, 1)):
        with pytest.raises(gdr.GdrError) as e:
            gdr.paged_decode_step(view(q, bad[0]), view(kc, bad[1]), view(vc, bad[2]), *args)
        assert e.value.code == 1


def test_rows_behind_the_last_sequence_stay_as_they_were():
    """Outputs in the first rows of a larger buffer."""
    dev = cuda_device()
    for B in (3, 50):
        q, kc, vc, table, n = (t.to(dev) for t in make(B, [30 + i for i in range(B)], 4, 2, 64, 16, torch.bfloat16, seed=11))
        buf = torch.full((B + 2, 4, 64), 3.0, dtype=torch.bfloat16, device=dev)
        o = gdr.paged_decode_step(q, kc, vc, table, n, out=buf[:B])
        assert torch.equal(o, gdr.paged_decode_step(q, kc, vc, table, n)) and (buf[B:] == 3.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B", [2, 60])
def test_values_that_are_none_are_not_hidden(B, dtype):
    """NaN in a query, a key or a value that is seen reaches the output, of that head alone; infinite keys as in the formula."""
    dev = cuda_device()
    q, kc, vc, table, n = make(B, [900 + b for b in range(B)], 4, 2, 64, 16, TYPES[dtype], seed=12)
    ref = decode(q, kc, vc, table, n)
    q[0, 1] = float("nan")
    page = table[1].long()
    kc[page[3], 5, 0, 7] = float("nan")  # heads 0 and 1 of entry 1
    vc[page[50], 2, 1, 3] = float("nan")  # heads 2 and 3, channel 3
    o = gdr.paged_decode_step(*(t.to(dev) for t in (q, kc, vc, table, n)))
    bad = torch.zeros(B, 4, 64, dtype=torch.bool, device=dev)
    bad[0, 1] = bad[1, :2] = bad[1, 2:, 3] = True
    assert torch.equal(o.isnan(), bad)
    bad = bad.cpu()
    bad[0, 1] = bad[1, 2:] = True  # whole heads, as the bound is one on heads
    good = ~bad[..., 0].flatten()
    assert rel_heads(o.flatten(0, 1)[good.to(dev)], ref.flatten(0, 1)[good], 0) <= TOL[dtype]
    q, kc, vc, table, n = make(B, [900 + b for b in range(B)], 4, 2, 64, 16, TYPES[dtype], seed=12)
    q[1] = q[1].abs()
    kc[table[1, 3].long(), 5] = -float("inf")  # a score of -inf: not seen
    x = (q, kc, vc, table, n)
    assert rel_heads(gdr.paged_decode_step(*(t.to(dev) for t in x)), decode(*x), 1) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("room", [0, 100, 390, 1300, 5000])
@pytest.mark.parametrize("B,Hk", [(1, 1), (5, 3), (8, 2), (9, 4), (37, 1), (19, 4), (77, 1), (38, 8), (61, 5)])
def test_walks_and_room(B, Hk, room, dtype):
    """Across the numbers of walks and the lengths of tables where CTAs alone, clusters and runs take them."""
    n = [(53 * i * i + 7) % 190 for i in range(B)]
    q, kc, vc, table, lengths = make(B, n, 2 * Hk, Hk, 128, 16, TYPES[dtype], seed=B)
    wide = torch.full((B, table.shape[1] + -(-room // 16)), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    check((q, kc, vc, wide, lengths), dtype, window=150, sinks=3)
