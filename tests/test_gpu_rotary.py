"""Rotary positions and the append to a paged cache on the GPU against their formulas in 64 bits.

Bounds, on each element against the length of its pair: the sine and cosine are off by up to 2^-22 (their own rounding,
2^-23 at most with sincospi's two last places, and the angle's 2^-32 of a turn), a product and a sum round once each: 4 x
2^-23 in all, and the result's rounding, 2^-24 in fp32 and 2^-8 in bf16."""
import pytest
import torch

import gated_delta_rule_31_gb300 as gdr
from attention_ref import make_cache, rows, turn
from gated_delta_rule_31_gb300.autograd import rotary
from util import cuda_device

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOL = {torch.float32: 4 * 2.0 ** -23 + 2.0 ** -24, torch.bfloat16: 4 * 2.0 ** -23 + 2.0 ** -8}


def freqs(pairs, dev=None):
    return (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(1, pairs))).float().to(dev)


def close(y, ref, x, dtype):
    """Elements against the largest of their head (a pair's length is at most sqrt 2 of that)."""
    assert y.dtype == dtype and y.shape == x.shape
    y, top = y.detach().double().cpu(), x.detach().double().cpu().abs().amax(-1, keepdim=True) * 2 ** 0.5
    assert torch.isfinite(y).all()
    assert ((y - ref).abs() <= TOL[dtype] * top).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R,sections", [(128, 64, None), (128, 64, (16, 24, 24)), (64, 32, (1, 31)), (128, 32, (0, 8, 8, 16)), (64, 12, (5, 7)),
                                          (96, 48, (16, 16, 16)), (32, 0, None), (10, 5, (2, 3)), (10, 3, None), (2, 1, None), (256, 7, (7, 0))])
def test_forms(D, R, sections, interleaved, dtype):
    dev = cuda_device()
    gen = torch.Generator().manual_seed(R + D)
    B, T, H = 2, 37, 5
    x = torch.randn(B, T, H, D, generator=gen).to(TYPES[dtype])
    p = torch.randint(0, 5000, (B, T, len(sections) if sections else 1), generator=gen, dtype=torch.int32)
    f = freqs(R)
    ref = turn(x, p, f, sections, interleaved)
    y = gdr.rotary(x.to(dev), p.to(dev), f.to(dev), sections=sections, interleaved=interleaved)
    close(y, ref, x, TYPES[dtype])
    assert torch.equal(y[..., 2 * R:].cpu(), x[..., 2 * R:])
    # in place, and back
    z = x.to(dev)
    assert gdr.rotary(z, p.to(dev), f.to(dev), sections=sections, interleaved=interleaved, out=z) is z and torch.equal(z, y)
    w = gdr.rotary(x.to(dev), p.to(dev), f.to(dev), sections=sections, interleaved=interleaved, inverse=True)
    close(w, turn(x, p, f, sections, interleaved, inverse=True), x, TYPES[dtype])


@pytest.mark.parametrize("H", [1, 2, 3, 4, 7, 32, 33])
@pytest.mark.parametrize("lead", [(1,), (3, 1), (2, 3, 4), (700,)])
def test_heads_and_leading_shapes(lead, H):
    dev = cuda_device()
    x = torch.randn(*lead, H, 64).bfloat16()
    p = torch.randint(-100, 1000, lead, dtype=torch.int32)
    ref = turn(x, p[..., None], freqs(32))
    close(gdr.rotary(x.to(dev), p.to(dev), freqs(32, dev)), ref, x, torch.bfloat16)
    close(gdr.rotary(x.to(dev), p[..., None].contiguous().to(dev), freqs(32, dev)), ref, x, torch.bfloat16)


def test_far_positions():
    """Angles of far positions keep their fraction of a turn; in fp32 they would be off by whole turns."""
    dev = cuda_device()
    p = torch.tensor([0, 1, -1, 2 ** 20 + 1, 2 ** 24 - 1, 10 ** 8 + 7, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    x = torch.randn(8, 2, 64)
    f = torch.cat((freqs(28), torch.tensor([0.0, -0.3, 1.0, 1e-20])))
    for inverse in (False, True):
        y = gdr.rotary(x.to(dev), p.to(dev), f.to(dev), inverse=inverse)
        # the reference's own angle, rounded to 53 bits: 2^31 x 2^-53 radians, below 2^-21
        ref = turn(x, p[:, None], f, inverse=inverse)
        top = x.double().abs().amax(-1, keepdim=True) * 2 ** 0.5
        assert ((y.double().cpu() - ref).abs() <= (TOL[torch.float32] + 2.0 ** -21) * top).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [1, 2, 3, 4])
def test_off_the_16_byte_grid(offset, dtype):
    dev = cuda_device()
    gen = torch.Generator().manual_seed(offset)
    flat = torch.randn(offset + 20 * 3 * 64, generator=gen).to(TYPES[dtype]).to(dev)
    x = flat[offset:].view(20, 3, 64)
    p = torch.arange(20, dtype=torch.int32, device=dev)
    close(gdr.rotary(x, p, freqs(32, dev)), turn(x.cpu(), p.cpu()[:, None], freqs(32)), x.cpu(), TYPES[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_autograd(dtype):
    dev = cuda_device()
    x = torch.randn(2, 9, 3, 64, device=dev).to(TYPES[dtype]).requires_grad_()
    p = torch.randint(0, 99999, (2, 9, 2), dtype=torch.int32, device=dev)
    g = torch.randn(2, 3, 9, 64, device=dev).to(TYPES[dtype])
    y = rotary(x, p, freqs(32, dev), sections=(10, 22))
    y.transpose(1, 2).backward(g)
    g = g.transpose(1, 2)
    close(x.grad, turn(g, p, freqs(32), (10, 22), inverse=True), g, TYPES[dtype])
    # against differences: the map is linear
    e = torch.randn_like(x)
    slope = float((g.double() * (gdr.rotary(e, p, freqs(32, dev), sections=(10, 22)).double())).sum())
    assert abs(slope - float((x.grad.double() * e.double()).sum())) <= 2 * TOL[TYPES[dtype]] * float(g.double().norm() * e.double().norm())
    with pytest.raises(ValueError):
        rotary(x, p, freqs(32, dev).requires_grad_(), sections=(10, 22))


def test_empty():
    dev = cuda_device()
    assert gdr.rotary(torch.empty(0, 4, 64, device=dev), torch.empty(0, dtype=torch.int32, device=dev), freqs(32, dev)).shape == (0, 4, 64)


def test_refusals():
    dev = cuda_device()
    x, p, f = torch.zeros(5, 2, 64, device=dev), torch.zeros(5, dtype=torch.int32, device=dev), freqs(32, dev)
    for bad in (lambda: gdr.rotary(x.cpu(), p, f), lambda: gdr.rotary(x, p.long(), f), lambda: gdr.rotary(x, p[:4], f),
                lambda: gdr.rotary(x, p, f.double()), lambda: gdr.rotary(x, p, f, sections=(16, 16)),
                lambda: gdr.rotary(x, p, f, sections=(16, 15, 1, 0, 0)), lambda: gdr.rotary(x, p, f, sections=(33, -1)),
                lambda: gdr.rotary(x, p, f, out=torch.empty(5, 2, 32, device=dev)), lambda: gdr.rotary(x[:, 0], p, f[None]),
                lambda: gdr.rotary(x.half(), p, f), lambda: gdr.rotary(x.transpose(0, 1), p, f)):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: gdr.rotary(x[..., :62].contiguous(), p, f), 1), (lambda: gdr.rotary(x[..., :33].contiguous(), p, f[:16].contiguous()), 2),
                      (lambda: gdr.rotary(x[:, :0].contiguous(), p, f), 1)):
        with pytest.raises(gdr.GdrError) as e:
            bad()
        assert e.value.code == code


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R,page", [(1, 1, 4, 1, 128, 64, 16), (5, 1, 3, 3, 64, 16, 1), (3, 40, 8, 2, 32, 16, 24), (2, 100, 0, 5, 128, 0, 64),
                                                (4, 33, 6, 2, 36, 9, 7)])
def test_append(B, T, Hq, Hk, D, R, page, dtype):
    """Ragged counts, some of them none, behind sequences of unequal lengths; every row that is not written stays as it was."""
    dev = cuda_device()
    gen = torch.Generator().manual_seed(T + D)
    dt = TYPES[dtype]
    q, k, v = (torch.randn(B, T, h, D, generator=gen).to(dt) for h in (Hq, Hk, Hk))
    counts = torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32) if T > 1 else None
    if counts is not None:
        counts[0], counts[-1] = T, 0
        for b in range(B):  # what lies past an entry's tokens is not used
            for x in (q, k, v):
                x[b, counts[b]:] = float("nan")
    lengths = torch.randint(0, 50, (B,), generator=gen, dtype=torch.int32)
    table, kc, vc = make_cache(B, 50 + T, page, Hk, D, dt, seed=B, fill=7.0)
    f = freqs(R) if R else None
    sections = (R // 2, R - R // 2) if R > 10 else None
    p = torch.randint(0, 10 ** 6, (B, T, 2 if sections else 1), generator=gen, dtype=torch.int32) if R else None
    dk, dv = kc.to(dev), vc.to(dev)
    y = gdr.kv_append(k.to(dev), v.to(dev), dk, dv, table.to(dev), lengths.to(dev), inv_freq=None if f is None else f.to(dev),
                      positions=None if p is None else p.to(dev), sections=sections,
                      counts=None if counts is None else counts.to(dev), q=q.to(dev) if Hq else None)
    assert (y is None) == (Hq == 0)
    want_k, want_v = kc.double(), vc.double()
    top = torch.ones_like(want_k[..., :1])
    for b in range(B):
        n = T if counts is None else int(counts[b])
        pg, r = (x[int(lengths[b]):] for x in rows(table, b, int(lengths[b]) + n, page))
        want_k[pg, r] = turn(k[b, :n], p[b, :n], f, sections) if R else k[b, :n].double()
        want_v[pg, r] = v[b, :n].double()
        if n:
            top[pg, r] = k[b, :n].double().abs().amax(-1, keepdim=True)
        if Hq:
            assert not y[b, n:].any()
            if n:
                close(y[b, :n], turn(q[b, :n], p[b, :n], f, sections) if R else q[b, :n].double(), q[b, :n], dt)
    assert torch.equal(dv.double().cpu(), want_v)
    assert ((dk.double().cpu() - want_k).abs() <= TOL[dt] * 2 ** 0.5 * top).all()


def test_append_without_positions_uses_the_place():
    dev = cuda_device()
    k, v, q = (torch.randn(2, 5, 2, 64, device=dev) for _ in range(3))
    lengths = torch.tensor([300000, 3], dtype=torch.int32, device=dev)
    table = torch.full((2, 300005 // 64 + 1), -1, dtype=torch.int32, device=dev)
    table[0, 300000 // 64], table[1, 0] = 1, 0
    a, b = torch.zeros(2, 2, 64, 2, 64, device=dev)
    y = gdr.kv_append(k, v, a, b, table, lengths, inv_freq=freqs(32, dev), q=q)
    place = lengths[:, None] + torch.arange(5, dtype=torch.int32, device=dev)
    assert torch.equal(y, gdr.rotary(q, place, freqs(32, dev)))
    want = gdr.rotary(k, place, freqs(32, dev))
    first = 300000 % 64
    assert torch.equal(a[1, first:first + 5], want[0]) and torch.equal(a[0, 3:8], want[1]) and torch.equal(b[0, 3:8], v[1])
    z = q.clone()
    assert gdr.kv_append(k, v, a, b, table, lengths, inv_freq=freqs(32, dev), q=z, q_out=z) is z and torch.equal(z, y)


def test_append_writes_nothing_where_there_is_no_page():
    """Page numbers below and above the cache, places past the table's end and before its beginning."""
    dev = cuda_device()
    k, v = torch.randn(2, 4, 12, 1, 32, device=dev)
    table = torch.tensor([[0, -1], [2, 1 << 30], [-2 ** 31, 1], [2 ** 31 - 1, 3]], dtype=torch.int32, device=dev)
    lengths = torch.tensor([4, 0, -6, 2 ** 31 - 4], dtype=torch.int32, device=dev)
    guard = torch.full((2, 3 + 2, 8, 1, 32), 5.0, device=dev)
    a, b = guard[0, 1:4], guard[1, 1:4]  # a cache of three pages between two that are somebody else's
    gdr.kv_append(k, v, a, b, table, lengths)
    want = torch.full_like(guard, 5.0)
    for i, x in enumerate((k, v)):
        want[i, 1, 4:8] = x[0, :4]      # entry 0: the rest goes to page -1
        want[i, 3, 0:8] = x[1, :8]      # entry 1: the rest to a page far away
    # entry 2: places -6 .. 5 are before the sequence or on no page; entry 3: past the table, past 2^31
    assert torch.equal(guard, want)


def test_append_refusals():
    dev = cuda_device()
    k = torch.zeros(2, 3, 2, 64, device=dev)
    cache, table, n = torch.zeros(4, 8, 2, 64, device=dev), torch.zeros(2, 2, dtype=torch.int32, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    f = freqs(32, dev)
    ok = dict(k=k, v=k, k_cache=cache, v_cache=cache.clone(), page_table=table, lengths=n)
    p = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    for bad in (dict(v=k[:, :2]), dict(k_cache=cache.bfloat16()), dict(v_cache=cache[:2]), dict(page_table=table.long()), dict(lengths=n[:1]),
                dict(page_table=table[:1]), dict(counts=n.float()), dict(positions=p), dict(inv_freq=f, positions=p[:, :2]), dict(q=k[0]),
                dict(q_out=k), dict(inv_freq=f, sections=(16, 16)), dict(k_cache=cache[..., :32].contiguous()), dict(q=k, q_out=k.double())):
        with pytest.raises(ValueError):
            gdr.kv_append(**{**ok, **bad})
