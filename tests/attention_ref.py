"""Plain 64-bit forms for the tests of the softmax attention layer: attention entry by entry and head by head with its
gradients from their formulas, rotation by complex numbers, and a paged cache kept as a list of rows."""
import torch


def make(B, T, Hq, Hk, D, dtype, seed=0, lengths=None, fill=float("nan"), std=1.0):
    """CPU inputs; tokens past the lengths hold `fill`."""
    gen = torch.Generator().manual_seed(seed)
    d = {n: (torch.randn(B, T, h, D, generator=gen) * s).to(dtype)
         for n, h, s in (("q", Hq, std), ("k", Hk, 1.0), ("v", Hk, 1.0), ("do", Hq, 1.0))}
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    if lengths is not None:
        for b, n in enumerate(lengths):
            for name in ("q", "k", "v", "do"):
                d[name][b, max(0, n):] = fill
    return d


def seen(t, j, window, sinks):
    ok = j <= t
    if window:
        ok = ok & ((t - j < window) | (j < sinks))
    return ok


def attention(q, k, v, lengths=None, do=None, window=0, sinks=0, scale=None):
    """o, lse and, with do, dq, dk, dv, and the sizes of what cancels in dq and dk: the same sums with every product's size."""
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    f = torch.float64
    out = {"o": torch.zeros(B, T, Hq, D, dtype=f), "lse": torch.full((B, Hq, T), -float("inf"), dtype=f)}
    if do is not None:
        out.update(dq=torch.zeros(B, T, Hq, D, dtype=f), dk=torch.zeros(B, T, Hk, D, dtype=f), dv=torch.zeros(B, T, Hk, D, dtype=f))
        out.update(dq_size=torch.zeros_like(out["dq"]), dk_size=torch.zeros_like(out["dk"]))
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        if n == 0:
            continue
        hide = ~seen(torch.arange(n)[:, None], torch.arange(n), window, sinks)
        for h in range(Hq):
            hk = h // (Hq // Hk)
            qh, kh, vh = (x[b, :n, i].detach().double().cpu() for x, i in ((q, h), (k, hk), (v, hk)))
            s = (scale * qh @ kh.T).masked_fill(hide, -float("inf"))
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None])
            o = p @ vh
            out["o"][b, :n, h], out["lse"][b, h, :n] = o, lse
            if do is not None:
                g = do[b, :n, h].detach().double().cpu()
                ds = p * (g @ vh.T - (g * o).sum(1, keepdim=True)) * scale
                out["dq"][b, :n, h] = ds @ kh
                out["dk"][b, :n, hk] += ds.T @ qh
                out["dv"][b, :n, hk] += p.T @ g
                size = p * (g.abs() @ vh.T.abs() + (g * o).abs().sum(1, keepdim=True)) * scale
                out["dq_size"][b, :n, h] = size @ kh.abs()
                out["dk_size"][b, :n, hk] += size.T @ qh.abs()
    return out


def turn(x, positions, inv_freq, sections=None, interleaved=False, inverse=False):
    """x [..., H, D] turned; positions [..., axes]."""
    R = inv_freq.numel()
    sections = [R] if sections is None else sections
    y = x.detach().double().cpu().clone()
    x = y.clone()
    p, f = positions.double().cpu(), inv_freq.double().cpu()
    i0 = 0
    for axis, n in enumerate(sections):
        for i in range(i0, i0 + n):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R)
            angle = p[..., axis] * f[i] * (-1.0 if inverse else 1.0)
            c, s = torch.cos(angle)[..., None], torch.sin(angle)[..., None]
            y[..., a], y[..., b] = c * x[..., a] - s * x[..., b], s * x[..., a] + c * x[..., b]
        i0 += n
    return y


def make_cache(B, tokens, page, Hk, D, dtype, seed=0, spare=2, fill=float("nan")):
    """(page table, k cache, v cache) with pages handed out in no order; every row holds `fill`."""
    gen = torch.Generator().manual_seed(seed)
    per = -(-tokens // page) if tokens else 1
    pages = B * per + spare
    table = torch.randperm(pages, generator=gen)[:B * per].view(B, per).to(torch.int32)
    return table, *(torch.full((pages, page, Hk, D), fill, dtype=dtype) for _ in range(2))


def rows(table, b, n, page):
    """(page, row) of the first n tokens of entry b."""
    j = torch.arange(n)
    return table[b].long().cpu()[j // page], j % page


def decode(q, k_cache, v_cache, table, lengths, window=0, sinks=0, scale=None):
    B, Hq, D = q.shape
    pages, page, Hk, _ = k_cache.shape
    scale = D ** -0.5 if scale is None else scale
    o = torch.zeros(B, Hq, D, dtype=torch.float64)
    kc, vc = k_cache.cpu(), v_cache.cpu()
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * page)
        j = torch.arange(n)
        ok = seen(torch.tensor(n - 1), j, window, sinks)
        pg = table[b].long().cpu()[j // page]
        j = j[ok & (pg >= 0) & (pg < pages)]
        if len(j) == 0:
            continue
        pg = table[b].long().cpu()[j // page]
        k, v = kc[pg, j % page].double(), vc[pg, j % page].double()  # [J, Hk, D]
        for h in range(Hq):
            hk = h // (Hq // Hk)
            p = torch.softmax(scale * k[:, hk] @ q[b, h].detach().double().cpu(), 0)
            o[b, h] = p @ v[:, hk]
    return o
