"""Plain 64-bit forms for the tests of linear attention with a decay per head and of the per-token
group norm: the recurrence token by token, its reverse, and the norm by its definition."""
import torch


def rel(x, ref):
    """||x - ref|| / ||ref||; a zero reference wants exact zeros."""
    x, ref = x.detach().double().cpu(), ref.detach().double().cpu()
    assert x.shape == ref.shape, (x.shape, ref.shape)
    assert torch.isfinite(x).all()
    d, n = float((x - ref).norm()), float(ref.norm())
    return d / n if n else (0.0 if d == 0 else float("inf"))


def rel_heads(x, ref, axis):
    """The largest rel() over the slices of one axis, so that no head hides behind another."""
    return max([rel(a, b) for a, b in zip(x.unbind(axis), ref.unbind(axis))], default=0.0)


def make(B, T, Hk, Hv, Dk, Dv, dtype, seed=0, initial=True, lengths=None, g=None, fill=float("nan"), grads=True):
    """CPU inputs; tokens past the lengths hold `fill`."""
    gen = torch.Generator().manual_seed(seed)

    def randn(*s, std=1.0, to=dtype):
        return (torch.randn(*s, generator=gen) * std).to(to)

    d = dict(q=randn(B, T, Hk, Dk), k=randn(B, T, Hk, Dk), v=randn(B, T, Hv, Dv), do=randn(B, T, Hv, Dv))
    d["g"] = -torch.exp2(-1.0 - 8.0 * torch.arange(Hv) / max(1, Hv - 1)) if g is None else torch.full((Hv,), float(g))
    d["g"] = d["g"].float()
    d["h0"] = randn(B, Hv, Dv, Dk, to=torch.float32) if initial else None
    d["dht"] = randn(B, Hv, Dv, Dk, std=0.3, to=torch.float32) if initial else None
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32)
    if lengths is not None:
        for b, n in enumerate(lengths):
            for name in ("q", "k", "v", "do"):
                d[name][b, max(0, n):] = fill
    return d


def linear(q, k, v, g, h0=None, lengths=None, do=None, dht=None, scale=None, decode=False, grads=True, **_):
    """o, ht and, with do, dq, dk, dv, dh0 in 64 bits."""
    B, T, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    G = Hv // Hk
    scale = Dk ** -0.5 if scale is None else scale
    lam = torch.exp(g.double())
    n = [T] * B if lengths is None else [min(max(int(x), 0), T) for x in lengths]
    f = lambda x: x.double().repeat_interleave(Hv // x.shape[2], 2)  # noqa: E731
    q, k, v = f(q), f(k), f(v)
    grads = grads and do is not None
    do = f(do) if grads else None
    o = torch.zeros(B, T, Hv, Dv, dtype=torch.float64)
    ht = torch.zeros(B, Hv, Dv, Dk, dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dh0 = torch.zeros_like(ht)
    for b in range(B):
        S = h0[b].double().clone() if h0 is not None else torch.zeros_like(ht[b])
        for t in range(n[b]):
            S = lam[:, None, None] * S + v[b, t, :, :, None] * k[b, t, :, None, :]
            o[b, t] = scale * torch.einsum("hvk,hk->hv", S, q[b, t])
            if grads:
                dq[b, t] = scale * torch.einsum("hvk,hv->hk", S, do[b, t])
        ht[b] = S
        if grads:
            D = dht[b].double().clone() if dht is not None else torch.zeros_like(S)
            for t in reversed(range(n[b])):
                D = D + scale * do[b, t, :, :, None] * q[b, t, :, None, :]
                dk[b, t] = torch.einsum("hvk,hv->hk", D, v[b, t])
                dv[b, t] = torch.einsum("hvk,hk->hv", D, k[b, t])
                D = lam[:, None, None] * D
            dh0[b] = D
    out = dict(o=o, ht=ht)
    if grads:
        s = lambda x: x.view(B, T, Hk, G, -1).sum(3)  # noqa: E731
        out.update(dq=s(dq), dk=s(dk), dv=dv, dh0=dh0)
    return out


def group_norm(x, groups, weight=None, bias=None, gate=None, activation="none", eps=1e-5, center=True):
    f = {"none": lambda u: u, "sigmoid": torch.sigmoid, "silu": lambda u: u * torch.sigmoid(u)}[activation]
    t = x.reshape(-1, groups, x.shape[-1] // groups)
    if center:
        t = t - t.mean(-1, keepdim=True)
    n = (t / torch.sqrt((t * t).mean(-1, keepdim=True) + eps)).reshape(x.shape)
    n = n * weight if weight is not None else n
    n = n + bias if bias is not None else n
    return f(n) if gate is None else n * f(gate)
