"""Measured cases of linear attention with a decay per head and of the per-token group norm.

Linear attention, per batch entry b and value head hv (key head hk = hv // (Hv / Hk)), with the
head's constant log-decay g[hv] <= 0, a state S [Dv, Dk] and n_b valid tokens:

    S_t = exp(g) S_{t-1} + v_t k_t^T,    o_t = scale S_t q_t,    scale = Dk^-1/2

Group norm of rows x [rows, C] whose channels form `groups` runs of C / groups, with statistics
per row and group, and the activation on the normalised value or on a gate z beside it:

    n = w (x - mean) / sqrt(var + eps) + b,    y = act(n)   or   y = n act(z)

`run` computes them in plain fp32 torch, or, where `own` is true, through the package.
"""
import math

import torch

own = False

EPS = 1e-5
CHUNK = 128
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOKEN_HEADS = 32768 * 32    # tokens x value heads of the largest prompt
STATE_HEADS = 128 * 32      # states of the largest decode batch
NORM_VALUES = 32768 * 4096  # elements of the largest normalised tensor


def listed():
    heads = {"Hk": 16, "Hv": 32, "Dk": 128, "Dv": 128}
    return [
        # one sequence generating: a token's latency is what the user waits for
        {"name": "step-1", "op": "step", "B": 1, "dtype": "bf16", **heads},
        # a full decode batch: 256 MB of states, larger than L2
        {"name": "step-128", "op": "step", "B": 128, "dtype": "bf16", **heads},
        # short prompts of unequal lengths batched together, continuing earlier states; narrow keys, three value heads a key
        {"name": "prompt-ragged", "op": "prompt", "B": 7, "T": 333, "Hk": 4, "Hv": 12, "Dk": 64, "Dv": 128, "dtype": "bf16",
         "ragged": True, "initial": True},
        # one ordinary prompt
        {"name": "prompt-4096", "op": "prompt", "B": 1, "T": 4096, "dtype": "bf16", "ragged": False, "initial": False, **heads},
        # one long context
        {"name": "prompt-32768", "op": "prompt", "B": 1, "T": 32768, "dtype": "bf16", "ragged": False, "initial": False, **heads},
        # full precision, as in a check of a model against its reference outputs
        {"name": "prompt-fp32", "op": "prompt", "B": 2, "T": 1000, "Hk": 8, "Hv": 8, "Dk": 64, "Dv": 64, "dtype": "fp32",
         "ragged": False, "initial": True},
        # a training batch of short sequences
        {"name": "train-8x512", "op": "train", "B": 8, "T": 512, "dtype": "bf16", "ragged": False, "initial": False, **heads},
        # the long-context training step, one state carried in and its gradient out
        {"name": "train-32768", "op": "train", "B": 1, "T": 32768, "dtype": "bf16", "ragged": False, "initial": True, **heads},
        # the output norm of one decoded token for each sequence of a batch
        {"name": "norm-128", "op": "norm", "rows": 128, "groups": 32, "D": 128, "dtype": "bf16", "act": "silu", "gate": True,
         "affine": True, "center": True},
        # the output norm of a long prompt, in its form without mean and offsets
        {"name": "norm-32768", "op": "norm", "rows": 32768, "groups": 32, "D": 128, "dtype": "bf16", "act": "silu", "gate": True,
         "affine": True, "center": False},
        # the same rows in training, mean and offsets included
        {"name": "norm-train-32768", "op": "norm_train", "rows": 32768, "groups": 32, "D": 128, "dtype": "bf16", "act": "silu",
         "gate": True, "affine": True, "center": True},
        # odd sizes in full precision, the activation on the normalised value itself
        {"name": "norm-train-odd", "op": "norm_train", "rows": 5001, "groups": 6, "D": 99, "dtype": "fp32", "act": "silu",
         "gate": False, "affine": True, "center": True},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["step", "prompt", "prompt", "train", "train", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("norm", "norm_train"):
        groups, D = rng.choice([1, 2, 5, 8, 16, 32, 64]), rng.choice([rng.randint(8, 600), 32, 64, 128, 256])
        rows = _log(rng, 1, max(1, NORM_VALUES // (groups * D * (1 if dtype == "bf16" else 2))) if groups * D > 4096 else 32768)
        return {"op": op, "rows": rows, "groups": groups, "D": D, "dtype": dtype, "act": rng.choice(["silu", "silu", "sigmoid", "none"]),
                "gate": rng.random() < 0.7, "affine": rng.random() < 0.7, "center": rng.random() < 0.6}
    Hk, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 2, 3, 4, 8])
    while Hk * G > 32:
        G -= 1
    heads = {"Hk": Hk, "Hv": Hk * G, "Dk": rng.choice([32, 64, 128, 128]), "Dv": rng.choice([32, 64, 128, 128]), "dtype": dtype}
    if op == "step":
        return {"op": op, "B": _log(rng, 1, STATE_HEADS // (Hk * G)), **heads}
    # the fp32 form's cost a token is that of eight bf16 tokens
    most = TOKEN_HEADS // (Hk * G) // (8 if dtype == "fp32" else 1)
    T = _log(rng, 1, min(32768, most))
    return {"op": op, "B": _log(rng, 1, max(1, min(64, most // T))), "T": T, "ragged": rng.random() < 0.4, "initial": rng.random() < 0.5, **heads}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def randn(*size, std=1.0, mean=0.0, to=dt):
        return (torch.randn(*size, generator=gen, device=dev) * std + mean).to(to)

    s = dict(case)
    if case["op"] in ("norm", "norm_train"):
        rows, C = case["rows"], case["groups"] * case["D"]
        grads = case["op"] == "norm_train"
        s["x"] = randn(rows, C, std=1.5, mean=0.3).requires_grad_(grads)
        s["z"] = randn(rows, C).requires_grad_(grads) if case["gate"] else None
        s["w"] = randn(C, std=0.1, mean=1.0, to=torch.float32).requires_grad_(grads) if case["affine"] else None
        s["b"] = randn(C, std=0.1, to=torch.float32).requires_grad_(grads) if case["affine"] and case["center"] else None
        s["dy"] = randn(rows, C) if grads else None
        return s
    B, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "Hk", "Hv", "Dk", "Dv"))
    # half-lives from a token or two to hundreds of tokens over the heads, as fixed decays are laid out
    slope = 1.0 + 8.0 * torch.arange(Hv, device=dev) / max(1, Hv - 1) + 0.5 * torch.rand(Hv, generator=gen, device=dev)
    s["g"] = -torch.exp2(-slope).float()
    if case["op"] == "step":
        s["q"], s["k"], s["v"] = randn(B, Hk, Dk), randn(B, Hk, Dk), randn(B, Hv, Dv)
        s["state"] = randn(B, Hv, Dv, Dk, to=torch.float32)
        return s
    T, grads = case["T"], case["op"] == "train"
    s["q"], s["k"], s["v"] = (randn(B, T, h, d).requires_grad_(grads) for h, d in ((Hk, Dk), (Hk, Dk), (Hv, Dv)))
    s["h0"] = randn(B, Hv, Dv, Dk, to=torch.float32).requires_grad_(grads) if case["initial"] else None
    s["lengths"] = None
    if case["ragged"]:  # one entry as long as the batch, one empty where there are three or more
        n = torch.randint(0, T + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        n[0] = T
        if B > 2:
            n[1] = 0
        s["lengths"] = n
    if grads:
        s["do"], s["dht"] = randn(B, T, Hv, Dv), randn(B, Hv, Dv, Dk, std=0.1, to=torch.float32)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gated_delta_rule_31_gb300 as gdr
    from gated_delta_rule_31_gb300.autograd import group_norm, linear_attention

    op = s["op"]
    if op == "step":
        o = gdr.linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"])
        return {"o": o, "state": s["state"]}
    if op == "prompt":
        o, ht = gdr.linear_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], lengths=s["lengths"])
        return {"o": o, "ht": ht}
    if op == "train":
        o, ht = linear_attention(s["q"], s["k"], s["v"], s["g"], s["h0"], lengths=s["lengths"])
        of = [x for x in (s["q"], s["k"], s["v"], s["h0"]) if x is not None]
        grads = torch.autograd.grad((o, ht), of, (s["do"], s["dht"]))
        return {"o": o.detach(), "ht": ht.detach(), **dict(zip(("dq", "dk", "dv", "dh0"), grads))}
    kw = {"activation": s["act"], "eps": EPS, "center": s["center"]}
    if op == "norm":
        return {"y": gdr.group_norm_fwd(s["x"], s["groups"], s["w"], s["b"], s["z"], **kw)}
    y = group_norm(s["x"], s["groups"], s["w"], s["b"], s["z"], **kw)
    of = [(n, s[k]) for n, k in (("dx", "x"), ("dz", "z"), ("dw", "w"), ("db", "b")) if s[k] is not None]
    return {"y": y.detach(), **dict(zip([n for n, _ in of], torch.autograd.grad(y, [x for _, x in of], s["dy"])))}


@torch.no_grad()
def _run_plain(s):
    op = s["op"]
    if op in ("norm", "norm_train"):
        return _plain_norm(s)
    G = s["Hv"] // s["Hk"]
    scale = s["Dk"] ** -0.5
    g = s["g"].float()
    if op == "step":
        q, k = (x.float().repeat_interleave(G, 1) for x in (s["q"], s["k"]))
        S = s["state"].mul_(torch.exp(g)[:, None, None]).add_(s["v"].float()[..., None] * k[:, :, None, :])
        return {"o": (scale * torch.matmul(S, q[..., None])[..., 0]).to(s["v"].dtype), "state": S}
    B, T, Hv = s["B"], s["T"], s["Hv"]
    dev = g.device
    pos = torch.arange(T, device=dev)
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=dev)
    valid = pos[None] < n[:, None]  # [B, T]

    def heads(x):  # [B, T, H, D] -> [B, Hv, T, D] in fp32, zero past each length
        x = torch.where(valid[..., None, None], x.float(), 0.0).transpose(1, 2)
        return x.repeat_interleave(Hv // x.shape[1], 1)

    q, k, v = heads(s["q"]), heads(s["k"]), heads(s["v"])
    since = torch.exp(g[:, None] * (pos + 1))[None, :, :, None]  # decay from before token 0 through t
    left = (n[:, None] - 1 - pos[None]).clamp(min=0)  # tokens after t
    until = torch.where(valid[:, None], torch.exp(g[None, :, None] * left[:, None]), 0.0)[..., None]
    over = torch.exp(g[None] * n[:, None])[..., None, None]  # decay over all of a row's tokens
    mask = valid[:, None, :, None]
    o = _mix(q, k, v, g)
    ht = torch.matmul((v * until).transpose(2, 3), k)
    if s["h0"] is not None:
        o = o + since * torch.matmul(q, s["h0"].transpose(2, 3))
        ht = ht + over * s["h0"]
    out = {"o": torch.where(mask, scale * o, 0.0).transpose(1, 2).to(s["v"].dtype).contiguous(), "ht": ht}
    if op == "prompt":
        return out
    do, dht = heads(s["do"]), s["dht"]
    dq = scale * _mix(do, v, k, g)
    dk = scale * _mix(v, do, q, g, reverse=True) + until * torch.matmul(v, dht)
    dv = scale * _mix(k, q, do, g, reverse=True) + until * torch.matmul(k, dht.transpose(2, 3))
    if s["h0"] is not None:
        dq = dq + scale * since * torch.matmul(do, s["h0"])
        out["dh0"] = over * dht + scale * torch.matmul((do * since).transpose(2, 3), q)

    def of_key_heads(x):  # the sum over the value heads that share a key head
        return torch.where(mask, x, 0.0).reshape(B, s["Hk"], G, T, -1).sum(2).transpose(1, 2).to(s["q"].dtype).contiguous()

    out["dq"], out["dk"] = of_key_heads(dq), of_key_heads(dk)
    out["dv"] = torch.where(mask, dv, 0.0).transpose(1, 2).to(s["v"].dtype).contiguous()
    return out


def _mix(a, b, c, g, reverse=False):
    """sum over j <= t (j >= t in reverse) of exp(g |t - j|) (a_t . b_j) c_j, by chunks of tokens."""
    if reverse:
        return _mix(a.flip(2), b.flip(2), c.flip(2), g).flip(2)
    B, H, T = a.shape[:3]
    N = -(-T // CHUNK)
    C = CHUNK if N > 1 else T
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, N * C - T)).reshape(B, H, N, C, -1) for x in (a, b, c))
    i = torch.arange(C, device=a.device)
    gh = g[:, None, None]
    E = torch.where(i[:, None] >= i, torch.exp(gh * (i[:, None] - i).clamp(min=0)), 0.0)
    out = torch.matmul(torch.matmul(a, b.transpose(3, 4)) * E[:, None], c)
    if N > 1:
        part = torch.matmul((b * torch.exp(gh * (C - 1 - i))[..., None]).transpose(3, 4), c)  # [B, H, N, D1, D2]
        m = torch.arange(N, device=a.device)
        L = torch.where(m[:, None] > m, torch.exp(gh * (C * (m[:, None] - 1 - m)).clamp(min=0)), 0.0)
        start = torch.matmul(L, part.reshape(B, H, N, -1)).reshape(part.shape)
        out = out + torch.matmul(a * torch.exp(gh * (i + 1))[..., None], start)
    return out.reshape(B, H, N * C, -1)[:, :, :T]


def _act(x, name):
    """The activation and its derivative."""
    if name == "none":
        return x, torch.ones_like(x)
    sig = 1.0 / (1.0 + torch.exp(-x))
    if name == "sigmoid":
        return sig, sig * (1.0 - sig)
    return x * sig, sig * (1.0 + x * (1.0 - sig))


def _plain_norm(s):
    dt = s["x"].dtype
    shape = (s["rows"], s["groups"], s["D"])
    x = s["x"].float().view(shape)
    w = s["w"].view(shape[1:]) if s["w"] is not None else 1.0
    b = s["b"].view(shape[1:]) if s["b"] is not None else 0.0
    if s["center"]:
        x = x - x.mean(2, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(2, keepdim=True) + EPS)
    h = x * r
    n = h * w + b
    z = s["z"].float().view(shape) if s["z"] is not None else None
    f, df = _act(n if z is None else z, s["act"])
    out = {"y": (f if z is None else n * f).to(dt).view(s["rows"], -1)}
    if s["op"] == "norm":
        return out
    dy = s["dy"].float().view(shape)
    dn = dy * (df if z is None else f)
    dh = dn * w
    dx = dh - h * (dh * h).mean(2, keepdim=True)
    if s["center"]:
        dx = dx - dh.mean(2, keepdim=True)
    out["dx"] = (dx * r).to(dt).view(s["rows"], -1)
    if z is not None:
        out["dz"] = (dy * n * df).to(dt).view(s["rows"], -1)
    if s["w"] is not None:
        out["dw"] = (dn * h).sum(0).view(-1)
    if s["b"] is not None:
        out["db"] = dn.sum(0).view(-1)
    return out


def exact(case, seed):
    """The definitions in 64 bits: the recurrence token by token and its reverse, and the norm with gradients by
    automatic differentiation of its definition."""
    s = prepare(case, seed)
    return _exact_norm(s) if case["op"] in ("norm", "norm_train") else _exact_linear(s)


def _exact_norm(s):
    x, z, w, b = (s[n].detach().double().requires_grad_() if s[n] is not None else None for n in "xzwb")
    rows, groups, D = s["rows"], s["groups"], s["D"]
    t = x.view(rows, groups, D)
    n = (t - t.mean(-1, keepdim=True) if s["center"] else t)
    n = (n / (n.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()).reshape(rows, groups * D)
    n = n if w is None else n * w
    n = n if b is None else n + b
    f = {"none": lambda u: u, "sigmoid": torch.sigmoid, "silu": torch.nn.functional.silu}[s["act"]]
    y = f(n) if z is None else n * f(z)
    out = {"y": y.detach()}
    if s["op"] == "norm_train":
        of = [(name, v) for name, v in (("dx", x), ("dz", z), ("dw", w), ("db", b)) if v is not None]
        out.update(zip([name for name, _ in of], torch.autograd.grad(y, [v for _, v in of], s["dy"].double(), materialize_grads=True)))
    return out


@torch.no_grad()
def _exact_linear(s):
    G = s["Hv"] // s["Hk"]
    scale = 1.0 / math.sqrt(s["Dk"])
    lam = s["g"].double().exp()
    if s["op"] == "step":
        q, k = (s[n].double()[:, torch.arange(s["Hv"], device=lam.device) // G] for n in "qk")
        S = lam[:, None, None] * s["state"].double() + torch.einsum("bhv,bhk->bhvk", s["v"].double(), k)
        return {"o": scale * torch.einsum("bhvk,bhk->bhv", S, q), "state": S}
    B, T, Hv, Dk, Dv = (s[n] for n in ("B", "T", "Hv", "Dk", "Dv"))
    dev = lam.device
    n = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
    steps = max(n)

    def tokens(name):  # [T, B * Hv, D], key heads repeated; zero past the lengths
        x = s[name].detach().double()
        x = x[:, :, torch.arange(Hv, device=dev) // (Hv // x.shape[2])].permute(1, 0, 2, 3).contiguous()
        for i, m in enumerate(n):
            x[m:, i] = 0
        return x.reshape(T, B * Hv, -1)

    q, k, v = tokens("q"), tokens("k"), tokens("v")
    S = torch.zeros(B, Hv, Dv, Dk, dtype=torch.float64, device=dev)
    if s["h0"] is not None:
        S += s["h0"].detach()
    S = S.view(B * Hv, Dv, Dk)
    live = torch.tensor([[t < m for m in n] for t in range(T)], device=dev)  # [T, B]
    fade = torch.where(live[:, :, None], lam, 1.0).reshape(T, B * Hv, 1, 1)
    train = s["op"] == "train"
    o = torch.zeros(T, B * Hv, Dv, dtype=torch.float64, device=dev)
    if train:
        do = tokens("do")
        dq, dk, dv = (torch.zeros_like(x) for x in (q, k, v))
    for t in range(steps):
        S.mul_(fade[t]).baddbmm_(v[t, :, :, None], k[t, :, None, :])
        o[t] = torch.bmm(S, q[t, :, :, None])[..., 0]
        if train:
            dq[t] = torch.bmm(do[t, :, None, :], S)[:, 0]
    keep = live.repeat_interleave(Hv, 1)[..., None]

    def back(x, heads=Hv, factor=scale):
        return (factor * torch.where(keep, x, 0.0)).view(T, B, heads, Hv // heads, -1).sum(3).transpose(0, 1).contiguous()

    out = {"o": back(o), "ht": S.clone().view(B, Hv, Dv, Dk)}
    if train:
        R = s["dht"].double().reshape(B * Hv, Dv, Dk).clone()
        for t in reversed(range(steps)):
            R.baddbmm_(do[t, :, :, None], q[t, :, None, :], alpha=scale)
            dk[t] = torch.bmm(v[t, :, None, :], R)[:, 0]
            dv[t] = torch.bmm(R, k[t, :, :, None])[..., 0]
            R.mul_(fade[t])
        out.update(dq=back(dq, s["Hk"]), dk=back(dk, s["Hk"], 1.0), dv=back(dv, factor=1.0))
        if s["h0"] is not None:
            out["dh0"] = R.view(B, Hv, Dv, Dk)
    return out


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        n, C = case["rows"] * case["groups"] * case["D"], case["groups"] * case["D"]
        tensors = (3 if case["gate"] else 2) if case["op"] == "norm" else (6 if case["gate"] else 4)
        # training reads x, z and dy once and writes y, dx and dz
        vectors = (1 + case["center"]) * case["affine"] * (1 if case["op"] == "norm" else 2)
        return {"bytes": n * e * tensors + C * 4 * vectors, "flops": n * (10 if case["op"] == "norm" else 30)}
    B, Hk, Hv, Dk, Dv = (case[n] for n in ("B", "Hk", "Hv", "Dk", "Dv"))
    states = B * Hv * Dv * Dk
    if case["op"] == "step":
        return {"bytes": 8 * states + e * B * (2 * Hk * Dk + 2 * Hv * Dv) + 4 * Hv, "flops": 5 * states}
    # a ragged batch's lengths are spread over 0..T: half of its tokens are there; o, and in training dq, dk and dv, are written whole
    tok = B * case["T"]
    read = tok * (0.5 if case["ragged"] and B > 1 else 1.0)
    qkv = 2 * Hk * Dk + Hv * Dv
    nbytes = e * (read * qkv + tok * Hv * Dv) + 4 * states * (2 if case["initial"] else 1) + 4 * Hv
    flops = 4.0 * read * Hv * Dv * Dk
    if case["op"] == "train":  # once over q, k, v, dO; the gradients in the inputs' type
        nbytes += e * (read * Hv * Dv + tok * qkv) + 4 * states * (2 if case["initial"] else 1)
        flops *= 3.5
    return {"bytes": nbytes, "flops": flops}
