"""Measured cases of the softmax attention layer of a mixed model: attention with a sliding window and visible
first tokens, rotary positions, the paged cache that a served sequence appends to, and the decode step that reads it.

Attention, per batch entry b with n_b valid tokens and query head h (key head h // (Hq / Hk)):

    o_t = sum_j p_tj v_j,   p_t = softmax over the visible j of scale q_t . k_j,   scale = D^-1/2,
    visible: j <= t, j < n_b, and t - j < window (0: any) or j < sinks.

Rotary: of the first R channels of a head, the pairs (i, i + R/2), or (2 i, 2 i + 1) when interleaved, are turned by
the angle positions[axis of i] * inv_freq[i]; `sections` says how many pairs each axis has, in order.

Paged cache [pages, page_size, Hk, D]: token j of entry b lies in page page_table[b, j // page_size], row j % page_size.

`run` computes them in plain fp32 torch (angles in 64 bits), or, where `own` is true, through the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
TOKEN_HEADS = 32768 * 32          # tokens x query heads of the longest prompt
PAIRS = 32768 * 1024 * 32         # visible pairs x query heads of the largest prompt with a window
CACHE_TOKENS = 64 * 16384 * 8     # cached tokens x key heads of the largest decode batch
ROTATED = 32768 * 32 * 128        # elements of the largest rotated tensor


def listed():
    heads = {"Hq": 32, "Hk": 8, "D": 128}
    full = {"window": 0, "sinks": 0}
    return [
        # one sequence generating: a token's latency is what the user waits for
        {"name": "decode-1", "op": "decode", "B": 1, "L": 4096, "page": 64, "dtype": "bf16", "ragged": False, **full, **heads},
        # a full batch of sequences of all lengths, some of them just begun
        {"name": "decode-64", "op": "decode", "B": 64, "L": 16384, "page": 16, "dtype": "bf16", "ragged": True, **full, **heads},
        # long sequences of a layer that sees a window and the first tokens
        {"name": "decode-window", "op": "decode", "B": 128, "L": 9000, "page": 64, "dtype": "bf16", "ragged": True, "window": 1024,
         "sinks": 4, **heads},
        # one token of each sequence of a batch written to the cache, far positions
        {"name": "append-64", "op": "append", "B": 64, "T": 1, "page": 16, "dtype": "bf16", "ragged": False, "R": 128, "before": 500,
         "sections": "64", "interleaved": False, "start": 300000, **heads},
        # prompts of unequal lengths written behind what is cached, half of the channels rotated
        {"name": "append-prompts", "op": "append", "B": 5, "T": 4001, "page": 64, "dtype": "bf16", "ragged": True, "R": 64, "before": 77,
         "sections": "32", "interleaved": False, "start": 0, **heads},
        # the queries of one image between text, time, height and width
        {"name": "rotary-image", "op": "rotary", "B": 1, "T": 1500, "H": 32, "D": 128, "dtype": "bf16", "R": 128,
         "sections": "16 24 24", "interleaved": False, "start": 100},
        # the queries of a long training sequence with video, and their gradient
        {"name": "rotary-train", "op": "rotary_train", "B": 1, "T": 32768, "H": 32, "D": 128, "dtype": "bf16", "R": 128,
         "sections": "16 24 24", "interleaved": True, "start": 0},
        # short prompts of unequal lengths batched together, narrow heads, three query heads a key head
        {"name": "prompt-ragged", "op": "prompt", "B": 7, "T": 333, "Hq": 12, "Hk": 4, "D": 64, "dtype": "bf16", "ragged": True,
         "window": 100, "sinks": 4},
        # one long prompt of a layer that sees everything
        {"name": "prompt-16384", "op": "prompt", "B": 1, "T": 16384, "dtype": "bf16", "ragged": False, **full, **heads},
        # a training batch of short sequences, a key head for each query head
        {"name": "train-8x512", "op": "train", "B": 8, "T": 512, "Hq": 16, "Hk": 16, "D": 128, "dtype": "bf16", "ragged": False, **full},
        # odd sizes in full precision, as in a check of a model against its reference outputs
        {"name": "train-fp32", "op": "train", "B": 2, "T": 777, "Hq": 8, "Hk": 4, "D": 64, "dtype": "fp32", "ragged": True,
         "window": 300, "sinks": 2},
        # the long-context training step
        {"name": "train-32768", "op": "train", "B": 1, "T": 32768, "dtype": "bf16", "ragged": False, "window": 1024, "sinks": 4, **heads},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _sections(rng, half):
    if half < 8 or rng.random() < 0.4:
        return f"{half}"
    if rng.random() < 0.3:
        a = rng.randint(1, half - 1)
        return f"{a} {half - a}"
    a = rng.randint(1, half // 3)
    b = rng.randint(1, half // 2)
    return f"{a} {b} {half - a - b}"


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "rotary", "rotary_train", "prompt", "prompt", "train", "train"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    D = rng.choice([32, 64, 128, 128])
    if op in ("rotary", "rotary_train", "append"):
        R = D if rng.random() < 0.6 else rng.choice([r for r in (8, 16, 32, 64, 96) if r <= D])
        turn = {"D": D, "dtype": dtype, "R": R, "sections": _sections(rng, R // 2), "interleaved": rng.random() < 0.4,
                "start": rng.choice([0, 0, 1000, 300000, 1000000])}
        H = rng.choice([1, 2, 3, 5, 8, 16, 32])
        T = _log(rng, 1, min(32768, ROTATED // (H * D)))
        if op != "append":
            return {"op": op, "B": _log(rng, 1, max(1, min(64, ROTATED // (H * D * T)))), "T": T, "H": H, **turn}
        G = rng.choice([1, 2, 3, 4, 8])
        T = min(T, ROTATED // (2 * H * G * D))
        return {"op": op, "B": _log(rng, 1, max(1, min(64, ROTATED // (4 * H * G * D * T)))), "T": T, "Hq": H * G, "Hk": H,
                "page": rng.choice([1, 16, 16, 24, 32, 64, 64, 128]), "ragged": rng.random() < 0.5, "before": _log(rng, 1, 3000), **turn}
    Hk, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 3, 4, 4, 8])
    while Hk * G > 32:
        G -= 1
    seen = {"window": 0, "sinks": 0}
    if rng.random() < 0.6:
        seen = {"window": _log(rng, 1, 4096), "sinks": rng.choice([0, 0, 1, 4, 4, 16, 130])}
    heads = {"Hq": Hk * G, "Hk": Hk, "D": D, "dtype": dtype, **seen}
    most = 2 if dtype == "fp32" else 1
    if op == "decode":
        L = _log(rng, 1, min(131072, CACHE_TOKENS // (Hk * most)))
        return {"op": op, "B": _log(rng, 1, max(1, min(256, CACHE_TOKENS // (Hk * L * most)))), "L": L,
                "page": rng.choice([1, 16, 16, 24, 32, 64, 64, 128, 256]), "ragged": rng.random() < 0.6, **heads}
    # in fp32 a pair's cost is that of sixteen bf16 pairs; half of all pairs are visible where there is no window
    pairs = PAIRS // (Hk * G) // (16 if dtype == "fp32" else 1)
    T = _log(rng, 1, min(32768, TOKEN_HEADS // (Hk * G)))
    cost = lambda t: t * (t / 2 if not seen["window"] else min(t, seen["window"] + seen["sinks"]))  # noqa: E731
    while cost(T) > pairs:
        T = T * 2 // 3
    return {"op": op, "B": _log(rng, 1, max(1, min(64, int(pairs / cost(T)), TOKEN_HEADS // (Hk * G * T)))), "T": T,
            "ragged": rng.random() < 0.4, **heads}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = TYPES[case["dtype"]]

    def randn(*size, std=1.0):
        return (torch.randn(*size, generator=gen, device=dev) * std).to(dt)

    def randint(low, high, *size):
        return torch.randint(low, high, size, generator=gen, device=dev, dtype=torch.int32)

    def ragged(B, T):  # one entry as long as the batch, one empty where there are three or more
        n = randint(1, T + 1, B)
        n[0] = T
        if B > 2:
            n[1] = 0
        return n

    def paged(B, tokens):  # pages handed out in no order, some of them nobody's
        per = -(-tokens // case["page"])
        pages = B * per + 3
        table = torch.randperm(pages, generator=gen, device=dev)[:B * per].view(B, per).to(torch.int32)
        size = (pages, case["page"], case["Hk"], case["D"])
        return table, randn(*size), randn(*size)

    s = dict(case)
    op = case["op"]
    if op in ("rotary", "rotary_train", "append"):
        half = case["R"] // 2
        s["sections"] = [int(x) for x in case["sections"].split()]
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
        B, T = case["B"], case["T"]
        # text, then a picture of some columns whose rows follow one another, by time, height and width
        t = torch.arange(T, device=dev)[None] + case["start"] + randint(0, 50, B)[:, None]
        axes = [t, case["start"] + t // 37 % 64, case["start"] + t % 37][:len(s["sections"])]
        s["positions"] = torch.stack(axes, -1).to(torch.int32).contiguous()
        if op == "append":
            s["q"], s["k"], s["v"] = randn(B, T, case["Hq"], case["D"]), randn(B, T, case["Hk"], case["D"]), randn(B, T, case["Hk"], case["D"])
            s["counts"] = ragged(B, T) if case["ragged"] else None
            s["lengths"] = randint(0, case["before"] + 1, B)
            s["table"], s["k_cache"], s["v_cache"] = paged(B, case["before"] + T)
        else:
            grads = op == "rotary_train"
            s["x"] = randn(B, T, case["H"], case["D"]).requires_grad_(grads)
            s["dy"] = randn(B, T, case["H"], case["D"]) if grads else None
        return s
    B, Hq, Hk, D = (case[n] for n in ("B", "Hq", "Hk", "D"))
    if op == "decode":
        s["q"] = randn(B, Hq, D)
        s["lengths"] = ragged(B, case["L"]) if case["ragged"] else torch.full((B,), case["L"], device=dev, dtype=torch.int32)
        s["table"], s["k_cache"], s["v_cache"] = paged(B, case["L"])
        return s
    T, grads = case["T"], op == "train"
    s["q"], s["k"], s["v"] = (randn(B, T, h, D).requires_grad_(grads) for h in (Hq, Hk, Hk))
    s["lengths"] = ragged(B, T) if case["ragged"] else None
    s["do"] = randn(B, T, Hq, D) if grads else None
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    import gated_delta_rule_31_gb300 as gdr
    from gated_delta_rule_31_gb300.autograd import rotary, window_attention

    op = s["op"]
    if op == "decode":
        return {"o": gdr.paged_decode_step(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], window=s["window"], sinks=s["sinks"])}
    if op in ("prompt", "train"):
        kw = {"window": s["window"], "sinks": s["sinks"], "lengths": s["lengths"]}
        if op == "prompt":
            return {"o": gdr.window_attention_fwd(s["q"], s["k"], s["v"], **kw)[0]}
        o = window_attention(s["q"], s["k"], s["v"], **kw)
        return {"o": o.detach(), **dict(zip(("dq", "dk", "dv"), torch.autograd.grad(o, (s["q"], s["k"], s["v"]), s["do"])))}
    kw = {"sections": tuple(s["sections"]), "interleaved": s["interleaved"]}
    if op == "append":
        q = gdr.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], inv_freq=s["inv_freq"],
                          positions=s["positions"], counts=s["counts"], q=s["q"], **kw)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "rotary":
        return {"y": gdr.rotary(s["x"], s["positions"], s["inv_freq"], **kw)}
    y = rotary(s["x"], s["positions"], s["inv_freq"], **kw)
    return {"y": y.detach(), "dx": torch.autograd.grad(y, s["x"], s["dy"])[0]}


@torch.no_grad()
def _run_plain(s):
    op = s["op"]
    if op == "decode":
        return _plain_decode(s)
    if op in ("prompt", "train"):
        return _plain_attention(s)
    cos, sin = _angles(s)
    if op == "rotary":
        return {"y": _turn(s["x"], cos, sin, s)}
    if op == "rotary_train":
        return {"y": _turn(s["x"], cos, sin, s), "dx": _turn(s["dy"], cos, -sin, s)}
    B, T, P = s["B"], s["T"], s["page"]
    t = torch.arange(T, device=cos.device)
    at = s["lengths"].long()[:, None] + t  # place of each token in its sequence
    page = torch.gather(s["table"].long(), 1, (at // P).clamp(max=s["table"].shape[1] - 1))
    row = page * P + at % P
    k, v = _turn(s["k"], cos, sin, s), s["v"]
    q = _turn(s["q"], cos, sin, s)
    if s["counts"] is not None:  # tokens past an entry's count go where another of its tokens goes, with that one's values
        live = t < s["counts"][:, None]
        q = torch.where(live[..., None, None], q, 0.0)
        last = (s["counts"].long() - 1).clamp(min=0)[:, None]
        from_ = torch.where(live, t.expand(B, T), last)
        rows = torch.gather(row, 1, from_)
        take = from_[..., None, None].expand(k.shape)
        k, v = torch.gather(k, 1, take), torch.gather(v, 1, take)
        kc, vc = (s[n].view(-1, s["Hk"], s["D"]) for n in ("k_cache", "v_cache"))
        some = (s["counts"] > 0)[:, None, None, None]
        k, v = torch.where(some, k, kc[rows]), torch.where(some, v, vc[rows])
        row = rows
    for name, x in (("k_cache", k), ("v_cache", v)):
        s[name].view(-1, s["Hk"], s["D"]).index_put_((row.reshape(-1),), x.reshape(-1, s["Hk"], s["D"]))
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _angles(s):
    """Cosines and sines [B, T, 1, R/2] in fp32 of angles in 64 bits."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"])), torch.tensor(s["sections"])).to(s["positions"].device)
    a = s["positions"].double()[..., axis] * s["inv_freq"].double()
    return a.cos().float()[:, :, None], a.sin().float()[:, :, None]


def _turn(x, cos, sin, s):
    R = s["R"]
    f = x[..., :R].float()
    if s["interleaved"]:
        a, b = f[..., 0::2], f[..., 1::2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = f[..., :R // 2], f[..., R // 2:]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y.to(x.dtype), x[..., R:]), -1)


def _plain_decode(s):
    B, Hk, D, P = s["B"], s["Hk"], s["D"], s["page"]
    n = s["lengths"].long()[:, None]
    L = s["table"].shape[1] * P
    if s["window"] and s["window"] + s["sinks"] < L:  # the first tokens, then the last ones
        w = torch.arange(s["window"], device=n.device)
        first = torch.arange(s["sinks"], device=n.device).expand(B, -1)
        start = (n - s["window"]).clamp(min=0)
        j = torch.cat((first, start + w), 1)
        seen = torch.cat((first < torch.minimum(n, start), start + w < n), 1)
    else:
        j = torch.arange(min(L, s["L"]), device=n.device).expand(B, -1)
        seen = j < n
        if s["window"]:
            seen = seen & ((n - 1 - j < s["window"]) | (j < s["sinks"]))
    j = torch.where(seen, j, 0)
    row = torch.gather(s["table"].long(), 1, j // P) * P + j % P
    k, v = (s[c].view(-1, Hk, D)[row].float().transpose(1, 2) for c in ("k_cache", "v_cache"))  # [B, Hk, J, D]
    q = s["q"].float().view(B, Hk, -1, D)
    sc = torch.matmul(q, k.transpose(2, 3)) * D ** -0.5
    sc = torch.where(seen[:, None, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return {"o": o.view(B, s["Hq"], D).to(s["q"].dtype)}


def _plain_attention(s):
    B, T, Hq, Hk, D = (s[n] for n in ("B", "T", "Hq", "Hk", "D"))
    G, W, sinks, scale = Hq // Hk, s["window"], s["sinks"], s["D"] ** -0.5
    dt, dev = s["q"].dtype, s["q"].device
    train = s["op"] == "train"
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=dev)

    def heads(x):  # [B, T, H, D] -> [B, Hk, H / Hk, T, D]
        live = torch.arange(T, device=dev) < n[:, None]
        return torch.where(live[..., None, None], x.float(), 0.0).permute(0, 2, 1, 3).reshape(B, Hk, -1, T, D)

    q, k, v = heads(s["q"]), heads(s["k"])[:, :, 0], heads(s["v"])[:, :, 0]
    o = torch.zeros_like(q)
    if train:
        do = heads(s["do"])
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    C = max(64, min(512, 2 ** 28 // (B * Hq * max(1, min(T, W + sinks + 512) if W else T))))
    for t0 in range(0, T, C):
        t1 = min(T, t0 + C)
        lo = max(0, t0 - W + 1) if W else 0
        parts = [(lo, t1)] if lo == 0 or sinks == 0 else [(0, min(sinks, lo)), (lo, t1)]
        t, j = torch.arange(t0, t1, device=dev)[:, None], torch.cat([torch.arange(a, b, device=dev) for a, b in parts])
        seen = j <= t
        if W:
            seen = seen & ((t - j < W) | (j < sinks))
        seen = seen & (j < n[:, None, None]) & (t < n[:, None, None])  # [B, t, j]
        seen = seen[:, None, None]
        kj, vj = (torch.cat([x[:, :, a:b] for a, b in parts], 2)[:, :, None] for x in (k, v))
        sc = torch.matmul(q[:, :, :, t0:t1], kj.transpose(3, 4)) * scale
        sc = torch.where(seen, sc, -math.inf)
        m = sc.amax(-1, keepdim=True)
        p = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
        ot = torch.matmul(p, vj)
        o[:, :, :, t0:t1] = ot
        if train:
            g = do[:, :, :, t0:t1]
            ds = p * (torch.matmul(g, vj.transpose(3, 4)) - (g * ot).sum(-1, keepdim=True)) * scale
            dq[:, :, :, t0:t1] = torch.matmul(ds, kj)
            rows = ds.transpose(3, 4), p.transpose(3, 4)
            dkj, dvj = torch.matmul(rows[0], q[:, :, :, t0:t1]).sum(2), torch.matmul(rows[1], g).sum(2)
            at = 0
            for a, b in parts:
                dk[:, :, a:b] += dkj[:, :, at:at + b - a]
                dv[:, :, a:b] += dvj[:, :, at:at + b - a]
                at += b - a

    def back(x, H):
        return x.reshape(B, H, T, D).transpose(1, 2).to(dt).contiguous()

    out = {"o": back(o, Hq)}
    if train:
        out.update(dq=back(dq, Hq), dk=back(dk, Hk), dv=back(dv, Hk))
    return out


def exact(case, seed):
    """The definitions in 64 bits: rotations as products of complex numbers, attention entry by entry with gradients
    by automatic differentiation."""
    if case["op"] in ("prompt", "train"):
        seen = case["T"] / 2 if not case["window"] else min(case["T"], case["window"] + case["sinks"] + 300)
        if case["B"] * case["T"] * seen * case["Hq"] * case["D"] * (4 if case["op"] == "prompt" else 14) > 6e12:
            return None
    s = prepare(case, seed)
    if case["op"] in ("prompt", "train"):
        return _exact_attention(s)
    with torch.no_grad():
        return _exact_decode(s) if case["op"] == "decode" else _exact_rotary(s)


def _exact_turn(x, s, sign=1.0):
    R = s["R"]
    y = x.detach().double().clone()
    first = 0
    for axis, pairs in enumerate(s["sections"]):
        i = torch.arange(first, first + pairs, device=y.device)
        a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + R // 2)
        angle = sign * s["positions"][..., axis, None].double() * s["inv_freq"][i].double()
        z = torch.complex(x.detach().double()[..., a], x.detach().double()[..., b]) * torch.polar(torch.ones_like(angle), angle)[:, :, None]
        y[..., a], y[..., b] = z.real, z.imag
        first += pairs
    return y


def _exact_rotary(s):
    if s["op"] != "append":
        out = {"y": _exact_turn(s["x"], s)}
        if s["op"] == "rotary_train":
            out["dx"] = _exact_turn(s["dy"], s, -1.0)
        return out
    q, k = _exact_turn(s["q"], s), _exact_turn(s["k"], s)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    n = s["counts"].tolist() if s["counts"] is not None else [s["T"]] * s["B"]
    for b, (m, before) in enumerate(zip(n, s["lengths"].tolist())):
        q[b, m:] = 0
        place = torch.arange(before, before + m, device=q.device)
        page = s["table"][b].long()[place // s["page"]]
        kc[page, place % s["page"]] = k[b, :m]
        vc[page, place % s["page"]] = s["v"][b, :m].double()
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _exact_decode(s):
    B, Hq, Hk, D, P = (s[n] for n in ("B", "Hq", "Hk", "D", "page"))
    o = torch.zeros(B, Hq, D, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(s["lengths"].tolist()):
        j = [x for x in range(n) if not s["window"] or n - 1 - x < s["window"] or x < s["sinks"]]
        if not j:
            continue
        j = torch.tensor(j, device=o.device)
        page = s["table"][b].long()[j // P]
        k, v = (s[c][page, j % P].double().repeat_interleave(Hq // Hk, 1) for c in ("k_cache", "v_cache"))
        w = torch.softmax(torch.einsum("hd,jhd->hj", s["q"][b].double(), k) / math.sqrt(D), -1)
        o[b] = torch.einsum("hj,jhd->hd", w, v)
    return {"o": o}


def _exact_attention(s):
    B, T, Hq, Hk, D = (s[n] for n in ("B", "T", "Hq", "Hk", "D"))
    G, W, sinks, train = Hq // Hk, s["window"], s["sinks"], s["op"] == "train"
    dev = s["q"].device
    z = lambda name: torch.zeros(s[name].shape, dtype=torch.float64, device=dev)  # noqa: E731
    out = {"o": z("q")}
    if train:
        out.update(dq=z("q"), dk=z("k"), dv=z("v"))
    n = s["lengths"].tolist() if s["lengths"] is not None else [T] * B
    step = 256
    for b in range(B):
        for h in range(Hk):
            hq = slice(h * G, (h + 1) * G)
            for t0 in range(0, n[b], step):
                t1 = min(n[b], t0 + step)
                j = torch.arange(t1, device=dev)
                if W:
                    j = j[(j < sinks) | (j > t0 - W)]
                t = torch.arange(t0, t1, device=dev)[:, None]
                hide = j > t
                if W:
                    hide = hide | ((t - j >= W) & (j >= sinks))
                q, k, v = (x.detach().double().requires_grad_(train)
                           for x in (s["q"][b, t0:t1, hq], s["k"][b, :, h][j], s["v"][b, :, h][j]))
                a = (torch.einsum("tgd,jd->gtj", q, k) / math.sqrt(D)).masked_fill(hide, -math.inf)
                o = torch.einsum("gtj,jd->tgd", torch.softmax(a, -1), v)
                out["o"][b, t0:t1, hq] = o.detach()
                if train:
                    gq, gk, gv = torch.autograd.grad(o, (q, k, v), s["do"][b, t0:t1, hq].double())
                    out["dq"][b, t0:t1, hq] = gq
                    out["dk"][b, :, h].index_add_(0, j, gk)
                    out["dv"][b, :, h].index_add_(0, j, gv)
    return out


def _mean_min(most, w):
    """The mean of min(u, w) for u spread evenly over 0 .. most."""
    return most / 2 if w >= most else w - w * w / (2 * most)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, B = case["op"], case["B"]
    if op in ("rotary", "rotary_train"):
        n = B * case["T"] * case["H"] * case["D"] * (2 if op == "rotary_train" else 1)
        return {"bytes": 2 * n * e + B * case["T"] * 4 * len(case["sections"].split()), "flops": 3 * n * case["R"] / case["D"]}
    D, Hq, Hk, W, sinks = case["D"], case["Hq"], case["Hk"], case.get("window", 0), case.get("sinks", 0)
    ragged = case["ragged"] and B > 1
    if op == "append":
        tok = B * case["T"]
        live = tok * (0.5 if ragged else 1.0)  # of a ragged batch; q's rows are written whole
        return {"bytes": e * D * (live * (Hq + 4 * Hk) + tok * Hq) + tok * 4 * len(case["sections"].split()), "flops": 3 * live * (Hq + Hk) * case["R"]}
    if op == "decode":
        w = min(case["L"], W + sinks) if W else case["L"]
        seen = B * (_mean_min(case["L"], w) if ragged else w)
        return {"bytes": e * (2 * seen * Hk * D + 2 * B * Hq * D), "flops": 4.0 * seen * Hq * D}

    def pairs(n):  # visible pairs of a sequence of n tokens
        if not W:
            return n * (n + 1) / 2
        w = min(n, W)
        return n * w - w * (w - 1) / 2 + min(sinks, max(0, n - w)) * max(0, n - w)

    T = case["T"]
    # lengths of a ragged batch are spread over 0 .. T
    seen = B * (sum(pairs(T * (i + 0.5) / 8) for i in range(8)) / 8 if ragged else pairs(T))
    live = B * T * (0.5 if ragged else 1.0)
    nbytes = e * D * (live * (Hq + 2 * Hk) + B * T * Hq)
    flops = 4.0 * seen * Hq * D
    if op == "train":  # do and the gradients; five products backwards
        nbytes += e * D * (live * Hq + B * T * (Hq + 2 * Hk))
        flops *= 3.5
    return {"bytes": nbytes, "flops": flops}
