"""Group layer norm, multi-axis rotary positions and document attention: what is measured.

Three operators of an EQ-ViT block, each in two forms: elementary torch
operations in 32 bits (``own`` false) and the calls a user makes of the
library (``own`` true).  ``exact`` evaluates the definitions in 64 bits.

Features are [C', T] per token, index c*T + t, as in every layer of this
library; attention heads split C'.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one image through the smallest model's norm: a serving call, latency counts
        {"name": "norm-one-image", "op": "norm", "dtype": "bf16", "N": 197, "Cp": 96, "T": 4, "res": False, "train": False},
        # EQ-ViT-B training: the norm after a residual add, both directions, 64 images
        {"name": "norm-vit-b-train", "op": "norm", "dtype": "bf16", "N": 12608, "Cp": 192, "T": 4, "res": True, "train": True},
        # EQ-Swin-T stage 1 training: very many short rows
        {"name": "norm-swin-train", "op": "norm", "dtype": "f16", "N": 401408, "Cp": 24, "T": 4, "res": False, "train": True},
        # one image's queries and keys, two axes (height, width): a serving call
        {"name": "rope-one-image", "op": "rope", "dtype": "bf16", "docs": 1, "grid": "1 14 14", "heads": 12, "extra": 6,
         "Ch": 16, "T": 4, "sections": "4 4", "inverse": False, "far": 0},
        # clips of 16 frames in a training batch, three axes, the gradient's direction, late in a long video
        {"name": "rope-video-back", "op": "rope", "dtype": "f16", "docs": 8, "grid": "16 14 14", "heads": 24, "extra": 12,
         "Ch": 16, "T": 4, "sections": "2 3 3", "inverse": True, "far": 100000},
        # one image of an EQ-ViT-B block, inference
        {"name": "attn-one-image", "op": "attn", "dtype": "bf16", "lens": "197", "lead": 0, "tail": 0, "heads": 12,
         "kv": 12, "D": 64, "cap": 30.0, "bias": 0, "train": False},
        # images of different sizes packed into one batch, inference, with padding behind the last
        {"name": "attn-packed-images", "op": "attn", "dtype": "f16",
         "lens": "197 1 577 50 0 1025 133 784 256 401 63 2049 320 129 900 17", "lead": 0, "tail": 55,
         "heads": 6, "kv": 2, "D": 64, "cap": 0.0, "bias": 2, "train": False},
        # an EQ-ViT-B training batch, capped scores and distance bias
        {"name": "attn-vit-b-train", "op": "attn", "dtype": "bf16", "docs": 64, "len": 197, "heads": 12, "kv": 12, "D": 64,
         "cap": 30.0, "bias": 2, "train": True},
        # the windows of EQ-Swin-T stage 1 (7 x 7 patches, 32 features per head), training
        {"name": "attn-swin-windows-train", "op": "attn", "dtype": "f16", "docs": 2048, "len": 49, "heads": 3, "kv": 3,
         "D": 32, "cap": 0.0, "bias": 2, "train": True},
        # one long clip (16 frames of 28 x 28 patches), training
        {"name": "attn-video-train", "op": "attn", "dtype": "bf16", "docs": 1, "len": 12544, "heads": 6, "kv": 6, "D": 64,
         "cap": 0.0, "bias": 3, "train": True},
        # wide heads, two query heads for each key head, training on ragged documents
        {"name": "attn-wide-heads-train", "op": "attn", "dtype": "bf16", "lens": "1500 700 2333 1 3011 555", "lead": 4,
         "tail": 24, "heads": 8, "kv": 4, "D": 128, "cap": 50.0, "bias": 0, "train": True},
        # 32-bit training of a small model
        {"name": "attn-f32-train", "op": "attn", "dtype": "f32", "docs": 16, "len": 197, "heads": 6, "kv": 6, "D": 64,
         "cap": 30.0, "bias": 2, "train": True},
    ]


def _ints(text):
    return [int(v) for v in text.split()]


def _text(values):
    return " ".join(str(v) for v in values)


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "rope", "rope", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    if op == "norm":
        T = rng.choice([1, 2, 3, 4, 4, 6, 8, 12, 16])
        quantum = 16 // ESIZE[dtype]
        Cp = _logint(rng, 1, 8192 // T)
        while (Cp * T) % quantum:
            Cp += 1
        if Cp * T > 8192:
            Cp = 8192 // T // quantum * quantum
        res, train = rng.random() < 0.5, rng.random() < 0.6
        tensors = 2 + 2 * res + (2 + res) * train
        N = _logint(rng, 1, max(1, min(401408, 280000000 // (tensors * ESIZE[dtype] * Cp * T))))
        return {"op": op, "dtype": dtype, "N": N, "Cp": Cp, "T": T, "res": res, "train": train}
    if op == "rope":
        T = rng.choice([1, 2, 4, 4, 8])
        Ch = 2 * _logint(rng, 2, 64 // T if T > 1 else 64)
        if T == 1:
            Ch = (Ch + 15) // 16 * 16
        while (Ch * T * ESIZE[dtype]) % 16:
            Ch += 2
        axes = rng.randint(1, 3)
        pairs = Ch // 2
        sections, left = [], pairs - (rng.randint(0, pairs // 4) if rng.random() < 0.3 else 0)
        for a in range(axes):
            n = left // (axes - a)
            sections.append(n)
            left -= n
        grid = [rng.randint(1, 16), rng.randint(1, 40), rng.randint(1, 40)]
        tokens = grid[0] * grid[1] * grid[2]
        room = 280000000 // (2 * ESIZE[dtype] * tokens * Ch * T)
        heads = rng.randint(1, max(1, min(32, room)))
        return {"op": op, "dtype": dtype, "docs": _logint(rng, 1, max(1, min(64, room // heads))), "grid": _text(grid),
                "heads": heads, "extra": rng.randint(0, 16), "Ch": Ch, "T": T, "sections": _text(sections),
                "inverse": rng.random() < 0.5, "far": rng.choice([0, 0, 1000, 1000000])}
    kv = rng.choice([1, 2, 3, 4, 6])
    heads = kv * rng.choice([1, 1, 2, 3])
    D = 8 * rng.randint(1, 16) if rng.random() < 0.4 else rng.choice([32, 64, 64, 64, 128])
    case = {"op": op, "dtype": dtype, "heads": heads, "kv": kv, "D": D, "cap": rng.choice([0.0, 0.0, 20.0, 50.0]),
            "bias": rng.choice([0, 1, 2, 3]), "train": rng.random() < 0.6}
    top = 6.0e10 if dtype != "f32" else 3.0e9          # heads * D * sum of squared lengths
    if rng.random() < 0.5:
        longest = min(8192, math.sqrt(top / (heads * D)))
        case["len"] = _logint(rng, 1, int(longest))
        room = min(top / (heads * D * case["len"] ** 2), 7.0e7 / (heads * D * ESIZE[dtype]) / 4 / case["len"])
        case["docs"] = _logint(rng, 1, max(1, min(4096, int(room))))
    else:
        n = rng.randint(1, 24)
        longest = min(4096, math.sqrt(top / (heads * D * n)))
        lens = [0 if rng.random() < 0.06 else _logint(rng, 1, int(longest)) for _ in range(n)]
        if sum(lens) == 0:
            lens[0] = 1
        case["lens"] = _text(lens)
        case["lead"] = rng.choice([0, 0, 5])
        case["tail"] = rng.choice([0, rng.randint(1, 200)])
    return case


# ------------------------------------------------------------------ inputs

def _tokens(case):
    """(documents' bounds on the host, tokens in all)"""
    if "docs" in case:
        n, L = case["docs"], case["len"]
        return [i * L for i in range(n + 1)], n * L
    bounds = [case["lead"]]
    for n in _ints(case["lens"]):
        bounds.append(bounds[-1] + n)
    return bounds, bounds[-1] + case["tail"]


def _grid_positions(n, axes, device):
    """Positions of n patches in reading order on a grid about as wide as high (and 16 frames deep)."""
    i = torch.arange(n, device=device)
    if axes == 1:
        return i[:, None].float()
    frames = 1 if axes == 2 else min(16, n)
    per = max(1, -(-n // frames))
    side = max(1, math.isqrt(per))
    p = [i % per // side, i % per % side]
    if axes == 3:
        p = [i // per] + p
    return torch.stack(p, 1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dt)

    st = {"case": case, "dtype": dt}
    if case["op"] == "norm":
        N, Cp, T = case["N"], case["Cp"], case["T"]
        F = Cp * T
        # a residual stream: channels with their own offsets and spreads
        off = torch.randn(F, generator=g, device=dev)
        spread = 0.5 + torch.rand(F, generator=g, device=dev)
        st["x"] = (torch.randn((N, F), generator=g, device=dev) * spread + off).to(dt)
        st["res"] = normal(N, F, std=0.5) if case["res"] else None
        st["w"] = normal(Cp, std=0.2, mean=1.0)
        st["b"] = normal(Cp, std=0.2)
        st["y"] = torch.empty_like(st["x"])
        st["xsum"] = torch.empty_like(st["x"]) if case["res"] else None
        st["mean"] = torch.empty(N, device=dev)
        st["rstd"] = torch.empty(N, device=dev)
        if case["train"]:
            st["gy"] = normal(N, F)
            st["gsum"] = normal(N, F) if case["res"] else None
            st["dx"] = torch.empty_like(st["x"])
            st["dw"] = torch.empty(Cp, device=dev)
            st["db"] = torch.empty(Cp, device=dev)
            if own:
                from group_circulant_linear_b200 import eqlin
                st["ws"] = eqlin.norm_workspace(T, Cp, N, device=dev)
    elif case["op"] == "rope":
        Ch, T, axes = case["Ch"], case["T"], len(_ints(case["sections"]))
        t, h, w = _ints(case["grid"])
        one = torch.stack(torch.meshgrid(torch.arange(t, device=dev), torch.arange(h, device=dev),
                                         torch.arange(w, device=dev), indexing="ij"), -1).reshape(-1, 3)
        pos = one[:, 3 - axes:].float().repeat(case["docs"], 1)
        st["pos"] = (pos + case["far"]).contiguous()
        N = st["pos"].shape[0]
        # queries and keys lie in front of the values in one packed row
        st["qkv"] = normal(N, case["heads"] + case["extra"], Ch * T)
        st["src"] = st["qkv"][:, :case["heads"]]
        st["dst"] = torch.empty((N, case["heads"], Ch * T), device=dev, dtype=dt)
        if own:
            from group_circulant_linear_b200 import eqlin
            st["plan"] = eqlin.Rope(T, Ch, _ints(case["sections"]), base=100.0)
    else:
        H, K, D = case["heads"], case["kv"], case["D"]
        bounds, N = _tokens(case)
        st["bounds"] = bounds
        # queries, keys and values of one packed projection; scores spread over several units
        qkv = torch.randn((N, H + 2 * K, D), generator=g, device=dev)
        qkv[:, :H] *= 2.0
        st["qkv"] = qkv.to(dt)
        st["q"], st["k"], st["v"] = st["qkv"][:, :H], st["qkv"][:, H:H + K], st["qkv"][:, H + K:]
        st["offsets"] = None if "docs" in case else torch.tensor(bounds, dtype=torch.int32, device=dev)
        st["pos"] = st["slopes"] = None
        if case["bias"]:
            if "docs" in case:
                p = _grid_positions(case["len"], case["bias"], dev).repeat(case["docs"], 1)
            else:
                p = torch.cat([torch.zeros(case["lead"], case["bias"], device=dev)]
                              + [_grid_positions(n, case["bias"], dev) for n in _ints(case["lens"])]
                              + [torch.zeros(case["tail"], case["bias"], device=dev)])
            st["pos"] = p.contiguous()
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device=dev)
        st["o"] = torch.empty((N, H, D), device=dev, dtype=dt)
        st["lse"] = torch.empty((H, N), device=dev)
        if case["train"]:
            st["go"] = normal(N, H, D)
            st["dqkv"] = torch.empty_like(st["qkv"])
            st["delta"] = torch.empty((H, N), device=dev)
    return st


# -------------------------------------------------------------- plain forms

def _plain_norm(st):
    c, dt = st["case"], st["dtype"]
    T, Cp, N = c["T"], c["Cp"], c["N"]
    s = st["x"].float()
    if c["res"]:
        s = s + st["res"].float()
    w = st["w"].float().repeat_interleave(T)
    b = st["b"].float().repeat_interleave(T)
    mean = s.mean(1)
    d = s - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
    xh = d * rstd[:, None]
    out = {"y": (xh * w + b).to(dt), "mean": mean, "rstd": rstd}
    if c["res"]:
        out["xsum"] = s.to(dt)
    if c["train"]:
        gy = st["gy"].float()
        gw = gy * w
        dx = rstd[:, None] * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
        if c["res"]:
            dx = dx + st["gsum"].float()
        out["dx"] = dx.to(dt)
        out["dw"] = (gy * xh).sum(0).view(Cp, T).sum(1)
        out["db"] = gy.sum(0).view(Cp, T).sum(1)
    return out


def _plain_rope(st):
    c, dt = st["case"], st["dtype"]
    Ch, T = c["Ch"], c["T"]
    half = Ch // 2
    x = st["src"].float().reshape(-1, c["heads"], Ch, T)
    angle = torch.zeros((x.shape[0], half), dtype=torch.float64, device=x.device)
    i = 0
    for a, n in enumerate(_ints(c["sections"])):
        f = 100.0 ** (-torch.arange(n, dtype=torch.float64, device=x.device) / n)
        angle[:, i:i + n] = st["pos"][:, a, None].double() * f
        i += n
    if c["inverse"]:
        angle = -angle
    cos = torch.cos(angle).float()[:, None, :, None]
    sin = torch.sin(angle).float()[:, None, :, None]
    x1, x2 = x[:, :, :half], x[:, :, half:]
    y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], 2)
    return y.reshape(-1, c["heads"], Ch * T).to(dt)


def _plain_scores(q, k, p, slopes, cap, scale):
    """q, k [docs, heads, L, D], p [docs, L, axes]: the scores, and 1 - tanh^2 where they are capped."""
    u = (q @ k.transpose(2, 3)) * scale
    slope = None
    if cap > 0:
        t = torch.tanh(u / cap)
        u = cap * t
        slope = 1.0 - t * t
    if p is not None:
        dist = (p[:, :, None, :] - p[:, None, :, :]).abs().sum(3)
        u = u - slopes[None, :, None, None] * dist[:, None]
    return u, slope


def _plain_attn_docs(st, lo, n, L, h0, h1, out):
    """Documents [lo, lo + n*L) of L tokens, query heads h0 to h1 (which share no key head with others)."""
    c = st["case"]
    H, K, D = c["heads"], c["kv"], c["D"]
    rep = H // K
    k0, k1 = h0 // rep, -(-h1 // rep)
    rows = slice(lo, lo + n * L)

    def heads(a, b0, b1):
        return a[rows, b0:b1].float().reshape(n, L, b1 - b0, D).transpose(1, 2)

    q = heads(st["q"], h0, h1)
    k = heads(st["k"], k0, k1).repeat_interleave(rep, 1)
    v = heads(st["v"], k0, k1).repeat_interleave(rep, 1)
    p = None if st["pos"] is None else st["pos"][rows].view(n, L, -1)
    slopes = None if p is None else st["slopes"][h0:h1]
    scale = D ** -0.5
    s, slope = _plain_scores(q, k, p, slopes, c["cap"], scale)
    top = s.amax(3, keepdim=True)
    e = torch.exp(s - top)
    z = e.sum(3, keepdim=True)
    prob = e / z
    o = prob @ v
    out["o"][rows, h0:h1] = o.transpose(1, 2).reshape(n * L, h1 - h0, D).to(st["dtype"])
    out["lse"][h0:h1, rows] = (top + torch.log(z))[..., 0].transpose(0, 1).reshape(h1 - h0, n * L)
    if c["train"]:
        go = heads(st["go"], h0, h1)
        dp = go @ v.transpose(2, 3)
        ds = prob * (dp - (go * o).sum(3, keepdim=True))
        if slope is not None:
            ds = ds * slope
        ds = ds * scale

        def put(at, grad, shared):
            if shared:
                grad = grad.reshape(n, k1 - k0, rep, L, D).sum(2)
            out["dqkv"][rows, at:at + grad.shape[1]] = grad.transpose(1, 2).reshape(n * L, -1, D).to(st["dtype"])

        put(h0, ds @ k, False)
        put(H + k0, ds.transpose(2, 3) @ q, True)
        put(H + K + k0, prob.transpose(2, 3) @ go, True)


def _plain_attn(st):
    c = st["case"]
    out = {"o": torch.zeros_like(st["o"]), "lse": torch.zeros_like(st["lse"])}
    if c["train"]:
        out["dqkv"] = torch.zeros_like(st["dqkv"])
    bounds, H = st["bounds"], c["heads"]
    rep = H // c["kv"]
    groups = [(bounds[0], c["docs"], c["len"])] if "docs" in c else \
        [(a, 1, b - a) for a, b in zip(bounds, bounds[1:]) if b > a]
    for lo, n, L in groups:
        step = H if n * H * L * L <= 2 ** 28 else rep       # all heads at once unless the scores are large
        for h0 in range(0, H, step):
            _plain_attn_docs(st, lo, n, L, h0, h0 + step, out)
    return out


# -------------------------------------------------------- the library's calls

def _own_norm(st):
    from group_circulant_linear_b200 import eqlin
    c = st["case"]
    eqlin.norm_forward(st["x"], st["w"], st["b"], st["y"], st["mean"], st["rstd"], c["T"], eps=EPS,
                       res=st["res"], xsum=st["xsum"])
    out = {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
    if c["res"]:
        out["xsum"] = st["xsum"]
    if c["train"]:
        eqlin.norm_backward(st["gy"], st["x"], st["w"], st["mean"], st["rstd"], st["dx"], st["dw"], st["db"], c["T"],
                            gsum=st["gsum"], res=st["res"], workspace=st["ws"])
        out.update(dx=st["dx"], dw=st["dw"], db=st["db"])
    return out


def _own_rope(st):
    from group_circulant_linear_b200 import eqlin
    eqlin.rope(st["plan"], st["pos"], st["src"], st["dst"], inverse=st["case"]["inverse"])
    return st["dst"]


def _own_attn(st):
    from group_circulant_linear_b200 import eqlin
    c = st["case"]
    if "docs" in c:
        kw = {"docs": c["docs"]}
    else:
        kw = {"offsets": st["offsets"], "max_len": max(_ints(c["lens"]))}
    kw.update(cap=c["cap"], pos=st["pos"], slopes=st["slopes"])
    eqlin.attention_forward(st["q"], st["k"], st["v"], st["o"], st["lse"], **kw)
    out = {"o": st["o"], "lse": st["lse"]}
    if c["train"]:
        H, K = c["heads"], c["kv"]
        d = st["dqkv"]
        eqlin.attention_backward(st["go"], st["q"], st["k"], st["v"], st["o"], st["lse"],
                                 d[:, :H], d[:, H:H + K], d[:, H + K:], st["delta"], **kw)
        out["dqkv"] = d
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "rope": _own_rope, "attn": _own_attn}[op](state)
    return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[op](state)


# --------------------------------------------------------------------- work

def work(case):
    e = ESIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["N"] * case["Cp"] * case["T"]
        tensors = 2 + (2 if case["res"] else 0)
        flops = 8 * n
        if case["train"]:
            tensors += 2 + (1 if case["res"] else 0)      # gy and dx, gsum; the rows are read already
            flops += 14 * n
        small = 8 * case["N"] + 2 * case["Cp"] * e + (8 * case["Cp"] if case["train"] else 0)
        return {"bytes": tensors * n * e + small, "flops": flops}
    if case["op"] == "rope":
        t, h, w = _ints(case["grid"])
        axes = len(_ints(case["sections"]))
        tokens = case["docs"] * t * h * w
        n = tokens * case["heads"] * case["Ch"] * case["T"]
        return {"bytes": 2 * n * e + 4 * tokens * axes, "flops": 3 * n}
    bounds, N = _tokens(case)
    sq = sum((b - a) ** 2 for a, b in zip(bounds, bounds[1:]))
    H, K, D = case["heads"], case["kv"], case["D"]
    flops = 4 * D * H * sq
    tensors = N * D * (2 * H + 2 * K)                       # q, o, k, v
    small = 4 * H * N + (4 * N * case["bias"])
    if case["train"]:
        flops += 10 * D * H * sq
        tensors += N * D * (2 * H + 2 * K)                  # go, dq, dk, dv
    return {"bytes": tensors * e + small, "flops": flops}


# -------------------------------------------------------------------- exact

def _exact_norm(st):
    c = st["case"]
    T = c["T"]
    x = st["x"].double()
    if c["res"]:
        x = x + st["res"].double()
    x = x.view(c["N"], c["Cp"], T).requires_grad_(c["train"])
    w = st["w"].double().requires_grad_(c["train"])
    b = st["b"].double().requires_grad_(c["train"])
    with torch.set_grad_enabled(c["train"]):
        var, mean = torch.var_mean(x, dim=(1, 2), correction=0)
        rstd = (var + EPS) ** -0.5
        y = (x - mean[:, None, None]) * rstd[:, None, None] * w[:, None] + b[:, None]
    out = {"y": y.detach().reshape(c["N"], -1), "mean": mean.detach(), "rstd": rstd.detach()}
    if c["res"]:
        out["xsum"] = x.detach().reshape(c["N"], -1)
    if c["train"]:
        dx, dw, db = torch.autograd.grad(y, (x, w, b), st["gy"].double().view_as(y))
        dx = dx.reshape(c["N"], -1)
        out.update(dx=dx + st["gsum"].double() if c["res"] else dx, dw=dw, db=db)
    return out


def _exact_rope(st):
    c = st["case"]
    half = c["Ch"] // 2
    x = st["src"].double().reshape(-1, c["heads"], 2, half, c["T"])
    z = torch.complex(x[:, :, 0], x[:, :, 1])
    phase = []
    for a, n in enumerate(_ints(c["sections"])):
        for j in range(n):
            phase.append(st["pos"][:, a].double() * math.exp(-math.log(100.0) * j / n))
    while len(phase) < half:
        phase.append(torch.zeros_like(phase[0]) if phase else st["pos"][:, 0].double() * 0)
    turn = torch.polar(torch.ones((z.shape[0], half), dtype=torch.float64, device=z.device), torch.stack(phase, 1))
    if c["inverse"]:
        turn = turn.conj()
    z = z * turn[:, None, :, None]
    return torch.stack([z.real, z.imag], 2).reshape(-1, c["heads"], c["Ch"] * c["T"])


def _exact_attn(st):
    c = st["case"]
    H, K, D = c["heads"], c["kv"], c["D"]
    N = st["q"].shape[0]
    f64 = dict(dtype=torch.float64, device=st["q"].device)
    o, lse = torch.zeros((N, H, D), **f64), torch.zeros((H, N), **f64)
    d = torch.zeros((N, H + 2 * K, D), **f64) if c["train"] else None
    bounds = st["bounds"]
    if "docs" in c:
        blocks = [(bounds[0], c["docs"], c["len"])]
    else:
        blocks = [(a, 1, b - a) for a, b in zip(bounds, bounds[1:]) if b > a]
    for lo, n, L in blocks:
        per = max(1, 2 ** 27 // (L * L))
        for at in range(0, n, per):
            m = min(per, n - at)
            r = slice(lo + at * L, lo + (at + m) * L)
            pos = None if st["pos"] is None else st["pos"][r].double().view(m, L, -1)
            far = None if pos is None else torch.cdist(pos, pos, p=1.0)
            for h in range(H):
                kh = h // (H // K)
                one = [st["q"][r, h], st["k"][r, kh], st["v"][r, kh]]
                q, k, v = (a.double().view(m, L, D).requires_grad_(c["train"]) for a in one)
                with torch.set_grad_enabled(c["train"]):
                    s = torch.einsum("bid,bjd->bij", q, k) / math.sqrt(D)
                    if c["cap"]:
                        s = torch.tanh(s / c["cap"]) * c["cap"]
                    if far is not None:
                        s = s - far * st["slopes"][h].double()
                    norm = torch.logsumexp(s, 2)
                    y = torch.einsum("bij,bjd->bid", torch.exp(s - norm[..., None]), v)
                o[r, h] = y.detach().reshape(m * L, D)
                lse[h, r] = norm.detach().reshape(m * L)
                if c["train"]:
                    gq, gk, gv = torch.autograd.grad(y, (q, k, v), st["go"][r, h].double().view(m, L, D))
                    d[r, h] += gq.reshape(m * L, D)
                    d[r, H + kh] += gk.reshape(m * L, D)
                    d[r, H + K + kh] += gv.reshape(m * L, D)
    out = {"o": o, "lse": lse}
    if c["train"]:
        out["dqkv"] = d
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attn":
        docs = case.get("docs", len(case.get("lens", "").split()))
        if case["heads"] * docs > 200000:
            return None
    return {"norm": _exact_norm, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](st)
