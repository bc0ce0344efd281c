"""Group layer norm, multi-axis rotary positions and document attention.

Each kernel is compared with its definition in 64 bits.  Tolerances are sums
of what the arithmetic may lose, element by element: half a step of the
output's type (``u``), half a step for each operand that the tensor cores take
in 16 bits (the probabilities P and the score gradients), and FP32 roundings
along the longest chain of additions (2^-24 each) on the sums of absolute
values.  They were fixed before the kernels first ran, and narrowed twice with
them since: where the norm's backward and the attention's no longer read a sum
or an output as stored (x + res, and o for delta).
"""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from group_circulant_linear_b200 import eqlin

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
W = 2.0 ** -24


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    # half the spacing of the type's subnormals
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def check(got, ref, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - tol
    worst = over.argmax() if over.numel() else 0
    assert not over.numel() or float(over.max()) <= 0, \
        f"{what}: {float(got.flatten()[worst])} for {float(ref.flatten()[worst])}, tolerance {float(tol.flatten()[worst])}"


# ------------------------------------------------------------------- norm

def norm_bounds(x, res, w, b, gy, gs, T, eps, dt):
    """Values and tolerances of the norm and its gradients, in 64 bits."""
    s = x.double() + (res.double() if res is not None else 0)
    N, F = s.shape
    u, z = half_step(dt), tiny(dt)
    wf, bf = w.double().repeat_interleave(T), b.double().repeat_interleave(T)
    mean = s.mean(1, keepdim=True)
    var = ((s - mean) ** 2).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    xh = (s - mean) * rstd
    mag = (s.abs() + s.abs().mean(1, keepdim=True)) * rstd       # what the FP32 roundings of xh scale with
    # longest chain: 32 terms in a thread, 5 shuffles, 16 warps, and a dozen elementwise steps
    c = 96 * W
    out = {"y": (xh * wf + bf, u * (xh * wf + bf).abs() + z + c * (mag * wf.abs() + bf.abs())),
           "mean": (mean[:, 0], c * s.abs().mean(1)),
           "rstd": (rstd[:, 0], c * rstd[:, 0] * (1 + (mag ** 2).mean(1) * W * 96))}
    if res is not None:
        out["xsum"] = (s, u * s.abs() + z)
    if gy is not None:
        exh = c * mag                                              # error of xh
        g = gy.double()
        gw = g * wf
        m1, m2 = gw.mean(1, keepdim=True), (gw * xh).mean(1, keepdim=True)
        dx = rstd * (gw - m1 - xh * m2)
        edx = rstd * (c * (gw.abs() + gw.abs().mean(1, keepdim=True) + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))
                      + exh * m2.abs() + xh.abs() * (gw.abs() * exh).mean(1, keepdim=True))
        if gs is not None:
            dx = dx + gs.double()
        out["dx"] = (dx, u * dx.abs() + z + edx + 2 * W * dx.abs())
        C = F // T
        terms = N * T + 64                                         # at most: every term in one chain
        dw = (g * xh).sum(0).view(C, T).sum(1)
        out["dw"] = (dw, ((g * xh).abs().sum(0).view(C, T).sum(1) * terms * W
                          + (g.abs() * exh).sum(0).view(C, T).sum(1)))
        out["db"] = (g.sum(0).view(C, T).sum(1), g.abs().sum(0).view(C, T).sum(1) * terms * W)
    return out


NORM_SHAPES = [  # N, C', T: lanes per row 1 .. 32, blocks per row, odd orders, one row, more rows than threads
    (1, 96, 4), (197, 96, 4), (5, 2, 4), (33, 24, 4), (1000, 24, 4), (77, 192, 4), (3, 16, 1), (64, 40, 3), (19, 8, 12),
    (7, 100, 2), (50, 128, 8), (9, 1024, 8), (4, 2048, 1), (2, 683 * 8, 1), (3, 512, 16), (300, 65, 8), (2500, 8, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("with_res", [False, True])
@pytest.mark.parametrize("N,Cp,T", NORM_SHAPES)
def test_norm(N, Cp, T, with_res, dtype):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(N * 31 + Cp)
    F = Cp * T

    def rnd(*s, std=1.0, mean=0.0):
        return (torch.randn(s, generator=g) * std + mean).to(dt)

    x = rnd(N, F, std=0.7, mean=3.0)
    res = rnd(N, F) if with_res else None
    w, b, gy = rnd(Cp, std=0.3, mean=1.0), rnd(Cp), rnd(N, F)
    gs = rnd(N, F) if with_res else None
    ref = norm_bounds(x, res, w, b, gy, gs, T, 1e-6, dt)
    d = {k: v.cuda() for k, v in dict(x=x, w=w, b=b, gy=gy).items()}
    guard = 7.0
    y = torch.full((N + 2, F), guard, dtype=dt, device="cuda")
    dx = torch.full((N + 2, F), guard, dtype=dt, device="cuda")
    mean, rstd = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    xsum = torch.empty((N, F), dtype=dt, device="cuda") if with_res else None
    dw, db = torch.empty(Cp, device="cuda"), torch.empty(Cp, device="cuda")
    eqlin.norm_forward(d["x"], d["w"], d["b"], y[1:-1], mean, rstd, T, res=None if res is None else res.cuda(), xsum=xsum)
    eqlin.norm_backward(d["gy"], d["x"], d["w"], mean, rstd, dx[1:-1], dw, db, T, gsum=None if gs is None else gs.cuda(),
                        res=None if res is None else res.cuda())
    torch.cuda.synchronize()
    got = {"y": y[1:-1], "mean": mean, "rstd": rstd, "dx": dx[1:-1], "dw": dw, "db": db}
    if with_res:
        got["xsum"] = xsum
    for k, (r, tol) in ref.items():
        check(got[k], r, tol, k)
    for t in (y, dx):                     # rows around the outputs stay as they were
        assert (t[0] == guard).all() and (t[-1] == guard).all()


@pytest.mark.gpu
def test_norm_in_place_empty_and_repeatable():
    dt = torch.bfloat16
    N, Cp, T = 700, 48, 4
    g = torch.Generator().manual_seed(5)
    x, r, gy = (torch.randn((N, Cp * T), generator=g).to(dt).cuda() for _ in range(3))
    w, b = torch.ones(Cp, dtype=dt, device="cuda"), torch.zeros(Cp, dtype=dt, device="cuda")
    mean, rstd = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    y, s = torch.empty_like(x), torch.empty_like(x)
    eqlin.norm_forward(x, w, b, y, mean, rstd, T, res=r, xsum=s)
    y2, s2 = torch.empty_like(x), x.clone()
    eqlin.norm_forward(s2, w, b, y2, mean, rstd, T, res=r, xsum=s2)      # the stream updated in place
    assert torch.equal(y, y2) and torch.equal(s, s2)
    outs = []
    for inplace in (False, True, False):
        dw, db = torch.empty(Cp, device="cuda"), torch.empty(Cp, device="cuda")
        gin = gy.clone()
        dx = gin if inplace else torch.empty_like(gy)
        eqlin.norm_backward(gin, s, w, mean, rstd, dx, dw, db, T)
        outs.append((dx, dw, db))
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(outs[0], o))
    e = torch.empty((0, Cp * T), dtype=dt, device="cuda")
    dw, db = torch.ones(Cp, device="cuda"), torch.ones(Cp, device="cuda")
    z = torch.empty(0, device="cuda")
    eqlin.norm_forward(e, w, b, e, z, z, T)
    eqlin.norm_backward(e, e, w, z, z, e, dw, db, T)
    assert not dw.any() and not db.any()


# ------------------------------------------------------------------- rope

def rope_ref(x, pos, r, inverse):
    N, H, _ = x.shape
    half = r.Ch // 2
    xd = x.double().view(N, H, 2, half, r.T)
    ang = torch.zeros(N, half, dtype=torch.float64)
    live = torch.zeros(half, dtype=torch.bool)
    i = 0
    for a, n in enumerate(r.sections):
        for k in range(n):
            ang[:, i] = pos[:, a].double() * r.freqs[i]
            live[i] = True
            i += 1
    if inverse:
        ang = -ang
    c, s = ang.cos()[:, None, :, None], ang.sin()[:, None, :, None]
    x1, x2 = xd[:, :, 0], xd[:, :, 1]
    return torch.stack([x1 * c - x2 * s, x2 * c + x1 * s], 2).view(N, H, -1), ang, live


ROPE_SHAPES = [  # N, heads, Ch, T, sections
    (1, 1, 16, 4, (4, 4)), (197, 12, 16, 4, (4, 4)), (50, 5, 16, 4, (2, 3, 3)), (33, 3, 10, 4, (2, 3)), (9, 2, 2, 1, (1,)),
    (20, 7, 64, 1, (10, 11, 11)), (20, 1, 6, 2, (1, 0, 2)), (15, 4, 18, 3, (4, 4)), (8, 2, 256, 1, (128,)), (3, 9, 12, 8, (2, 1)),
    (70, 33, 8, 2, (4,)), (5, 2, 4, 16, (1, 1)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("far", [0.0, 1.0e6])
@pytest.mark.parametrize("N,H,Ch,T,sections", ROPE_SHAPES)
def test_rope(N, H, Ch, T, sections, far, dtype):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(N + H)
    r = eqlin.Rope(T, Ch, sections, base=100.0)
    D = Ch * T
    x = torch.randn((N, H, D), generator=g).to(dt)
    pos = torch.randint(0, 40, (N, len(sections)), generator=g).float() + far
    big = torch.full((N, (H + 2) * D), 5.0, dtype=dt, device="cuda")       # heads inside a wider row
    big[:, D:(H + 1) * D] = x.view(N, -1).cuda()
    src = big[:, D:(H + 1) * D].view(N, H, D)
    u = half_step(dt)
    for inverse in (False, True):
        want, ang, live = rope_ref(x, pos, r, inverse)
        dst = torch.empty((N, H, D), dtype=dt, device="cuda")
        eqlin.rope(r, pos.cuda(), src, dst, inverse=inverse)
        # the angle: 2^-23 turns plus the 2^-48 of the frequency's two parts; sincospi 2^-22; three FP32 steps
        x1, x2 = x.double().view(N, H, 2, -1).unbind(2)
        mag = (x1.abs() + x2.abs()).repeat(1, 1, 2)
        tol = u * want.abs() + tiny(dt) + mag * (2 * math.pi * (2.0 ** -23 + ang.abs().max() * 2.0 ** -48) + 2.0 ** -22 + 3 * W)
        check(dst, want, tol, f"rope inverse={inverse}")
        # pairs of no axis are copied bit for bit
        keep = (~live).repeat_interleave(T).repeat(2)
        assert torch.equal(dst.cpu()[..., keep], x[..., keep])
    eqlin.rope(r, pos.cuda(), src, src)                                    # in place
    dst = torch.empty((N, H, D), dtype=dt, device="cuda")
    eqlin.rope(r, pos.cuda(), x.cuda(), dst)
    assert torch.equal(src, dst)
    assert (big[:, :D] == 5.0).all() and (big[:, (H + 1) * D:] == 5.0).all()


@pytest.mark.gpu
def test_rope_unaligned_rows_and_group_shift():
    T, Ch, N, H = 4, 16, 21, 3
    r = eqlin.Rope(T, Ch, (4, 2))
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 14, (N, 2), generator=g).float().cuda()
    x = torch.randn((N, H, Ch * T), generator=g).to(torch.bfloat16).cuda()
    want = torch.empty_like(x)
    eqlin.rope(r, pos, x, want)
    for pad in (1, 2, 4):                                                  # 2-, 4- and 8-byte vectors
        row = torch.zeros((N, H * Ch * T + pad), dtype=x.dtype, device="cuda")
        v = row.as_strided((N, H, Ch * T), (row.shape[1], Ch * T, 1), pad)
        v.copy_(x)
        eqlin.rope(r, pos, v, v)
        assert torch.equal(v, want)
    rolled = x.view(N, H, Ch, T).roll(1, -1).reshape(N, H, -1).contiguous()
    out = torch.empty_like(x)
    eqlin.rope(r, pos, rolled, out)
    assert torch.equal(out, want.view(N, H, Ch, T).roll(1, -1).reshape(N, H, -1))


# -------------------------------------------------------------- attention

def attention_bounds(q, k, v, go, lens, lead, cap, pos, slopes, scale, dt, p16):
    """o, lse, dq, dk, dv in 64 bits with their tolerances; p16: P and the
    score gradients pass through 16 bits on their way into a product."""
    N, H, D = q.shape
    K = k.shape[1]
    u, z = half_step(dt), tiny(dt)
    # P in (0, 1] and du as 16-bit operands: half a step each, plus what falls below the type's smallest step
    up = u if p16 else 0.0
    zp = tiny(dt) if p16 else 0.0
    f64 = dict(dtype=torch.float64)
    val = {n: torch.zeros(s, **f64) for n, s in dict(o=q.shape, lse=(H, N), dq=q.shape, dk=k.shape, dv=k.shape).items()}
    tol = {n: torch.zeros_like(t) for n, t in val.items()}
    lo = lead
    for n in lens:
        r = slice(lo, lo + n)
        lo += n
        if n == 0:
            continue
        for h in range(H):
            kh = h // (H // K)
            Q, Kh, V, G = q[r, h].double(), k[r, kh].double(), v[r, kh].double(), go[r, h].double()
            uu = scale * Q @ Kh.T
            mag = scale * Q.abs() @ Kh.abs().T
            t = torch.tanh(uu / cap) if cap else torch.zeros_like(uu)
            s = cap * t if cap else uu
            slope = 1 - t * t
            bias = torch.zeros_like(s)
            if pos is not None:
                P_ = pos[r].double()
                bias = slopes[h].double() * (P_[:, None] - P_[None]).abs().sum(2)
            s = s - bias
            lse = torch.logsumexp(s, 1)
            P = torch.exp(s - lse[:, None])
            # relative error of P: D + 2 products' roundings in the score, a dozen on the score itself
            # (cap, bias, its scale to base 2), the exponential's 2^-21, and as much again in lse
            e1 = ((D + 4) * W * mag + 12 * W * (s.abs() + bias.abs() + cap) + 2.0 ** -21).max(1, keepdim=True).values
            eta = 2 * e1 + n * W
            o = P @ V
            aPV = P @ V.abs()
            eo = (up + eta) * aPV + zp * V.abs().sum(0) + n * W * aPV
            val["o"][r, h], tol["o"][r, h] = o, u * o.abs() + z + eo
            val["lse"][h, r], tol["lse"][h, r] = lse, e1[:, 0] + n * W + 4 * W * lse.abs()
            dP = G @ V.T
            delta = (G * o).sum(1, keepdim=True)
            du = P * (dP - delta) * slope
            edp = D * W * G.abs() @ V.abs().T
            # delta: the FP32 sum of P dP; and in dq the correction by eps = delta - do.o as stored, whose
            # product passes through 16 bits
            eps = (G.abs() * tol["o"][r, h]).sum(1, keepdim=True) + D * W * (G * o).abs().sum(1, keepdim=True)
            edelta = (eta * P * dP.abs() + P * edp + (n + 8) * W * P * (dP.abs() + delta.abs())).sum(1, keepdim=True) \
                + (up + eta + n * W) * eps
            if not p16:
                edelta = edelta + eps                              # the CUDA-core kernel takes do.o itself
            # 1 - tanh^2 to a few 2^-24 absolute, and its argument's error
            eslope = (8 * W + 2 * (D + 4) * W * mag / cap) if cap else torch.zeros_like(uu)
            edu = P * slope * (eta * (dP - delta).abs() + edelta + edp + 4 * W * (dP.abs() + delta.abs())) \
                + P * (dP - delta).abs() * eslope
            edu = edu + up * (du.abs() + edu) + zp
            steps = (n * (H // K) + 64) * W
            dq = scale * du @ Kh
            val["dq"][r, h] = dq
            tol["dq"][r, h] = u * dq.abs() + z + scale * (edu @ Kh.abs() + steps * du.abs() @ Kh.abs())
            val["dk"][r, kh] += scale * du.T @ Q
            tol["dk"][r, kh] += scale * (edu.T @ Q.abs() + (steps + W) * du.abs().T @ Q.abs())
            val["dv"][r, kh] += P.T @ G
            tol["dv"][r, kh] += ((up + eta) * P).T @ G.abs() + zp * G.abs().sum(0) + steps * P.T @ G.abs()
        tol["dk"][r] += u * val["dk"][r].abs() + z
        tol["dv"][r] += u * val["dv"][r].abs() + z
    return val, tol


def run_attention(lens, lead, tail, H, K, D, cap, axes, dtype, seed=0, uniform=False, packed=True, scale=None,
                  q_std=2.0, poison=True, max_len="max", slope=0.3):
    dt = DT[dtype]
    g = torch.Generator().manual_seed(seed)
    N = lead + sum(lens) + tail
    qkv = torch.randn((N, H + 2 * K, D), generator=g)
    qkv[:, :H] *= q_std
    qkv = qkv.to(dt)
    go = torch.randn((N, H, D), generator=g).to(dt)
    pos = torch.randint(0, 30, (N, axes), generator=g).float() if axes else None
    slopes = torch.rand(H, generator=g) * slope if axes else None
    scale = D ** -0.5 if scale is None else scale
    val, tol = attention_bounds(qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:], go, lens, lead, cap, pos, slopes, scale, dt,
                                dtype != "f32")
    inside = torch.zeros(N, dtype=torch.bool)
    inside[lead:lead + sum(lens)] = True
    dev = qkv.cuda()
    gdev = go.cuda()
    if poison:                            # what lies outside the documents is not looked at
        dev[~inside.cuda()] = float("nan")
        gdev[~inside.cuda()] = float("inf")
    q, k, v = dev[:, :H], dev[:, H:H + K], dev[:, H + K:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    bounds = [lead]
    for n in lens:
        bounds.append(bounds[-1] + n)
    kw = dict(docs=len(lens)) if uniform else dict(offsets=torch.tensor(bounds, dtype=torch.int32, device="cuda"),
                                                   max_len=max(lens + [0]) if max_len == "max" else max_len)
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    kw.update(cap=cap, scale=scale, err=err, pos=None if pos is None else pos.cuda(),
              slopes=None if slopes is None else slopes.cuda())
    o = torch.full((N, H, D), 9.0, dtype=dt, device="cuda")
    lse = torch.full((H, N), 9.0, device="cuda")
    eqlin.attention_forward(q, k, v, o, lse, **kw)
    dqkv = torch.full((N, H + 2 * K, D), 9.0, dtype=dt, device="cuda")
    delta = torch.empty((H, N), device="cuda")
    eqlin.attention_backward(gdev, q, k, v, o, lse, dqkv[:, :H], dqkv[:, H:H + K], dqkv[:, H + K:], delta, **kw)
    torch.cuda.synchronize()
    assert not err.any()
    got = dict(o=o, lse=lse, dq=dqkv[:, :H], dk=dqkv[:, H:H + K], dv=dqkv[:, H + K:])
    for n in val:
        check(got[n], val[n], tol[n], n)
    for n in ("o", "dq", "dk", "dv"):
        assert not got[n].cpu()[~inside].any(), n
    assert not lse.cpu()[:, ~inside].any()
    return got


ATTN_CASES = [  # lens, lead, tail, H, K, D, cap, axes
    ([1], 0, 0, 1, 1, 64, 0.0, 0),
    ([197], 0, 0, 2, 2, 64, 30.0, 2),
    ([0, 5, 0], 3, 4, 2, 1, 64, 0.0, 1),
    ([64, 65, 63], 0, 0, 2, 2, 32, 0.0, 2),
    ([128, 129, 1, 257, 127], 5, 9, 2, 2, 64, 20.0, 3),
    ([49] * 6, 0, 0, 3, 3, 32, 0.0, 2),
    ([130, 31], 0, 1, 4, 2, 128, 50.0, 0),
    ([96, 200], 2, 0, 6, 2, 96, 0.0, 0),
    ([33, 16, 17, 15], 0, 0, 3, 1, 40, 0.0, 1),
    ([300], 0, 0, 2, 2, 8, 5.0, 0),
    ([257, 255], 1, 1, 2, 2, 104, 25.0, 2),
    ([513, 2, 640], 0, 70, 1, 1, 64, 0.0, 0),
    ([2, 3, 4] * 8, 0, 0, 1, 1, 24, 0.0, 0),
    ([385], 0, 0, 1, 1, 128, 0.0, 3),
    # many documents in a block's 128 tokens, runs of empty ones, whole blocks outside
    ([1] * 150 + [0] * 70 + [3] * 20 + [0] * 3 + [130, 0, 1], 140, 150, 2, 1, 64, 0.0, 1),
    ([0] * 40 + [127, 1, 128, 129], 128, 1, 1, 1, 32, 9.0, 0),
    # documents of 384 (768 with a cap or bias) tokens and more on average: the forward's wide form
    ([1100], 0, 0, 1, 1, 64, 20.0, 2),
    ([2177, 150], 3, 5, 1, 1, 32, 0.0, 3),
    ([1024 + 65], 0, 0, 2, 1, 56, 0.0, 0),
    ([1281], 0, 0, 1, 1, 64, 0.0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens,lead,tail,H,K,D,cap,axes", ATTN_CASES)
def test_attention(lens, lead, tail, H, K, D, cap, axes, dtype):
    run_attention(lens, lead, tail, H, K, D, cap, axes, dtype, seed=len(lens) + D)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_equal_documents_and_separate_tensors(D, dtype):
    a = run_attention([75] * 4, 0, 0, 2, 2, D, 0.0, 2, dtype, uniform=True)
    b = run_attention([75] * 4, 0, 0, 2, 2, D, 0.0, 2, dtype, uniform=False, packed=False)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_len", [None, 1, 100000])
def test_attention_results_do_not_depend_on_max_len(max_len, dtype):
    args = ([300, 7, 150], 2, 3, 2, 1, 64, 20.0, 2, dtype)
    a, b = run_attention(*args), run_attention(*args, max_len=max_len)
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,tail", [([], 9), ([], 200), ([0, 0, 0], 5)])
def test_attention_without_documents(lens, tail, dtype):
    run_attention(lens, 3, tail, 2, 2, 64, 0.0, 0, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cap", [0.0, 6.0])
def test_attention_documents_do_not_see_each_other(dtype, cap):
    # a document's results, bit for bit, whatever its neighbours in the same tiles hold
    dt = DT[dtype]
    lens, H, D = [37, 100, 70, 5], 2, 64
    N = sum(lens)
    off = torch.tensor([0, 37, 137, 207, 212], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(12)
    base = torch.randn((4, N, H, D), generator=g).to(dt).cuda()
    outs = []
    for fill in (None, float("nan"), float("inf"), 3.0e4):
        t = base.clone()
        if fill is not None:
            t[:, :37] = fill
            t[:, 137:] = fill
        q, k, v, go = t
        o, dq, dk, dv = (torch.empty_like(q) for _ in range(4))
        lse, delta = torch.empty((H, N), device="cuda"), torch.empty((H, N), device="cuda")
        eqlin.attention_forward(q, k, v, o, lse, offsets=off, cap=cap)
        eqlin.attention_backward(go, q, k, v, o, lse, dq, dk, dv, delta, offsets=off, cap=cap)
        outs.append([x[37:137].clone() for x in (o, dq, dk, dv)] + [lse[:, 37:137].clone()])
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))
    assert all(torch.isfinite(x).all() for x in outs[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("cap", [0.0, 8.0])
@pytest.mark.parametrize("slope,scale", [(-0.5, None), (0.0, 0.01), (4.0, 1.5)])
def test_attention_any_slopes_and_scales(slope, scale, cap, dtype):
    # a bias that grows with the distance, none at all, and one that leaves next to nothing
    run_attention([70, 33, 101], 1, 2, 2, 2, 64, cap, 2, dtype, slope=slope, scale=scale)
    run_attention([70, 33, 101], 1, 2, 2, 1, 128, cap, 3, dtype, slope=slope, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attention_large_scores(dtype):
    # scores of several hundred units: the running maximum moves far, capped and not
    run_attention([190, 300], 0, 0, 2, 2, 64, 0.0, 0, dtype, q_std=60.0, seed=4)
    run_attention([190, 300], 0, 0, 2, 2, 64, 30.0, 0, dtype, q_std=60.0, seed=4)
    run_attention([1150], 0, 0, 1, 1, 64, 30.0, 1, dtype, q_std=20.0, seed=4)   # some tiles near the cap, some not
    run_attention([1150], 0, 0, 1, 1, 64, 0.0, 0, dtype, q_std=60.0, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lead,rest,cap", [(1, 60, 0.0), (130, 90, 5.0), (300, 900, 0.0), (300, 900, 5.0)])
def test_attention_keys_infinitely_far_away(lead, rest, cap, dtype):
    # whole tiles of keys at an infinite distance come first: the others must not notice
    H, D, N = 2, 64, lead + rest
    dt = DT[dtype]
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn((N, H, D), generator=g).to(dt).cuda() for _ in range(3))
    pos = torch.randint(0, 20, (N, 2), generator=g).float().cuda()
    pos[:lead, 1] = math.inf
    slopes = torch.tensor([0.5, 0.125], device="cuda")
    o, lse = torch.empty_like(q), torch.empty((H, N), device="cuda")
    eqlin.attention_forward(q, k, v, o, lse, pos=pos, slopes=slopes, cap=cap)
    near = [t[lead:].contiguous() for t in (q, k, v)]
    o2, lse2 = torch.empty_like(near[0]), torch.empty((H, rest), device="cuda")
    eqlin.attention_forward(*near, o2, lse2, pos=pos[lead:].contiguous(), slopes=slopes, cap=cap)
    # either result: P and o rounded to the type, half a step each (f32: neither), sums of up to N
    # terms in another order, 2^-21 for each exponential and score
    half = 0.0 if dtype == "f32" else torch.finfo(dt).eps / 2
    tol = 2 * (2 * half + N * 2.0 ** -24 + 2.0 ** -20 * (8 + float(lse2.abs().max())))
    assert float((o[lead:].float() - o2.float()).abs().max()) <= tol * float(v.float().abs().max())
    assert float((lse[:, lead:] - lse2).abs().max()) <= 2 * (N * 2.0 ** -24 + 2.0 ** -20 * (8 + float(lse2.abs().max())))


@pytest.mark.gpu
@pytest.mark.parametrize("N", [700, 1200])
def test_attention_rising_scores(N):
    # keys ordered so that each tile's maximum is above the last one's
    H, D = 1, 64
    for dtype in ("bf16", "f32"):
        dt = DT[dtype]
        q = torch.full((N, H, D), 0.5)
        k = (torch.arange(N)[:, None, None] / 8.0).expand(N, H, D) / 4.0
        g = torch.Generator().manual_seed(1)
        v, go = torch.randn((N, H, D), generator=g), torch.randn((N, H, D), generator=g)
        q, k, v, go = (t.to(dt).contiguous() for t in (q, k, v, go))
        val, tol = attention_bounds(q, k, v, go, [N], 0, 0.0, None, None, 0.125, dt, dtype != "f32")
        o, lse = torch.empty((N, H, D), dtype=dt, device="cuda"), torch.empty((H, N), device="cuda")
        c = [t.cuda() for t in (q, k, v)]
        eqlin.attention_forward(*c, o, lse, scale=0.125)
        check(o, val["o"], tol["o"], "o")
        check(lse, val["lse"], tol["lse"], "lse")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_gradients_against_differences(dtype):
    # d(o . go) along a direction, by central differences of the 64-bit formula
    dt = DT[dtype]
    got = run_attention([40, 25], 0, 0, 2, 1, 32, 4.0, 2, dtype, seed=9)
    g = torch.Generator().manual_seed(9)
    N, H, K, D = 65, 2, 1, 32
    qkv = torch.randn((N, H + 2 * K, D), generator=g)
    qkv[:, :H] *= 2.0
    qkv = qkv.to(dt).double()
    go = torch.randn((N, H, D), generator=g).to(dt).double()
    pos = torch.randint(0, 30, (N, 2), generator=g).float()
    slopes = torch.rand(H, generator=g) * 0.3
    way = torch.randn(qkv.shape, generator=g, dtype=torch.float64)

    def f(step):
        x = qkv + step * way
        val, _ = attention_bounds(x[:, :H], x[:, H:H + K], x[:, H + K:], go, [40, 25], 0, 4.0, pos, slopes, D ** -0.5,
                                  dt, False)
        return float((val["o"] * go).sum())

    h = 1e-5
    want = (f(h) - f(-h)) / (2 * h)
    d = torch.cat([got["dq"], got["dk"], got["dv"]], 1).double().cpu()
    # each element is off by its tolerance at most; a direction of unit-variance steps adds them as their norm, 5 sigma
    _, tol = attention_bounds(qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:], go, [40, 25], 0, 4.0, pos, slopes, D ** -0.5,
                              dt, dtype != "f32")
    room = 5 * torch.cat([tol["dq"], tol["dk"], tol["dv"]], 1).norm() + 1e-6 * abs(want)
    assert abs(float((d * way).sum()) - want) <= float(room)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_repeats_bit_for_bit_and_in_a_graph(dtype):
    dt = DT[dtype]
    N, H, D = 400, 3, 64
    g = torch.Generator().manual_seed(2)
    q, k, v, go = (torch.randn((N, H, D), generator=g).to(dt).cuda() for _ in range(4))
    off = torch.tensor([0, 150, 390], dtype=torch.int32, device="cuda")

    def buffers():
        return [torch.empty_like(q) for _ in range(4)] + [torch.empty((H, N), device="cuda") for _ in range(2)]

    def both(o, dq, dk, dv, lse, delta):
        eqlin.attention_forward(q, k, v, o, lse, offsets=off)
        eqlin.attention_backward(go, q, k, v, o, lse, dq, dk, dv, delta, offsets=off)

    first, second, third = buffers(), buffers(), buffers()
    both(*first)
    both(*second)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        both(*third)
        with torch.cuda.graph(graph, stream=side):
            both(*third)
    torch.cuda.current_stream().wait_stream(side)
    for b in third:
        b.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        if a is first[5]:                 # delta outside the documents is not written
            a, b, c = a[:, :390], b[:, :390], c[:, :390]
        assert torch.equal(a, b) and torch.equal(a, c)


# ---------------------------------------------------------------- refusals

def test_norm_refusals():
    L = eqlin.lib()
    one = ctypes.c_void_p(4096)           # never followed: each call is refused first
    bf = eqlin.BF16

    def fwd(T=4, Cp=8, dt=bf, x=one, res=None, w=one, b=one, eps=1e-6, s=None, y=one, mean=one, rstd=one, N=3):
        return L.eqlin_norm_forward(T, Cp, dt, x, res, w, b, eps, s, y, mean, rstd, N, None)

    assert fwd(T=0) == -1 and fwd(Cp=0) == -1 and fwd(N=-1) == -1 and fwd(dt=9) == -1
    assert fwd(T=17) == -2 and fwd(Cp=4096) == -2 and fwd(Cp=2 ** 40) == -2
    assert fwd(T=1, Cp=7) == -3 and fwd(T=3, Cp=2, dt=eqlin.F32) == -3
    assert fwd(w=None) == -1 and fwd(b=None) == -1 and fwd(eps=-1.0) == -1 and fwd(eps=math.nan) == -1
    assert fwd(res=one) == -1 and fwd(s=one) == -1 and fwd(x=None) == -1 and fwd(y=None) == -1
    assert fwd(mean=None) == -1 and fwd(rstd=None) == -1 and fwd(x=ctypes.c_void_p(4104)) == -3
    assert fwd(N=0) == 0

    def bwd(T=4, Cp=8, dt=bf, gy=one, gs=None, x=one, res=None, w=one, mean=one, rstd=one, dx=one, dw=one, db=one, ws=one, N=3):
        return L.eqlin_norm_backward(T, Cp, dt, gy, gs, x, res, w, mean, rstd, dx, dw, db, ws, N, None)

    for name in ("gy", "x", "w", "mean", "rstd", "dx", "dw", "db", "ws"):
        assert bwd(**{name: None}) == -1, name
    for name in ("mean", "rstd", "dw", "db"):
        assert bwd(**{name: ctypes.c_void_p(4098)}) == -3, name
    for name in ("w", "b", "mean", "rstd"):
        assert fwd(**{name: ctypes.c_void_p(4097)}) == -3, name
    assert L.eqlin_norm_workspace_bytes(4, 2 ** 62, 2) == -1
    for name in ("gy", "gs", "x", "res", "dx", "ws"):
        assert bwd(**{name: ctypes.c_void_p(4100)}) == -3, name
    assert bwd(T=17) == -2 and bwd(Cp=3) == -3 and bwd(N=-2) == -1
    assert L.eqlin_norm_workspace_bytes(4, 8, 2) == 2 * 2 * 8 * 4
    assert L.eqlin_norm_workspace_bytes(4, 8, 10 ** 6) == L.eqlin_norm_workspace_bytes(4, 8, 10 ** 9)
    assert L.eqlin_norm_workspace_bytes(0, 8, 2) == -1 and L.eqlin_norm_workspace_bytes(4, 8, -2) == -1
    with pytest.raises(TypeError):
        eqlin.norm_forward(torch.zeros(2, 32), *[torch.zeros(8)] * 2, *[None] * 3, 4)


def test_rope_refusals():
    for bad in (dict(T=0, Ch=8, sections=(1,)), dict(T=4, Ch=7, sections=(1,)), dict(T=4, Ch=8, sections=(5,)),
                dict(T=4, Ch=8, sections=(1,), freqs=(math.inf,)), dict(T=17, Ch=8, sections=(1,)),
                dict(T=1, Ch=258, sections=(1,)), dict(T=1, Ch=16, sections=(1, 1, 1, 1, 1))):
        with pytest.raises(eqlin.EqlinError):
            eqlin.Rope(**bad)
    with pytest.raises(ValueError):
        eqlin.Rope(4, 8, ())
    with pytest.raises(ValueError):
        eqlin.Rope(4, 8, (-1, 2))
    with pytest.raises(ValueError):
        eqlin.Rope(4, 8, (2,), freqs=(1.0,))
    r = eqlin.Rope(4, 8, (2, 2))
    L = eqlin.lib()
    one = ctypes.c_void_p(4096)

    def call(r=r.ptr, dt=eqlin.BF16, pos=one, src=one, ss=64, dst=one, ds=64, heads=2, N=3):
        return L.eqlin_rope_apply(r, dt, pos, src, ss, dst, ds, heads, 0, N, None)

    assert call(r=None) == -1 and call(dt=5) == -1 and call(heads=0) == -1 and call(N=-1) == -1
    assert call(ss=63) == -1 and call(ds=63) == -1 and call(pos=None) == -1 and call(src=None) == -1
    assert call(dst=None) == -1 and call(src=ctypes.c_void_p(4097)) == -3 and call(heads=70000, ss=2 ** 40, ds=2 ** 40) == -2
    assert call(heads=2 ** 62) == -2
    assert call(ds=72) == -1                     # in place, but to other rows
    assert call(N=0) == 0
    import copy
    import pickle
    assert pickle.loads(pickle.dumps(r)).freqs == r.freqs and copy.deepcopy(r) is r
    with pytest.raises(ValueError):
        eqlin.rope(r, None, torch.zeros(3, 32), None)


def test_attention_refusals():
    L = eqlin.lib()
    one = ctypes.c_void_p(4096)
    base = dict(tokens=6, heads=4, kv_heads=2, head_dim=8, q_stride=64, k_stride=64, v_stride=64, o_stride=32, docs=2,
                offsets=None, max_len=0, pos=None, slopes=None, axes=0, scale=1.0, cap=0.0, err=None, wait_limit=0)

    def call(dt=eqlin.BF16, q=one, k=one, v=one, o=one, lse=one, **kw):
        d = eqlin.AttentionDesc(**{**base, **kw})
        return L.eqlin_attention_forward(ctypes.byref(d), dt, q, k, v, o, lse, None)

    assert L.eqlin_attention_forward(None, 2, one, one, one, one, one, None) == -1
    assert call(dt=7) == -1 and call(tokens=-1) == -1 and call(heads=0) == -1 and call(kv_heads=3) == -1
    assert call(docs=0) == -1 and call(docs=4) == -1 and call(docs=-1) == -1 and call(max_len=-1) == -1
    assert call(scale=math.nan) == -1 and call(scale=0.0) == -1 and call(scale=-1.0) == -1 and call(cap=-1.0) == -1 and call(cap=math.inf) == -1
    assert call(axes=1) == -1 and call(axes=1, slopes=4096) == -1 and call(axes=4, slopes=4096, pos=4096) == -2
    assert call(head_dim=136, q_stride=1024, k_stride=1024, v_stride=1024, o_stride=1024) == -2
    assert call(head_dim=12) == -3 and call(head_dim=0) == -1
    assert call(q_stride=24) == -1 and call(k_stride=8) == -1 and call(v_stride=8) == -1 and call(o_stride=31) == -1
    assert call(q_stride=33) == -3 and call(tokens=2 ** 31, docs=1) == -2 and call(docs=2 ** 30, offsets=4096) == -2
    for name in ("q", "k", "v", "o"):
        assert call(**{name: None}) == -1 and call(**{name: ctypes.c_void_p(4098)}) == -3, name
    assert call(lse=None) == -1 and call(lse=ctypes.c_void_p(4098)) == -3 and call(docs=2 ** 62, offsets=4096) == -2
    for name in ("offsets", "err", "pos", "slopes"):
        assert call(**{name: 4097}) == -3, name
    assert call(tokens=0) == 0 and call(tokens=0, docs=0) == 0

    def back(dt=eqlin.BF16, go=one, gs=32, dq=one, dqs=32, dk=one, dks=16, dv=one, dvs=16, delta=one, **kw):
        d = eqlin.AttentionDesc(**{**base, **kw})
        return L.eqlin_attention_backward(ctypes.byref(d), dt, go, gs, one, one, one, one, one, dq, dqs, dk, dks, dv, dvs,
                                          delta, None)

    for name in ("go", "dq", "dk", "dv", "delta"):
        assert back(**{name: None}) == -1, name
    for name in ("go", "dq", "dk", "dv"):
        assert back(**{name: ctypes.c_void_p(4098)}) == -3, name
    assert back(gs=31) == -1 and back(dqs=33) == -3 and back(dks=8) == -1 and back(dvs=17) == -3
    assert back(tokens=0) == 0
    with pytest.raises(TypeError):
        eqlin.attention_forward(None, None, None, None, None)
