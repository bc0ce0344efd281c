"""Attention's gradients over the range of magnitudes that training meets.

An f16 gradient is small (a mean over a long batch), or large (a loss scale),
and so are the score gradients du that pass through 16 bits on their way into
a product.  What the results may be off, in the root mean square over a
tensor's values: every rounding to 16 bits is off by at most half a step, u
relative, hence u / sqrt(3) in the mean of values spread over a step, and half
the subnormals' spacing z where the output itself is that small.  Roundings
are independent, so those of a sum's terms add up as their squares.  A quarter
on top is room for the sample.  The FP32 part (scores, exponentials, sums)
counts in full."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from group_circulant_linear_b200 import eqlin

W = 2.0 ** -24


def formula(q, k, v, go, lens, cap, scale):
    """dq, dk, dv in 64 bits, and for each the mean squares that 16-bit operands add (in u^2), and the FP32 part."""
    N, H, D = q.shape
    K = k.shape[1]
    val, sq, lin = ({n: torch.zeros(s, dtype=torch.float64, device=q.device) for n, s in
                     dict(dq=(N, H, D), dk=(N, K, D), dv=(N, K, D)).items()} for _ in range(3))
    lo = 0
    for n in lens:
        r = slice(lo, lo + n)
        lo += n
        for h in range(H):
            kh = h // (H // K)
            Q, Kh, V, G = q[r, h].double(), k[r, kh].double(), v[r, kh].double(), go[r, h].double()
            s = scale * Q @ Kh.T
            mag = scale * Q.abs() @ Kh.abs().T
            g = torch.ones_like(s)
            if cap:
                t = torch.tanh(s / cap)
                s, g = cap * t, 1 - t * t
            P = torch.softmax(s, 1)
            dP = G @ V.T
            du = P * (dP - (P * dP).sum(1, keepdim=True)) * g
            # relative error of P: D + 4 roundings of the score's products, a dozen of the score, the exponential's
            # 2^-21; twice, for lse has them too; and a sum's n roundings
            e = 2 * float(((D + 4) * W * mag + 12 * W * (s.abs() + cap) + 2.0 ** -21).max()) + math.sqrt(n) * W
            e = e + 2 * D * W + (16 * W if cap else 0.0)              # dP, delta; 1 - tanh^2
            val["dq"][r, h] = scale * du @ Kh
            sq["dq"][r, h] = scale ** 2 * (du ** 2 @ Kh ** 2)
            lin["dq"][r, h] = e * scale * (du ** 2 @ Kh ** 2).sqrt() + e * scale * (du @ Kh).abs()
            val["dk"][r, kh] += scale * du.T @ Q
            sq["dk"][r, kh] += scale ** 2 * (du.T ** 2 @ Q ** 2)
            lin["dk"][r, kh] += e * scale * (du.T ** 2 @ Q ** 2).sqrt() + e * scale * (du.T @ Q).abs()
            val["dv"][r, kh] += P.T @ G
            sq["dv"][r, kh] += P.T ** 2 @ G ** 2
            lin["dv"][r, kh] += e * (P.T ** 2 @ G ** 2).sqrt() + e * (P.T @ G).abs()
    return val, sq, lin


def gradients(q, k, v, go, lens, cap, scale):
    N, H, _ = q.shape
    off = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    o, lse, delta = torch.empty_like(q), torch.empty((H, N), device="cuda"), torch.empty((H, N), device="cuda")
    d = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v))
    eqlin.attention_forward(q, k, v, o, lse, offsets=off, cap=cap, scale=scale)
    eqlin.attention_backward(go, q, k, v, o, lse, d["dq"], d["dk"], d["dv"], delta, offsets=off, cap=cap, scale=scale)
    return d


def compare(got, val, sq, lin, dt, weight=None):
    u = torch.finfo(dt).eps / 2
    z = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    for n in val:
        w = 1.0 if weight is None else weight[n]
        assert torch.isfinite(got[n]).all(), n
        off = float((w * (got[n].double() - val[n])).norm())
        room = 1.25 * math.sqrt(float((w ** 2 * (u * u * (val[n] ** 2 + sq[n]) + z * z) / 3).sum())) + float((w * lin[n]).norm())
        assert off <= room, f"{n}: off by {off}, {room} allowed, norm {float((w * val[n]).norm())}"


def inputs(lens, H, K, D, dt, seed, spread, v_std=1.0, per_token=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = sum(lens)

    def rnd(heads, std):
        return (torch.randn((N, heads, D), generator=g, device="cuda") * std).to(dt)

    q, k, v = rnd(H, 0.7), rnd(K, 0.7), rnd(K, v_std)
    go = torch.randn((N, H, D), generator=g, device="cuda") * spread
    if per_token is not None:
        scale = 10.0 ** (torch.rand((N, 1, 1), generator=g, device="cuda") * per_token)
        return q, k, v, (go * scale).to(dt), scale.double()
    return q, k, v, go.to(dt), None


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("spread", [1.0, 1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("lens,H,K,D,cap", [([8192], 1, 1, 64, 0.0), ([2048], 2, 1, 128, 0.0), ([1500, 37, 700], 2, 2, 64, 6.0),
                                            ([3001], 1, 1, 32, 0.0), ([1500, 37, 700], 2, 1, 104, 6.0)])
def test_small_gradients_keep_their_bits(lens, H, K, D, cap, spread, dtype):
    q, k, v, go, _ = inputs(lens, H, K, D, dtype, D + len(lens), spread)
    scale = D ** -0.5
    compare(gradients(q, k, v, go, lens, cap, scale), *formula(q, k, v, go, lens, cap, scale), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[2, 3, 5, 1, 40], [150, 300]])
def test_large_f16_gradients_stay_finite(lens, D):
    # a loss scale: dP is past f16's largest number, the results are not
    dt, scale = torch.float16, D ** -0.5
    q, k, v, go, _ = inputs(lens, 2, 2, D, dt, 5, 3.0e3, v_std=4.0)
    val, sq, lin = formula(q, k, v, go, lens, 0.0, scale)
    assert all(float(t.abs().max()) < 6.0e4 for t in val.values())
    compare(gradients(q, k, v, go, lens, 0.0, scale), val, sq, lin, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_f16_gradients_of_tokens_of_very_different_weight(D):
    # each token's dq by its own measure: go spans four decades between tokens
    lens, dt, scale = [1200, 900], torch.float16, D ** -0.5
    q, k, v, go, by = inputs(lens, 2, 1, D, dt, 6, 1e-4, per_token=4.0)
    val, sq, lin = formula(q, k, v, go, lens, 0.0, scale)
    got = gradients(q, k, v, go, lens, 0.0, scale)
    compare(got, val, sq, lin, dt)
    compare({"dq": got["dq"]}, {"dq": val["dq"]}, sq, lin, dt, weight={"dq": 1 / by})


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_f16_gradients_that_grow_along_a_document(D):
    # the factor of a row follows what passes by: values (queries' gradients) grow from 1e-4 to 1e4 and fall again
    n, dt, scale = 1300, torch.float16, D ** -0.5
    up = 10.0 ** torch.linspace(-4, 4, n // 2, device="cuda")
    for turn in (torch.cat([up, up.flip(0)]), torch.cat([up.flip(0), up])):
        q, k, v, go, _ = inputs([n], 1, 1, D, dt, 7, 1.0)
        v = (v.float() * turn[:, None, None].sqrt()).to(dt)
        go = (go.float() * turn[:, None, None].sqrt() * 0.01).to(dt)
        val, sq, lin = formula(q, k, v, go, [n], 0.0, scale)
        compare(gradients(q, k, v, go, [n], 0.0, scale), val, sq, lin, dt)
        zero = torch.zeros_like(go)
        zero[-3:] = go[-3:]                      # gradients of the last tokens only, nothing but zeros before
        val, sq, lin = formula(q, k, v, zero, [n], 0.0, scale)
        compare(gradients(q, k, v, zero, [n], 0.0, scale), val, sq, lin, dt)
    assert not any(t.any() for t in gradients(q, k, v, torch.zeros_like(go), [n], 0.0, scale).values())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [1.0e4, 1.0e6])
def test_a_cap_far_above_the_scores_is_as_good_as_none(cap, D, dtype):
    # cap tanh(u / cap) is u (1 - (u / cap)^2 / 3), and u is 30 at most: nothing beside the roundings.  Short documents:
    # all of their columns lie in a last, partial tile.
    lens, scale = [31, 20, 7, 100, 1000], D ** -0.5
    q, k, v, go, _ = inputs(lens, 2, 1, D, dtype, 8, 1.0)
    q = q * 4
    val, sq, lin = formula(q, k, v, go, lens, 0.0, scale)
    compare(gradients(q, k, v, go, lens, cap, scale), val, sq, lin, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n", [40, 1000])
def test_scores_far_below_a_cap_beside_one_near_it(n, dtype):
    # one query's scores come near a large cap; the others' must not take its form of the tanh
    D, cap, odd = 64, 3.0e4, 3
    scale = D ** -0.5
    q, k, v, go, _ = inputs([n], 1, 1, D, dtype, 9, 1.0)
    q[odd] *= 4.0e3 / float(q[odd].abs().max())
    k[5] = q[odd, 0] / 4.0e3 * 50.0                    # u = 0.125 |q| |k|, of the order of the cap
    assert 0.7 * cap < float(scale * (q[odd, 0].double() @ k[5, 0].double())) < 30 * cap
    go[odd] = 0                                        # its own gradients, one-hot, are another matter
    keep = torch.arange(n, device="cuda") != odd
    o, lse = torch.empty_like(q), torch.empty((1, n), device="cuda")
    eqlin.attention_forward(q, k, v, o, lse, cap=cap, scale=scale)
    val, sq, lin = formula(q, k, v, go, [n], cap, scale)
    # formula's bound of the FP32 part, of the rows that are looked at; a dozen roundings of the score, not of the cap
    u = scale * q[keep, 0].double() @ k[:, 0].double().T
    mag = scale * q[keep, 0].double().abs() @ k[:, 0].double().abs().T
    e = 2 * float(((D + 4) * W * mag + 12 * W * u.abs() + 2.0 ** -21).max()) + math.sqrt(n) * W + 2 * D * W
    P = torch.softmax(cap * torch.tanh(u / cap), 1)
    V = v[:, 0].double()
    half = torch.finfo(dtype).eps / 2
    want = P @ V
    room = 1.25 * half * math.sqrt(float((want ** 2).sum() + (P ** 2 @ V ** 2).sum()) / 3) \
        + e * float((P ** 2 @ V ** 2).sqrt().norm() + want.norm())
    assert float((o[keep, 0].double() - want).norm()) <= room
    got = gradients(q, k, v, go, [n], cap, scale)["dq"][keep]
    room = 1.25 * half * math.sqrt(float((val["dq"][keep] ** 2).sum() + sq["dq"][keep].sum()) / 3) \
        + e * float(sq["dq"][keep].sqrt().norm() + val["dq"][keep].norm())
    assert float((got.double() - val["dq"][keep]).norm()) <= room


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("n,D", [(300, 64), (4096, 64), (65536, 64), (4096, 128)])
def test_many_small_probabilities_beside_a_large_one(n, D, dtype):
    # one key takes nearly all of each query's attention, and its value is 0: what is left are the other keys'
    # probabilities, e^-17.4 each, below f16's smallest number
    g = torch.Generator(device="cuda").manual_seed(n + D)
    scale = D ** -0.5
    q = torch.full((n, 1, D), 1.0, device="cuda", dtype=dtype)
    k = torch.zeros((n, 1, D), device="cuda", dtype=dtype)
    at = n // 3
    k[at] = 17.4 / (scale * D)
    v = (1 + torch.rand((n, 1, D), generator=g, device="cuda")).to(dtype)
    v[at] = 0
    o, lse = torch.empty_like(q), torch.empty((1, n), device="cuda")
    eqlin.attention_forward(q, k, v, o, lse, scale=scale)
    s = scale * q[:1, 0].double() @ k[:, 0].double().T              # every query is the same
    P = torch.softmax(s, 1)
    want, mass = P @ v[:, 0].double(), P @ v[:, 0].double().abs()
    u = torch.finfo(dtype).eps / 2
    z = torch.finfo(dtype).smallest_normal * u
    # the output's rounding, P's, and in f16 half a step of its subnormals, 2^-25, on a P that carries 2^7; the FP32 part:
    # score and exponential (as in formula), sums of n terms
    e = 2 * ((D + 4) * W * 17.4 + 12 * W * 17.4 + 2.0 ** -21) + n * W
    tol = u * want + z + (u + e) * mass + (2.0 ** -32 if dtype == torch.float16 else 0.0) * v[:, 0].double().sum(0)
    assert bool(((o[:, 0].double() - want).abs() <= tol).all())
    assert float((lse.double() - torch.logsumexp(s, 1)).abs().max()) <= e + 4 * W * 17.4


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.0, 6.0])
@pytest.mark.parametrize("D", [40, 64, 128])
def test_f16_gradients_scale_exactly_with_powers_of_two(D, cap):
    # go times 2^s leaves every f16 operand's bits as they are: so are the results', times 2^s
    lens, scale = [700, 1, 64, 300], D ** -0.5
    q, k, v, go, by = inputs(lens, 4, 2, D, torch.float16, 10, 0.05, per_token=1.5)
    # only what has all its bits times 2^-7, too: an f16 below 2^-7 would fall among the subnormals (2^-14 and less) there
    go = (go.float() * 2.0 ** -7).half().float().mul(2.0 ** 7).half()
    base = gradients(q, k, v, go, lens, cap, scale)
    for s in (-7, -3, 4, 8):
        for n, got in gradients(q, k, v, go * 2.0 ** s, lens, cap, scale).items():
            # 2^-14 itself may come of a subnormal, which has fewer bits
            normal = (got.abs() > 2.0 ** -14) & (base[n].abs() > 2.0 ** -14)
            assert int(normal.sum()) > normal.numel() // 4
            assert torch.equal(got.double()[normal], base[n].double()[normal] * 2.0 ** s), (n, s)


def test_scales_and_caps_beyond_fp32_are_refused():
    L, one = eqlin.lib(), ctypes.c_void_p(4096)      # never followed: each call is refused first

    def call(scale, cap):
        d = eqlin.AttentionDesc(tokens=6, heads=2, kv_heads=2, head_dim=8, q_stride=16, k_stride=16, v_stride=16, o_stride=16,
                                docs=2, scale=scale, cap=cap)
        fwd = L.eqlin_attention_forward(ctypes.byref(d), eqlin.BF16, one, one, one, one, one, None)
        bwd = L.eqlin_attention_backward(ctypes.byref(d), eqlin.BF16, one, 16, one, one, one, one, one, one, 16, one, 16, one,
                                         16, one, None)
        assert fwd == bwd
        return fwd

    assert call(0.125, 1.0e38) == -2 and call(0.125, 1.0e-38) == -2 and call(1.0e-38, 0.0) == -2 and call(1.0e38, 0.0) == -2
    assert call(2.0 ** -70, 2.0 ** 70) == -2 and call(2.0 ** 70, 2.0 ** -70) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_the_largest_cap(dtype):
    lens, scale = [31, 100, 200], 0.125
    q, k, v, go, _ = inputs(lens, 2, 1, 64, dtype, 8, 1.0)
    compare(gradients(q, k, v, go, lens, 2.0 ** 116, scale), *formula(q, k, v, go, lens, 0.0, scale), dtype)
