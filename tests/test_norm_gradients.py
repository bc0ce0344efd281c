"""Gradients of the group layer norm of a residual sum, at the size of a training batch.

The statistics, y and the gradients follow from x + res before the sum is
rounded to the tensors' type, so the backward takes x and res as the forward
did: the stored sum in their place would put its rounding into dw, where a
long batch of it is far above the FP32 sums' own roundings."""
from __future__ import annotations

import pytest
import torch

from group_circulant_linear_b200 import eqlin, ops


def exact(x, res, w, gy, gs, T, eps):
    s = x.double() + res.double()
    mean = s.mean(1, keepdim=True)
    rstd = (((s - mean) ** 2).mean(1, keepdim=True) + eps) ** -0.5
    xh, g = (s - mean) * rstd, gy.double()
    gw = g * w.double().repeat_interleave(T)
    dx = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) + gs.double()
    C = x.shape[1] // T
    per = (g * xh).view(-1, C, T)
    return dx, per.sum((0, 2)), g.view(-1, C, T).sum((0, 2)), (per ** 2).sum().sqrt(), (g ** 2).sum().sqrt()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("call", ["buffers", "function"])
def test_weight_gradient_of_a_sum_has_no_16_bit_rounding(call, dtype):
    N, Cp, T = 64 * 197, 192, 4
    gen = torch.Generator(device="cuda").manual_seed(3)

    def rnd(*s, std=1.0, mean=0.0):
        return (torch.randn(s, generator=gen, device="cuda") * std + mean).to(dtype)

    x, res, gy, gs = rnd(N, Cp * T, mean=1.0), rnd(N, Cp * T, std=0.5), rnd(N, Cp * T), rnd(N, Cp * T)
    w, b = rnd(Cp, std=0.2, mean=1.0), rnd(Cp, std=0.2)
    dx, dw, db, rss_w, rss_b = exact(x, res, w, gy, gs, T, 1e-6)
    if call == "buffers":
        y, s, gx = (torch.empty_like(x) for _ in range(3))
        mean, rstd = (torch.empty(N, device="cuda") for _ in range(2))
        gw, gb = (torch.empty(Cp, device="cuda") for _ in range(2))
        eqlin.norm_forward(x, w, b, y, mean, rstd, T, res=res, xsum=s)
        eqlin.norm_backward(gy, x, w, mean, rstd, gx, gw, gb, T, gsum=gs, res=res)
        # At most 96 FP32 roundings go into a value of xh and 64 additions into the longest chain of a channel's
        # sum (rows of a thread, warps, slices of blocks, a tree), half a step of 2^-24 each, relative to terms whose
        # signs are independent: they add up as their root sum of squares.
        out = 0.0
    else:
        x.requires_grad_(True)
        w.requires_grad_(True)
        b.requires_grad_(True)
        y, s = ops.group_layer_norm(x, w, b, T, res=res)
        gx, gw, gb = torch.autograd.grad((y, s), (x, w, b), (gy, gs))
        out = torch.finfo(dtype).eps / 2              # the parameters' gradients come in their own type
    tol = 160 * 2.0 ** -24
    assert float((gw.double() - dw).norm()) <= tol * float(rss_w) + out * float(dw.norm())
    assert float((gb.double() - db).norm()) <= tol * float(rss_b) + out * float(db.norm())
    half = torch.finfo(dtype).eps / 2
    assert float((gx.double() - dx).norm()) <= (half + tol) * float(dx.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_start_anywhere(dtype):
    # contiguous tensors at an odd element of a larger buffer, as attention takes them
    N, Cp, T = 37, 24, 4
    gen = torch.Generator(device="cuda").manual_seed(1)

    def odd(t):
        buf = torch.empty(t.numel() + 1, dtype=dtype, device="cuda")
        buf[1:] = t.flatten()
        return buf[1:].view(t.shape)

    x, r, gy, gs = (torch.randn((N, Cp * T), generator=gen, device="cuda").to(dtype) for _ in range(4))
    w, b = (torch.randn(Cp, generator=gen, device="cuda").to(dtype) for _ in range(2))
    outs = []
    for place in (lambda t: t.clone(), odd):
        leaves = [place(t).requires_grad_(True) for t in (x, r, w, b)]
        y, s = ops.group_layer_norm(leaves[0], leaves[2], leaves[3], T, res=leaves[1])
        outs.append([y, s, *torch.autograd.grad((y, s), leaves, (place(gy), place(gs)))])
    assert all(torch.equal(p, q) for p, q in zip(*outs))
