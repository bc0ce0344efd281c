"""The block's other operators as differentiable torch functions.

* ``group_layer_norm`` -- LayerNorm over all C'*T features with affine
  parameters shared along the group axis, the residual add fused.
* ``rotary`` -- rotary positions with several axes.
* ``attention`` -- attention within documents, with capped scores and a
  distance bias.
* ``qkv_attention`` -- rotary positions and attention on a packed projection,
  with one packed gradient.

They run the kernels of ``include/eqlin.h`` on the tensors' device and current
stream, in the tensors' type (float16, bfloat16 or float32), and have first
derivatives only.  Positions, slopes and offsets are not differentiated.

In float16 and bfloat16 attention's kernels wait for their copies and products
within bounds.  ``err``, an int32 tensor of four zeros, records a wait that ran
out in either direction (results are then undefined); read it with
``eqlin.attention_error``.  Without one it goes unnoticed.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import eqlin


def _no_grad_for(**tensors):
    for name, t in tensors.items():
        if t is not None and t.requires_grad:
            raise ValueError(f"{name} is not differentiable here; detach it")


# -------------------------------------------------------------------- norm

def _rows(x, F):
    """[..., F] as the norm's kernels read it: [N, F], one row after the other from a 16-byte boundary on."""
    x = x.reshape(-1, F).contiguous()
    return x.clone() if x.data_ptr() % 16 else x


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, res, w, b, T, eps):
        x2 = _rows(x, x.shape[-1])
        r2 = None if res is None else _rows(res, x.shape[-1])
        y = torch.empty_like(x2)
        s = None if res is None else torch.empty_like(x2)
        mean = torch.empty(x2.shape[0], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        w, b = w.contiguous(), b.contiguous()
        eqlin.norm_forward(x2, w, b, y, mean, rstd, T, eps=eps, res=r2, xsum=s)
        ctx.save_for_backward(x2, r2, w, mean, rstd)
        ctx.T = T
        ctx.set_materialize_grads(False)
        return (y.view(x.shape), s.view(x.shape)) if s is not None else y.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gs=None):
        x, r, w, mean, rstd = ctx.saved_tensors
        if gy is None and gs is None:
            return None, None, None, None, None, None
        shape = (gy if gy is not None else gs).shape
        if gy is None:                        # only the sum was used
            return gs, (gs if r is not None else None), torch.zeros_like(w), torch.zeros_like(w), None, None
        gy = _rows(gy, x.shape[1])
        gs = None if gs is None else _rows(gs, x.shape[1])
        dx = torch.empty_like(x)
        dw = torch.empty(w.shape, dtype=torch.float32, device=w.device)
        db = torch.empty_like(dw)
        eqlin.norm_backward(gy, x, w, mean, rstd, dx, dw, db, ctx.T, gsum=gs, res=r)
        dx = dx.view(shape)
        return dx, (dx if r is not None else None), dw.to(w.dtype), db.to(w.dtype), None, None


def group_layer_norm(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor, T: int, eps: float = 1e-6,
                     res: torch.Tensor | None = None):
    """y [..., C'*T] from x and w, b [C']; with ``res`` the pair (y, x + res),
    where y is the norm of the sum.  The backward keeps both x and ``res``
    rather than the sum, so that the weight's gradient is free of its rounding."""
    if res is not None and res.shape != x.shape:
        raise ValueError(f"res must have the shape of x, {tuple(x.shape)}, got {tuple(res.shape)}")
    return _Norm.apply(x, res, w, b, int(T), float(eps))


# ------------------------------------------------------------------ rotary

def _flat_heads(x):
    """[..., heads, D] as [N, heads, D] with the heads of a token one after the other."""
    H, D = x.shape[-2:]
    x = x.reshape(-1, H, D)
    if x.numel() and not ((D == 1 or x.stride(2) == 1) and (H == 1 or x.stride(1) == D)
                          and (x.shape[0] == 1 or x.stride(0) >= H * D)):
        x = x.contiguous()
    return x


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos, plan, inverse):
        src = _flat_heads(x)
        dst = torch.empty(src.shape, dtype=x.dtype, device=x.device)
        eqlin.rope(plan, pos, src, dst, inverse=inverse)
        ctx.save_for_backward(pos)
        ctx.plan, ctx.inverse = plan, inverse
        return dst.view(x.shape)

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        (pos,) = ctx.saved_tensors
        src = _flat_heads(gy)
        dst = torch.empty(src.shape, dtype=gy.dtype, device=gy.device)
        eqlin.rope(ctx.plan, pos, src, dst, inverse=not ctx.inverse)
        return dst.view(gy.shape), None, None, None


def _flat_pos(pos, N, axes, period):
    """Positions of N tokens as float32 [N, axes]; ``period`` rows repeat (one
    grid for every image of a batch)."""
    if axes and pos.shape[-1] != axes:
        raise ValueError(f"pos must have {axes} axes, got {pos.shape[-1]}")
    if N == 0:                                # the grid of every image of an empty batch
        return pos.new_empty((0, pos.shape[-1]), dtype=torch.float32)
    p = pos.reshape(-1, pos.shape[-1]).to(torch.float32)
    if p.shape[0] != N:
        if p.shape[0] != period or period == 0 or N % period:
            raise ValueError(f"pos has {p.shape[0]} rows for {N} tokens")
        p = p.repeat(N // period, 1)
    return p.contiguous()


def rotary(x: torch.Tensor, pos: torch.Tensor, plan: eqlin.Rope, inverse: bool = False) -> torch.Tensor:
    """x [..., tokens, heads, Ch*T] turned by the positions of its tokens, pos
    [..., tokens, axes] or [tokens, axes]."""
    _no_grad_for(pos=pos)
    if x.dim() < 3:
        raise ValueError("x must be [..., heads, Ch*T]")
    N = x.numel() // max(1, x.shape[-1] * x.shape[-2])
    return _Rotary.apply(x, _flat_pos(pos, N, plan.axes, x.shape[-3]), plan, bool(inverse))


# --------------------------------------------------------------- attention

def _aligned(x):
    """[N, heads, D] as the attention kernels read it: 16-byte rows and start."""
    x = _flat_heads(x)
    e = x.element_size()
    if x.numel() and (x.data_ptr() % 16 or (x.shape[0] > 1 and x.stride(0) * e % 16)):
        x = x.clone(memory_format=torch.contiguous_format)
    return x


_SHARED = ("offsets", "pos", "slopes")        # tensors that both directions read


def _read_again(ctx, kw, *tensors):
    """Save a call's tensors, the shared ones with them: changed in place before
    the backward, they would be read as something else, which torch refuses."""
    ctx.save_for_backward(*tensors, *(kw[n] for n in _SHARED))
    ctx.kw = {n: v for n, v in kw.items() if n not in _SHARED}


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, kw):
        q, k, v = _aligned(q), _aligned(k), _aligned(v)
        N, H, _ = q.shape
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty((H, N), dtype=torch.float32, device=q.device)
        eqlin.attention_forward(q, k, v, o, lse, **kw)
        _read_again(ctx, kw, q, k, v, o, lse)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, go):
        q, k, v, o, lse, *shared = ctx.saved_tensors
        go = _aligned(go)
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        eqlin.attention_backward(go, q, k, v, o, lse, dq, dk, dv, torch.empty_like(lse), **ctx.kw,
                                 **dict(zip(_SHARED, shared)))
        return dq, dk, dv, None


def _period(N, docs, offsets):
    """Tokens of each document, where all have as many."""
    return N // docs if offsets is None and docs > 0 else 0


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, docs: int = 1, offsets: torch.Tensor | None = None,
              max_len: int | None = None, pos: torch.Tensor | None = None, slopes: torch.Tensor | None = None,
              scale: float | None = None, cap: float = 0.0, err: torch.Tensor | None = None) -> torch.Tensor:
    """Attention within documents on packed tokens: q [N, heads, D], k and v
    [N, kv_heads, D] -> [N, heads, D]; see ``eqlin.attention_forward``."""
    _no_grad_for(pos=pos, slopes=slopes)
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [N, heads, D]")
    kw = dict(docs=docs, offsets=offsets, max_len=max_len, slopes=slopes, scale=scale, cap=cap, err=err,
              pos=None if pos is None else _flat_pos(pos, q.shape[0], 0, _period(q.shape[0], docs, offsets)))
    return _Attention.apply(q, k, v, kw)


class _QkvAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, qkv, heads, kv_heads, plan, rope_pos, kw):
        qkv = _aligned(qkv)
        N, _, D = qkv.shape
        H, K = heads, kv_heads
        qk = qkv[:, :H + K]
        if plan is not None:
            turned = torch.empty((N, H + K, D), dtype=qkv.dtype, device=qkv.device)
            eqlin.rope(plan, rope_pos, qk, turned)
            qk = turned
        o = torch.empty((N, H, D), dtype=qkv.dtype, device=qkv.device)
        lse = torch.empty((H, N), dtype=torch.float32, device=qkv.device)
        eqlin.attention_forward(qk[:, :H], qk[:, H:], qkv[:, H + K:], o, lse, **kw)
        _read_again(ctx, kw, qkv, qk if plan is not None else None, o, lse, rope_pos)
        ctx.heads, ctx.kv_heads, ctx.plan = H, K, plan
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, go):
        qkv, qk, o, lse, rope_pos, *shared = ctx.saved_tensors
        H, K = ctx.heads, ctx.kv_heads
        qk = qkv[:, :H + K] if qk is None else qk
        d = torch.empty(qkv.shape, dtype=qkv.dtype, device=qkv.device)
        eqlin.attention_backward(_aligned(go), qk[:, :H], qk[:, H:], qkv[:, H + K:], o, lse, d[:, :H], d[:, H:H + K],
                                 d[:, H + K:], torch.empty_like(lse), **ctx.kw, **dict(zip(_SHARED, shared)))
        if ctx.plan is not None:
            eqlin.rope(ctx.plan, rope_pos, d[:, :H + K], d[:, :H + K], inverse=True)
        return d, None, None, None, None, None


def qkv_attention(qkv: torch.Tensor, heads: int, kv_heads: int | None = None, *, plan: eqlin.Rope | None = None,
                  pos: torch.Tensor | None = None, slopes: torch.Tensor | None = None, docs: int = 1,
                  offsets: torch.Tensor | None = None, max_len: int | None = None, scale: float | None = None,
                  cap: float = 0.0, err: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of a packed projection qkv [N, heads + 2 kv_heads, D] (queries,
    keys, values), whose queries and keys ``plan`` turns first.  ``pos`` [N,
    axes] (or one grid for each of ``docs`` documents) serves both the plan
    and, with ``slopes`` [heads], the distance bias.

    In float16 and bfloat16 the turned queries and keys are rounded to the type,
    as ``rotary`` rounds them, and so are their gradients before they are turned
    back: two roundings of half a step each where the others have one."""
    kv_heads = heads if kv_heads is None else kv_heads
    _no_grad_for(pos=pos, slopes=slopes)
    if qkv.dim() != 3 or qkv.shape[1] != heads + 2 * kv_heads:
        raise ValueError(f"qkv must be [N, {heads + 2 * kv_heads}, D], got {tuple(qkv.shape)}")
    if pos is None and (plan is not None or slopes is not None):
        raise ValueError("rotary positions and the distance bias need pos")
    if plan is not None and plan.Ch * plan.T != qkv.shape[2]:
        raise ValueError(f"the plan turns heads of {plan.Ch} * {plan.T} features, qkv has {qkv.shape[2]}")
    p = None if pos is None else _flat_pos(pos, qkv.shape[0], plan.axes if plan is not None else 0,
                                             _period(qkv.shape[0], docs, offsets))
    kw = dict(docs=docs, offsets=offsets, max_len=max_len, slopes=slopes, pos=p if slopes is not None else None,
              scale=scale, cap=cap, err=err)
    return _QkvAttention.apply(qkv, int(heads), int(kv_heads), plan, p if plan is not None else None, kw)
