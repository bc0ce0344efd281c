"""EQ-Linear as a torch autograd layer, and a synthetic EQ-ViT block built on it.

The pages present Flash EQ-Linear as a drop-in replacement for the naive
equivariant linear layer, with no retraining, and time it inside EQ-ViT
blocks ("Flash EQ-Linear", technical summary, sections "Implementacao" and
"Resultados Experimentais").  This module is that drop-in:

* ``EQLinearFunction`` -- when gradients are needed and every pass runs on
  the tensor cores, forward runs ``eqlin_forward_stash`` and keeps the input's
  spectrum X = DFT(x) (instead of x) for the backward, which is one
  ``eqlin_backward`` call: dx with G = DFT(gy) stashed, then dW and db from
  the two spectra.  Otherwise forward runs ``eqlin_forward`` and backward
  ``eqlin_backward_dx`` and ``eqlin_backward_dw``.  All through the C ABI
  binding.
* ``EQLinear`` -- an ``nn.Module`` holding W [D', C', T] and b [D'] as
  parameters and one library handle; it re-runs the weight transform
  (``eqlin_set_weights``) only when the parameters have changed.
* ``GroupLayerNorm`` and ``EQViTBlock`` -- a pre-norm transformer block whose
  qkv, projection and MLP layers are EQ-Linear.  Features are [C', T]: the
  norm's statistics run over all C'T features and its affine parameters are
  shared along the group axis, attention heads split C', and GELU is
  pointwise, so the block commutes with a cyclic shift of the group axis.
  Weights are synthetic (random).
  With ``native=True`` the norms and the attention run the library's kernels
  too (``ops.py``), and the block takes rotary positions, capped scores, a
  distance bias, shared key heads and packed images of different sizes.
* ``expand_dense`` and ``DenseEQViTBlock`` -- the naive layer the pages
  compare against: the block-circulant dense matrix W_dense[d*T+s, c*T+t] =
  W[d, c, (s-t) mod T] applied with an ordinary (cuBLAS) linear.  It is
  timed beside the Flash block for context only.

``python -m group_circulant_linear_b200.block`` times one block, forward and
forward + backward, both ways, and prints one JSON line; ``--native`` adds the
block with the library's norms and attention.
"""
from __future__ import annotations

import argparse
import json
import math

import torch
import torch.nn as nn
import torch.nn.functional as F

from . import eqlin, ops


class EQLinearFunction(torch.autograd.Function):
    """y = EQ-Linear(x; W, b) with the library's kernels in both directions."""

    @staticmethod
    def forward(ctx, x, W, b, layer):
        lead = x.shape[:-1]
        x2 = x.reshape(-1, layer.Cp * layer.T).to(layer.dtype).contiguous()
        layer.sync_weights(W, b)
        N = x2.shape[0]
        y = torch.empty((N, layer.Dp * layer.T), dtype=layer.dtype, device=x.device)
        fused = layer.fused and any(ctx.needs_input_grad[:3]) and N > 0
        if fused:
            xs = eqlin.empty_spectra(layer.h, "x", N, device=x.device)
            eqlin.forward_stash(layer.h, x2, y, xs)
            ctx.save_for_backward(xs)
        else:
            eqlin.forward(layer.h, x2, y)
            ctx.save_for_backward(x2)
        ctx.fused = fused
        ctx.N = N
        ctx.layer = layer
        ctx.lead = lead
        ctx.x_dtype = x.dtype
        ctx.w_dtype = W.dtype
        ctx.b_dtype = None if b is None else b.dtype
        return y.reshape(*lead, layer.Dp * layer.T)

    @staticmethod
    def backward(ctx, gy):
        (saved,) = ctx.saved_tensors
        L = ctx.layer
        gy2 = gy.reshape(-1, L.Dp * L.T).to(L.dtype).contiguous()
        dx = dW = db = None
        want_w = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx2 = torch.empty((ctx.N, L.Cp * L.T), dtype=L.dtype, device=gy.device) \
            if (ctx.needs_input_grad[0] or (ctx.fused and want_w)) else None
        if want_w:
            dWf = torch.empty((L.Dp, L.Cp, L.T), dtype=torch.float32, device=gy.device)
            dbf = torch.empty((L.Dp,), dtype=torch.float32, device=gy.device)
        if ctx.fused and want_w:
            # one pass over gy: dx and G = DFT(gy), then dW, db from the spectra
            gs = eqlin.empty_spectra(L.h, "gy", ctx.N, device=gy.device)
            eqlin.backward(L.h, gy2, saved, dx2, gs, dWf, dbf)
        else:
            if dx2 is not None:
                eqlin.backward_dx(L.h, gy2, dx2)
            if want_w:
                eqlin.backward_dw(L.h, saved, gy2, dWf, dbf)
        if ctx.needs_input_grad[0]:
            dx = dx2.reshape(*ctx.lead, L.Cp * L.T).to(ctx.x_dtype)
        if ctx.needs_input_grad[1]:
            dW = dWf.to(ctx.w_dtype)
        if ctx.needs_input_grad[2]:
            db = dbf.to(ctx.b_dtype)
        return dx, dW, db, None


class EQLinear(nn.Module):
    """Group-circulant linear layer: [..., C'*T] -> [..., D'*T].

    ``dtype`` is the compute dtype of the library handle (bf16, f16 or f32);
    the parameters are created in it.  Init: W and b uniform in
    +-1/sqrt(C'*T), as for an ordinary linear layer with C'*T inputs.
    """

    def __init__(self, Cp: int, Dp: int, T: int = 4, bias: bool = True, dtype=torch.bfloat16,
                 device="cuda", generator: torch.Generator | None = None):
        super().__init__()
        self.Cp, self.Dp, self.T, self.dtype = int(Cp), int(Dp), int(T), dtype
        bound = 1.0 / math.sqrt(Cp * T)
        w = (torch.rand((Dp, Cp, T), generator=generator) * 2 - 1) * bound
        self.weight = nn.Parameter(w.to(device=device, dtype=dtype))
        if bias:
            bb = (torch.rand((Dp,), generator=generator) * 2 - 1) * bound
            self.bias = nn.Parameter(bb.to(device=device, dtype=dtype))
        else:
            self.register_parameter("bias", None)
        self.h = eqlin.create(T, Cp, Dp, dtype)
        # the stash forms (fused backward) serve f16/bf16 layers of order T | 8
        # whose passes all run on tensor cores
        self.fused = (self.h.backend() == "fwd=tcgen05 dx=tcgen05 dw=tcgen05" and self.h.T in (1, 2, 4, 8)
                      and self.dtype != torch.float32)
        self._seen = None

    def sync_weights(self, W: torch.Tensor, b: torch.Tensor | None):
        """Run the weight transform if W or b changed since it last ran."""
        # the handle's identity too: a deep copy of the module gets a new,
        # empty handle and must load its weights again
        key = (id(self.h), W.data_ptr(), W._version, None if b is None else (b.data_ptr(), b._version))
        if key != self._seen:
            eqlin.set_weights(self.h, W.detach().to(self.dtype).contiguous(),
                              None if b is None else b.detach().to(self.dtype).contiguous())
            self._seen = key

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return EQLinearFunction.apply(x, self.weight, self.bias, self)

    def extra_repr(self) -> str:
        return f"C'={self.Cp}, D'={self.Dp}, T={self.T}, dtype={self.dtype}, backend={self.h.backend()}"


class GroupLayerNorm(nn.Module):
    """LayerNorm over all C'*T features, with one scale and shift per channel
    c shared by its T group positions (so it commutes with a cyclic shift).

    ``native`` runs the library's kernel, which also takes a residual: then
    ``norm(x, res)`` is the pair of the normalised sum and the sum itself.  It
    takes inputs of the parameters' type, and does not promote others."""

    def __init__(self, Cp: int, T: int, eps: float = 1e-6, dtype=torch.bfloat16, device="cuda", native: bool = False):
        super().__init__()
        self.Cp, self.T, self.eps, self.native = Cp, T, eps, bool(native)
        self.weight = nn.Parameter(torch.ones(Cp, dtype=dtype, device=device))
        self.bias = nn.Parameter(torch.zeros(Cp, dtype=dtype, device=device))

    def forward(self, x: torch.Tensor, res: torch.Tensor | None = None):
        if self.native:
            return ops.group_layer_norm(x, self.weight, self.bias, self.T, self.eps, res)
        if res is not None:
            x = x + res
            return self.forward(x), x
        y = F.layer_norm(x, (self.Cp * self.T,), None, None, self.eps)
        y = y.view(*x.shape[:-1], self.Cp, self.T) * self.weight[:, None] + self.bias[:, None]
        return y.view(x.shape)


def _attention(h: torch.Tensor, heads: int, Cp: int, T: int) -> torch.Tensor:
    """Multi-head self-attention on qkv features [B, L, 3*C'*T]; heads split C'."""
    B, L, _ = h.shape
    q, k, v = h.view(B, L, 3, heads, (Cp // heads) * T).permute(2, 0, 3, 1, 4)
    o = F.scaled_dot_product_attention(q, k, v)
    return o.transpose(1, 2).reshape(B, L, Cp * T)


class EQViTBlock(nn.Module):
    """Pre-norm ViT block on features [B, L, C'*T] with EQ-Linear layers.

    The options from ``kv_heads`` on need ``native=True``:

    * ``kv_heads``: key and value heads (a divisor of ``heads``), each shared
      by heads / kv_heads query heads;
    * ``rope_sections``: channel pairs of a head that turn with each axis of
      the positions (``rope_base`` sets their frequencies, ``eqlin.Rope``);
    * ``cap``: scores are capped to +-cap by a tanh (0: not);
    * ``distance``: a bias of -slope * city-block distance between positions,
      head h's slope being 2^(-8 (h+1) / heads).

    All of them keep the block's commutation with a shift of the group axis.
    ``forward(x, pos)`` takes positions [L, axes] (the same grid for every
    image), [B, L, axes] or [N, axes]; ``forward(x [N, C'*T], pos, offsets,
    max_len)`` takes packed images of different sizes (``offsets`` int32
    [images + 1])."""

    def __init__(self, Cp: int, heads: int, T: int = 4, mlp_ratio: int = 4, dtype=torch.bfloat16,
                 device="cuda", seed: int = 0, native: bool = False, kv_heads: int | None = None, rope_sections=None,
                 rope_base: float = 100.0, cap: float = 0.0, distance: bool = False):
        super().__init__()
        if Cp % heads:
            raise ValueError("heads must divide C'")
        self.kv_heads = heads if kv_heads is None else int(kv_heads)
        if self.kv_heads < 1 or heads % self.kv_heads:
            raise ValueError("kv_heads must divide heads")
        if not native and (self.kv_heads != heads or rope_sections is not None or cap or distance):
            raise ValueError("kv_heads, rope_sections, cap and distance need native=True")
        g = torch.Generator().manual_seed(seed)
        self.Cp, self.T, self.heads, self.native, self.cap = Cp, T, heads, bool(native), float(cap)
        self.rope = None if rope_sections is None else eqlin.Rope(T, Cp // heads, rope_sections, rope_base)
        # a plain attribute: a buffer would follow the module into 16 bits
        self.slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)], dtype=torch.float32,
                                   device=device) if distance else None
        self.errs = {}                             # the attention's records by device, see get_error
        if native:
            self._err(torch.empty(0, device=device).device)
        self.norm1 = GroupLayerNorm(Cp, T, dtype=dtype, device=device, native=native)
        self.qkv = EQLinear(Cp, (heads + 2 * self.kv_heads) * (Cp // heads), T, dtype=dtype, device=device, generator=g)
        self.proj = EQLinear(Cp, Cp, T, dtype=dtype, device=device, generator=g)
        self.norm2 = GroupLayerNorm(Cp, T, dtype=dtype, device=device, native=native)
        self.fc1 = EQLinear(Cp, mlp_ratio * Cp, T, dtype=dtype, device=device, generator=g)
        self.fc2 = EQLinear(mlp_ratio * Cp, Cp, T, dtype=dtype, device=device, generator=g)

    def forward(self, x: torch.Tensor, pos: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                max_len: int | None = None) -> torch.Tensor:
        if not self.native:
            if pos is not None or offsets is not None:
                raise ValueError("positions and packed images need native=True")
            x = x + self.proj(_attention(self.qkv(self.norm1(x)), self.heads, self.Cp, self.T))
            return x + self.fc2(F.gelu(self.fc1(self.norm2(x))))
        if offsets is None and x.dim() != 3:
            raise ValueError("x must be [B, L, C'*T], or [N, C'*T] with offsets")
        if pos is None and (self.rope is not None or self.slopes is not None):
            raise ValueError("rotary positions and the distance bias need pos")
        if self.slopes is not None and self.slopes.device != x.device:
            self.slopes = self.slopes.to(x.device)
        h = self.qkv(self.norm1(x))
        o = ops.qkv_attention(h.reshape(-1, self.heads + 2 * self.kv_heads, (self.Cp // self.heads) * self.T), self.heads,
                              self.kv_heads, plan=self.rope, pos=pos,
                              slopes=self.slopes,
                              docs=x.shape[0] if offsets is None else 1, offsets=offsets, max_len=max_len, cap=self.cap,
                              err=self._err(x.device))
        y, x = self.norm2(x, self.proj(o.reshape(x.shape)))
        return x + self.fc2(F.gelu(self.fc1(y)))

    def _err(self, device: torch.device) -> torch.Tensor:
        if device not in self.errs:
            self.errs[device] = torch.zeros(4, dtype=torch.int32, device=device)
        return self.errs[device]

    def get_error(self) -> int:
        """Device-side status of the block's layers and, where it is native, its
        attention, in either direction: 0, or -6 for a wait that timed out
        (results are then undefined); clears it.  Synchronise streams other than
        the current one before."""
        status = [eqlin.get_error(layer.h) for layer in (self.qkv, self.proj, self.fc1, self.fc2)]
        return min(status + [eqlin.attention_error(err) for err in self.errs.values()])


def grid_positions(height: int, width: int, frames: int | None = None, lead: int = 0, device="cuda") -> torch.Tensor:
    """Positions [lead + patches, axes] of an image's patches in reading order
    (axes: height, width) or of a clip's (frame, height, width), after ``lead``
    tokens (class tokens, say) at the origin."""
    dims = (height, width) if frames is None else (frames, height, width)
    grid = torch.stack(torch.meshgrid(*(torch.arange(n, device=device) for n in dims), indexing="ij"), -1)
    grid = grid.reshape(-1, len(dims)).float()
    return torch.cat([torch.zeros((lead, len(dims)), device=device), grid])


def expand_dense(W: torch.Tensor) -> torch.Tensor:
    """The naive layer's matrix: W_dense[d*T+s, c*T+t] = W[d, c, (s-t) mod T]."""
    Dp, Cp, T = W.shape
    s = torch.arange(T, device=W.device)
    idx = (s[:, None] - s[None, :]) % T               # [s, t]
    return W[:, :, idx].permute(0, 2, 1, 3).reshape(Dp * T, Cp * T)


class DenseEQViTBlock(nn.Module):
    """The same block with every EQ-Linear applied as the expanded dense
    matrix (``F.linear``), sharing the parameters of ``src``.  Context only:
    the naive layer the pages measure against.  It has plain attention: a
    block with rotary positions, a cap, a distance bias or shared key heads is
    refused."""

    def __init__(self, src: EQViTBlock, dtype=None):
        super().__init__()
        if src.rope is not None or src.cap or src.slopes is not None or src.kv_heads != src.heads:
            raise ValueError("the dense block has no rotary positions, cap, distance bias or shared key heads")
        self.src, self.dtype = src, dtype

    def _lin(self, layer: EQLinear, x: torch.Tensor) -> torch.Tensor:
        W, b = layer.weight, layer.bias
        if self.dtype is not None:
            W, b = W.to(self.dtype), None if b is None else b.to(self.dtype)
        return F.linear(x, expand_dense(W), None if b is None else b.repeat_interleave(layer.T))

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        s = self.src

        def norm(n, v):
            w, b = n.weight, n.bias
            if self.dtype is not None:
                w, b = w.to(self.dtype), b.to(self.dtype)
            y = F.layer_norm(v, (n.Cp * n.T,), None, None, n.eps)
            return (y.view(*v.shape[:-1], n.Cp, n.T) * w[:, None] + b[:, None]).view(v.shape)

        x = x + self._lin(s.proj, _attention(self._lin(s.qkv, norm(s.norm1, x)), s.heads, s.Cp, s.T))
        return x + self._lin(s.fc2, F.gelu(self._lin(s.fc1, norm(s.norm2, x))))


MODELS = {  # name: (C' at T = 4, heads); tokens per image 197 (224 x 224, patch 16)
    "eq-vit-s": (96, 6),
    "eq-vit-b": (192, 12),
}


def _time(fn, iters: int, warmup: int) -> float:
    for _ in range(warmup):
        fn()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(iters):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / iters


def main(argv=None):
    ap = argparse.ArgumentParser(description="Time one synthetic EQ-ViT block, Flash EQ-Linear vs the dense matrix.")
    ap.add_argument("--model", default="eq-vit-b", choices=sorted(MODELS))
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--tokens", type=int, default=197)
    ap.add_argument("--dtype", default="bf16", choices=("bf16", "f16"))
    ap.add_argument("--iters", type=int, default=50)
    ap.add_argument("--warmup", type=int, default=5)
    ap.add_argument("--native", action="store_true", help="also time the block with the library's norms and attention")
    args = ap.parse_args(argv)
    dt = {"bf16": torch.bfloat16, "f16": torch.float16}[args.dtype]
    Cp, heads = MODELS[args.model]
    T = 4
    blk = EQViTBlock(Cp, heads, T, dtype=dt)
    dense = DenseEQViTBlock(blk)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((args.batch, args.tokens, Cp * T), generator=g, device="cuda", dtype=dt, requires_grad=True)
    gy = torch.randn((args.batch, args.tokens, Cp * T), generator=g, device="cuda", dtype=dt)

    def fwd(m):
        with torch.no_grad():
            m(x)

    def fwd_bwd(m):
        m(x).backward(gy)

    out = {"model": args.model, "batch": args.batch, "tokens": args.tokens, "dtype": args.dtype, "T": T,
           "C_prime": Cp, "heads": heads, "unit": "ms", "weights": "synthetic (random)"}
    timed = [("flash", blk), ("dense_matrix", dense)]
    if args.native:
        timed.append(("native", EQViTBlock(Cp, heads, T, dtype=dt, native=True)))
    for name, m in timed:
        out[f"{name}_fwd_ms"] = _time(lambda: fwd(m), args.iters, args.warmup)
        out[f"{name}_fwd_bwd_ms"] = _time(lambda: fwd_bwd(m), args.iters, args.warmup)
    out["speedup_fwd"] = out["dense_matrix_fwd_ms"] / out["flash_fwd_ms"]
    out["speedup_fwd_bwd"] = out["dense_matrix_fwd_bwd_ms"] / out["flash_fwd_bwd_ms"]
    if args.native:
        out["native_speedup_fwd_bwd"] = out["flash_fwd_bwd_ms"] / out["native_fwd_bwd_ms"]
    if any(m.get_error() != 0 for _, m in timed if isinstance(m, EQViTBlock)):
        raise RuntimeError("device-side timeout in a kernel")
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
