"""The EQ-ViT block with the library's norm, rotary positions and attention:
the three operators together, as a user runs them, against the same block in
plain torch (FP32 or FP64, dense matrices), packed and padded batches, the
group shift, and graph capture."""
from __future__ import annotations

import pytest
import torch
import torch.nn.functional as F

from group_circulant_linear_b200 import eqlin, ops
from group_circulant_linear_b200.block import EQViTBlock, GroupLayerNorm, expand_dense, grid_positions

# Seven roundings to bf16 lie between x and y in each branch of the block (as in the block's other
# comparison, which allows 3e-2 in relative Frobenius norm), each 2^-9 relative in the mean.
TOL_BLOCK = 3e-2
# FP32: each of the seven steps is a 3xTF32 product or an FP32 kernel, held to 1e-5 on its own.
TOL_F32 = 7e-5


def rel(a, b):
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    return float((a - b).norm() / b.norm())


def plain_block(blk, x, pos, lens, dt):
    """The block's definition with dense matrices on packed tokens x [N, F]."""
    T, H, K = blk.T, blk.heads, blk.kv_heads
    ch = blk.Cp // H

    def lin(layer, v):
        return F.linear(v, expand_dense(layer.weight.to(dt)), layer.bias.to(dt).repeat_interleave(T))

    def norm(n, v):
        y = F.layer_norm(v, (v.shape[-1],), None, None, n.eps)
        return y * n.weight.to(dt).repeat_interleave(T) + n.bias.to(dt).repeat_interleave(T)

    qkv = lin(blk.qkv, norm(blk.norm1, x)).view(-1, H + 2 * K, ch, T)
    qk, v = qkv[:, :H + K], qkv[:, H + K:]
    if blk.rope is not None:
        half = ch // 2
        ang = torch.zeros(x.shape[0], half, dtype=torch.float64, device=x.device)
        i = 0
        for a, n in enumerate(blk.rope.sections):
            for _ in range(n):
                ang[:, i] = pos[:, a].double() * blk.rope.freqs[i]
                i += 1
        c, s = ang.cos().to(dt)[:, None, :, None], ang.sin().to(dt)[:, None, :, None]
        a, b = qk[:, :, :half], qk[:, :, half:]
        qk = torch.cat([a * c - b * s, b * c + a * s], 2)
    q, k, v = qk[:, :H].flatten(2), qk[:, H:].flatten(2), v.flatten(2)
    outs, lo = [], 0
    for n in lens:
        r = slice(lo, lo + n)
        lo += n
        s = torch.einsum("ihd,jhd->hij", q[r], k[r].repeat_interleave(H // K, 1)) * (ch * T) ** -0.5
        if blk.cap:
            s = blk.cap * torch.tanh(s / blk.cap)
        if blk.slopes is not None:
            s = s - blk.slopes.to(dt)[:, None, None] * (pos[r][:, None] - pos[r][None]).abs().sum(2).to(dt)
        outs.append(torch.einsum("hij,jhd->ihd", s.softmax(2), v[r].repeat_interleave(H // K, 1)).flatten(1))
    if lo < x.shape[0]:
        outs.append(torch.zeros((x.shape[0] - lo, H * ch * T), dtype=dt, device=x.device))
    x = x + lin(blk.proj, torch.cat(outs))
    return x + lin(blk.fc2, F.gelu(lin(blk.fc1, norm(blk.norm2, x))))


def make(dtype, T=4, Cp=32, heads=4, **kw):
    kw = dict(kv_heads=2, rope_sections=(2, 2), cap=8.0, distance=True) if not kw else kw
    blk = EQViTBlock(Cp, heads, T, dtype=dtype, seed=5, native=True, **kw)
    g = torch.Generator().manual_seed(8)
    with torch.no_grad():
        for n in (blk.norm1, blk.norm2):
            n.weight.copy_(1 + 0.2 * torch.randn(n.weight.shape, generator=g))
            n.bias.copy_(0.2 * torch.randn(n.bias.shape, generator=g))
    return blk


def grads(blk, x, y, gy):
    return dict(zip(["x"] + [n for n, _ in blk.named_parameters()],
                    torch.autograd.grad(y, [x] + list(blk.parameters()), gy)))


def test_options_need_native():
    for kw in (dict(kv_heads=1), dict(rope_sections=(1,)), dict(cap=3.0), dict(distance=True)):
        with pytest.raises(ValueError):
            EQViTBlock(8, 2, 4, device="cpu", **kw)
    with pytest.raises(ValueError):
        EQViTBlock(8, 2, 4, device="cpu", native=True, kv_heads=3)


def test_grid_positions():
    p = grid_positions(2, 3, lead=1, device="cpu")
    assert p.tolist() == [[0, 0], [0, 0], [0, 1], [0, 2], [1, 0], [1, 1], [1, 2]]
    assert grid_positions(2, 2, frames=3, device="cpu").shape == (12, 3)


def test_functions_refuse():
    x = torch.zeros(4, 2, 32)
    plan = eqlin.Rope(4, 8, (2, 2))
    with pytest.raises(ValueError):
        ops.rotary(x, torch.zeros(4, 2, requires_grad=True), plan)
    with pytest.raises(ValueError):
        ops.rotary(x, torch.zeros(3, 2), plan)
    with pytest.raises(ValueError):
        ops.rotary(x, torch.zeros(4, 3), plan)
    with pytest.raises(ValueError):
        ops.rotary(x, torch.zeros(2, 2), plan)           # a grid repeats over leading dimensions, not within one
    with pytest.raises(ValueError):
        ops.qkv_attention(torch.zeros(4, 6, 32), 2, plan=plan, pos=torch.zeros(2, 2))
    with pytest.raises(ValueError):                      # packed documents need a position for every token
        ops.qkv_attention(torch.zeros(4, 6, 32), 2, plan=plan, pos=torch.zeros(2, 2), docs=2,
                          offsets=torch.tensor([0, 2, 4], dtype=torch.int32))
    with pytest.raises(TypeError):
        ops.rotary(x, torch.zeros(4, 2), plan)           # not on a GPU
    with pytest.raises(ValueError):
        ops.qkv_attention(x, 2)
    with pytest.raises(ValueError):
        ops.qkv_attention(torch.zeros(4, 6, 32), 2, plan=plan)
    with pytest.raises(ValueError):
        ops.qkv_attention(torch.zeros(4, 6, 16), 2, plan=plan, pos=torch.zeros(4, 2))
    with pytest.raises(ValueError):
        ops.group_layer_norm(torch.zeros(2, 32), torch.ones(8), torch.ones(8), 4, res=torch.zeros(1, 32))
    with pytest.raises(ValueError):
        ops.attention(torch.zeros(4, 32), torch.zeros(4, 32), torch.zeros(4, 32))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,tol", [(torch.bfloat16, TOL_BLOCK), (torch.float16, TOL_BLOCK), (torch.float32, TOL_F32)])
@pytest.mark.parametrize("T,opts", [(4, {}), (4, dict(cap=0.0)), (2, dict(rope_sections=(1, 2, 1))), (8, dict(distance=True))])
def test_native_block_against_plain(T, opts, dtype, tol):
    blk = make(dtype, T=T, **opts)
    axes = 3 if opts.get("rope_sections") == (1, 2, 1) else 2
    B, L = 3, 49
    g = torch.Generator().manual_seed(2)
    x = torch.randn((B, L, 32 * T), generator=g).to(dtype).cuda().requires_grad_(True)
    gy = torch.randn((B, L, 32 * T), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 7, (L, axes), generator=g).float().cuda()
    y = blk(x, pos)
    got = grads(blk, x, y, gy)
    ref_dt = torch.float64 if dtype == torch.float32 else torch.float32
    xr = x.detach().to(ref_dt).requires_grad_(True)
    yr = plain_block(blk, xr.view(B * L, -1), pos.repeat(B, 1), [L] * B, ref_dt)
    want = grads(blk, xr, yr, gy.to(ref_dt).view(B * L, -1))
    assert rel(y.view(B * L, -1), yr) <= tol
    for n in got:
        assert rel(got[n], want[n]) <= tol, n
    for layer in (blk.qkv, blk.proj, blk.fc1, blk.fc2):
        assert eqlin.get_error(layer.h) == 0


@pytest.mark.gpu
def test_native_block_packed_and_padded():
    dtype = torch.bfloat16
    blk = make(dtype)
    lens, tail = [49, 1, 130, 64], 12
    g = torch.Generator().manual_seed(4)
    N = sum(lens)
    x = torch.randn((N + tail, 128), generator=g).to(dtype).cuda().requires_grad_(True)
    gy = torch.randn((N + tail, 128), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 9, (N + tail, 2), generator=g).float().cuda()
    off = torch.tensor([0, 49, 50, 180, 244], dtype=torch.int32, device="cuda")
    y = blk(x, pos, offsets=off, max_len=130)
    got = grads(blk, x, y, gy)
    xr = x.detach().float().requires_grad_(True)
    yr = plain_block(blk, xr, pos, lens, torch.float32)
    want = grads(blk, xr, yr, gy.float())
    assert rel(y, yr) <= TOL_BLOCK
    for n in got:
        assert rel(got[n], want[n]) <= TOL_BLOCK, n
    # an image alone gives what it gives in the pack, bit for bit
    with torch.no_grad():
        alone = blk(x[50:180].view(1, 130, -1), pos[50:180])
        assert torch.equal(alone[0], blk(x, pos, offsets=off)[50:180])


@pytest.mark.gpu
def test_native_block_commutes_with_group_shift():
    T = 4
    blk = make(torch.bfloat16)
    g = torch.Generator().manual_seed(6)
    x = torch.randn((2, 60, 128), generator=g).bfloat16().cuda()
    pos = torch.randint(0, 8, (60, 2), generator=g).float().cuda()

    def roll(a, r):
        return a.view(*a.shape[:-1], -1, T).roll(r, -1).reshape(a.shape)

    with torch.no_grad():
        y = blk(x, pos)
        for r in range(1, T):
            assert rel(blk(roll(x, r), pos), roll(y, r)) <= 2e-2


@pytest.mark.gpu
def test_native_block_trains_inside_a_graph():
    blk = make(torch.bfloat16)
    g = torch.Generator().manual_seed(7)
    x = torch.randn((2, 49, 128), generator=g).bfloat16().cuda().requires_grad_(True)
    gy = torch.randn((2, 49, 128), generator=g).bfloat16().cuda()
    pos = grid_positions(7, 7)
    want = [t.clone() for t in grads(blk, x, blk(x, pos), gy).values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        grads(blk, x, blk(x, pos), gy)
        with torch.cuda.graph(graph, stream=side):
            outs = list(grads(blk, x, blk(x, pos), gy).values())
    torch.cuda.current_stream().wait_stream(side)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.gpu
def test_norm_module_with_residual_and_unused_outputs():
    n = GroupLayerNorm(24, 4, native=True)
    m = GroupLayerNorm(24, 4)
    g = torch.Generator().manual_seed(1)
    x, r, gy = (torch.randn((5, 7, 96), generator=g).bfloat16().cuda().requires_grad_(True) for _ in range(3))
    y, s = n(x, r)
    y2, s2 = m(x, r)
    assert torch.equal(s, s2) and rel(y, y2) <= 2e-2
    # only the sum used: the gradient passes through; only the norm used: both inputs get the same
    dx, dr = torch.autograd.grad(s, (x, r), gy.detach(), retain_graph=True)
    assert torch.equal(dx, gy) and torch.equal(dr, gy)
    dx, dr = torch.autograd.grad(y, (x, r), gy.detach())
    assert torch.equal(dx, dr)
    assert rel(dx, torch.autograd.grad(y2, x, gy.detach())[0]) <= 2e-2
    # a slice along the tokens and a transposed gradient
    z = ops.group_layer_norm(x[:, ::2], n.weight, n.bias, 4)
    dz = torch.autograd.grad(z, x, gy.detach()[:, ::2].transpose(0, 1).contiguous().transpose(0, 1))[0]
    assert rel(dz[:, ::2], torch.autograd.grad(m(x[:, ::2]), x, gy.detach()[:, ::2])[0][:, ::2]) <= 2e-2
    assert not dz[:, 1::2].any()
    with pytest.raises(RuntimeError):     # first derivatives only
        a = ops.group_layer_norm(x, n.weight, n.bias, 4)
        (d,) = torch.autograd.grad(a, x, gy, create_graph=True)
        d.sum().backward()


@pytest.mark.gpu
def test_rotary_and_attention_functions_take_any_strides():
    g = torch.Generator().manual_seed(3)
    plan = eqlin.Rope(4, 8, (2, 1))
    x = torch.randn((2, 3, 50, 32), generator=g).bfloat16().cuda().requires_grad_(True)   # heads before tokens
    pos = grid_positions(5, 10)
    v = x.transpose(1, 2)
    y = ops.rotary(v, pos, plan)
    w = ops.rotary(v.contiguous(), pos, plan)
    assert torch.equal(y, w)
    back = ops.rotary(y, pos, plan, inverse=True)
    assert rel(back, v) <= 1e-2
    gy = torch.randn(y.shape, generator=g).bfloat16().cuda()
    (dx,) = torch.autograd.grad(y, x, gy)
    assert torch.equal(dx.transpose(1, 2), ops.rotary(gy, pos, plan, inverse=True))
    q, k, u = (t.reshape(100, 3, 32) for t in (y.detach(), v.detach(), w.detach()))
    odd = torch.empty((100, 3 * 32 + 1), dtype=q.dtype, device="cuda")
    qs = odd.as_strided((100, 3, 32), (97, 32, 1), 1)
    qs.copy_(q)
    a = [t.clone().requires_grad_(True) for t in (q, k, u)]
    b = [qs.requires_grad_(True), a[1], a[2]]
    o1, o2 = ops.attention(*a, docs=2), ops.attention(*b, docs=2)
    assert torch.equal(o1, o2)
    go = torch.randn(o1.shape, generator=g).bfloat16().cuda()
    for d1, d2 in zip(torch.autograd.grad(o1, a, go), torch.autograd.grad(o2, b, go.transpose(1, 2).contiguous().transpose(1, 2))):
        assert torch.equal(d1, d2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_than_2_to_the_31_elements(dtype):
    # images are independent: the last ones of a long batch come out as they do alone, bit for bit
    T, Ch, H, L, images, tail = 4, 16, 12, 197, 4800, 3
    D = Ch * T
    assert images * L * 3 * H * D > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(8)
    plan = eqlin.Rope(T, Ch, (4, 4))
    kw = dict(plan=plan, pos=grid_positions(14, 14, lead=1), slopes=torch.full((H,), 0.1, device="cuda"), cap=20.0)
    qkv = torch.randn((images * L, 3 * H, D), generator=g, device="cuda", dtype=dtype)
    last = qkv[-tail * L:].clone()
    outs = []
    for x, n in ((qkv, images), (last, tail)):
        x.requires_grad_(True)
        o = ops.qkv_attention(x, H, docs=n, **kw)
        go = torch.zeros_like(o)
        go[-tail * L:] = torch.linspace(-1, 1, D, device="cuda")
        o.backward(go)
        outs.append([o[-tail * L:].detach().clone(), x.grad[-tail * L:].clone()])
        x.grad = None
    assert all(torch.equal(a, b) for a, b in zip(*outs)) and torch.isfinite(outs[0][1]).all()
    del x, o, go
    Cp, rows = H * 3 * Ch, 50
    w, b = (torch.randn(Cp, generator=g, device="cuda", dtype=dtype) for _ in range(2))
    feats = qkv.detach().view(images * L, Cp * T)
    y = ops.group_layer_norm(feats, w, b, T)
    assert torch.equal(y[-rows:], ops.group_layer_norm(feats[-rows:].clone(), w, b, T))


@pytest.mark.gpu
def test_two_threads_on_two_streams():
    from concurrent.futures import ThreadPoolExecutor
    plan = eqlin.Rope(4, 8, (2, 2))
    g = torch.Generator().manual_seed(2)
    pos, slopes = grid_positions(9, 11), torch.tensor([0.5, 0.25, 0.125], device="cuda")
    w, c = (torch.randn(72, generator=g).bfloat16().cuda().requires_grad_(True) for _ in range(2))
    xs = [torch.randn((b, 99, 288), generator=g).bfloat16().cuda() for b in (2, 5)]
    torch.cuda.synchronize()

    def run(x):
        with torch.cuda.stream(torch.cuda.Stream()):
            outs = []
            for _ in range(20):
                x = x.detach().requires_grad_(True)
                h = ops.group_layer_norm(x, w, c, 4).reshape(-1, 9, 32)
                y = ops.qkv_attention(h, 3, plan=plan, pos=pos, slopes=slopes, docs=x.shape[0], cap=20.0)
                outs.append((y.detach(), *torch.autograd.grad(y.float().square().sum(), (x, w, c))))
            torch.cuda.current_stream().synchronize()
            return outs

    alone = [run(x)[0] for x in xs]
    with ThreadPoolExecutor(2) as pool:
        for want, got in zip(alone, pool.map(run, xs)):
            assert all(torch.equal(a, b) for once in got for a, b in zip(once, want))


@pytest.mark.gpu
@pytest.mark.parametrize("changed", ["offsets", "pos", "slopes"])
def test_shared_tensors_changed_before_the_backward_are_refused(changed):
    g = torch.Generator().manual_seed(4)
    t = dict(offsets=torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda"), pos=grid_positions(5, 10),
             slopes=torch.tensor([0.5, 0.25], device="cuda"))
    qkv = torch.randn((50, 6, 32), generator=g).bfloat16().cuda().requires_grad_(True)
    for run in (lambda: ops.qkv_attention(qkv, 2, **t), lambda: ops.attention(qkv[:, :2], qkv[:, 2:4], qkv[:, 4:], **t)):
        o = run()
        o.sum().backward(retain_graph=True)
        t[changed].mul_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            o.sum().backward()


@pytest.mark.gpu
def test_attention_on_another_stream_and_wait_limit():
    N, H, D = 300, 2, 64
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((N, H, D), generator=g).bfloat16().cuda() for _ in range(3))
    o1, l1 = torch.empty_like(q), torch.empty((H, N), device="cuda")
    o2, l2 = torch.empty_like(q), torch.empty((H, N), device="cuda")
    eqlin.attention_forward(q, k, v, o1, l1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    eqlin.attention_forward(q, k, v, o2, l2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    # a wait that runs out is recorded and the kernel returns
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    eqlin.attention_forward(q, k, v, o2, l2, err=err, wait_limit=1)
    torch.cuda.synchronize()
    status = err.tolist()
    assert status[0] in (0, 1) and (status[0] == 0 or status[1] >> 8 == 4)
    eqlin.attention_forward(q, k, v, o2, l2)
    torch.cuda.synchronize()
    assert torch.equal(o1, o2)


@pytest.mark.gpu
def test_block_command_times_the_native_block(capsys):
    import json

    from group_circulant_linear_b200 import block
    block.main(["--native", "--model", "eq-vit-s", "--batch", "2", "--iters", "2", "--warmup", "1"])
    out = json.loads(capsys.readouterr().out)
    assert out["native_fwd_ms"] > 0 and out["native_fwd_bwd_ms"] > 0


@pytest.mark.gpu
def test_native_block_deepcopy_and_16_bit_cast():
    import copy
    blk = make(torch.bfloat16)
    twin = copy.deepcopy(blk).to(torch.bfloat16)
    assert twin.slopes.dtype == torch.float32 and torch.equal(twin.slopes, blk.slopes)
    x = torch.randn((1, 20, 128), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    with torch.no_grad():
        assert torch.equal(blk(x, grid_positions(4, 5)), twin(x, grid_positions(4, 5)))
