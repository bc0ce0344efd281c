"""Attention's bounded waits: a wait that runs out is recorded, the kernels give up and return, and the next call is
as ever.  Without polls every wait for a copy or a product runs out, since it is looked at once, as it begins."""
from __future__ import annotations

import pytest
import torch

from group_circulant_linear_b200 import block, eqlin, ops
from group_circulant_linear_b200.block import EQViTBlock

FWD, DQ = 4, 5                            # kernels in the record


def tensors(lens, H, K, D, dtype, axes):
    g = torch.Generator().manual_seed(D + axes)
    N = sum(lens)
    q, go = (torch.randn((N, H, D), generator=g).to(dtype).cuda() for _ in range(2))
    k, v = (torch.randn((N, K, D), generator=g).to(dtype).cuda() for _ in range(2))
    kw = dict(offsets=torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda"))
    if axes:
        kw.update(pos=torch.randint(0, 20, (N, axes), generator=g).float().cuda(), slopes=torch.full((H,), 0.1, device="cuda"))
    return q, k, v, go, kw


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,H,K,D,cap,axes", [
    ([300], 2, 2, 64, 0.0, 0), ([1100, 13, 700], 2, 1, 64, 0.0, 0), ([1100, 13, 700], 2, 1, 128, 8.0, 2),
    ([7, 90, 1, 33, 200] * 4, 3, 1, 40, 8.0, 1), ([49] * 300, 3, 3, 32, 0.0, 2)])
def test_a_wait_that_runs_out_is_recorded_and_harmless(lens, H, K, D, cap, axes, dtype):
    q, k, v, go, kw = tensors(lens, H, K, D, dtype, axes)
    N = q.shape[0]

    def outputs():
        return [torch.full_like(t, 9.0) for t in (q, q, k, v)] + [torch.full((H, N), 9.0, device="cuda") for _ in range(2)]

    def run(o, dq, dk, dv, lse, delta, fwd, bwd):
        eqlin.attention_forward(q, k, v, o, lse, cap=cap, **fwd, **kw)
        eqlin.attention_backward(go, q, k, v, o, lse, dq, dk, dv, delta, cap=cap, **bwd, **kw)

    want, e = outputs(), torch.zeros(4, dtype=torch.int32, device="cuda")
    run(*want, dict(err=e), dict(err=e))
    torch.cuda.synchronize()
    assert not e.any()

    ef, eb = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(2))
    given_up = outputs()
    none = dict(wait_limit=eqlin.NO_POLLS)
    run(*given_up, dict(err=ef, **none), dict(err=eb, **none))
    torch.cuda.synchronize()
    for err, kernel in ((ef, FWD), (eb, DQ)):
        status, site, _, polls = err.tolist()
        assert status == 1 and site >> 8 == kernel and polls == 0
    # every row warp gave up before its scores, in the kernel for dk and dv, too
    assert all(bool((t == 9.0).all()) for t in given_up)
    # without a record they give up just so
    run(*given_up, none, none)
    torch.cuda.synchronize()
    assert all(bool((t == 9.0).all()) for t in given_up)

    after = outputs()
    run(*after, dict(err=e), dict(err=e))
    torch.cuda.synchronize()
    assert not e.any() and all(torch.equal(a, b) for a, b in zip(want, after))


@pytest.mark.gpu
def test_waits_of_calls_that_give_up_do_not_disturb_others():
    # the same tensors from two streams, one of which gives up every time
    lens, H, K, D = [500, 64, 130], 4, 2, 64
    q, k, v, _, kw = tensors(lens, H, K, D, torch.bfloat16, 0)
    o, lse = torch.empty_like(q), torch.empty((H, q.shape[0]), device="cuda")
    eqlin.attention_forward(q, k, v, o, lse, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other, l2, e = torch.empty_like(q), torch.empty_like(lse), torch.zeros(4, dtype=torch.int32, device="cuda")
    mine, l3, e3 = torch.empty_like(q), torch.empty_like(lse), torch.zeros(4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        eqlin.attention_forward(q, k, v, other, l2, err=e, wait_limit=eqlin.NO_POLLS, stream=side, **kw)
        eqlin.attention_forward(q, k, v, mine, l3, err=e3, **kw)
    torch.cuda.synchronize()
    assert int(e[0]) == 1 and not e3.any() and torch.equal(o, mine) and torch.equal(lse, l3)


def without_polls(monkeypatch):
    """Give every attention call no polls for its waits."""
    desc = eqlin._attention_desc
    monkeypatch.setattr(eqlin, "_attention_desc", lambda *a: desc(*a[:-1], eqlin.NO_POLLS))


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [False, True])
def test_functions_record_a_wait_that_runs_out(packed, monkeypatch):
    err = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.randn((90, 6, 32), device="cuda").bfloat16().requires_grad_(True)
    run = (lambda: ops.qkv_attention(x, 2, err=err)) if packed else \
        (lambda: ops.attention(x[:, :2], x[:, 2:4], x[:, 4:], err=err))
    o = run()
    o.sum().backward()
    assert eqlin.attention_error(err) == 0
    with monkeypatch.context() as m:
        without_polls(m)
        run()
        assert eqlin.attention_error(err) == -6 and eqlin.attention_error(err) == 0
        o = run()
        assert eqlin.attention_error(err) == -6
        o.sum().backward()                # the backward records it, too
        assert eqlin.attention_error(err) == -6
    assert torch.equal(run(), run()) and eqlin.attention_error(err) == 0


@pytest.mark.gpu
def test_the_block_reports_a_wait_that_runs_out(monkeypatch):
    import copy

    blk = EQViTBlock(32, 4, 4, native=True)
    twin = copy.deepcopy(blk)
    x = torch.randn((2, 60, 128), device="cuda").bfloat16()
    blk(x)
    assert blk.get_error() == 0
    with monkeypatch.context() as m:
        without_polls(m)
        blk(x)
        assert twin.get_error() == 0 and blk.get_error() == -6 and blk.get_error() == 0
        with pytest.raises(RuntimeError, match="timeout"):
            block.main(["--native", "--model", "eq-vit-s", "--batch", "2", "--iters", "1", "--warmup", "1"])
    blk(x)
    assert blk.get_error() == 0 and EQViTBlock(32, 4, 4).get_error() == 0


def test_attention_error_takes_a_record():
    assert eqlin.attention_error(torch.zeros(4, dtype=torch.int32)) == 0
    err = torch.tensor([1, 1040, 0, 0], dtype=torch.int32)
    assert eqlin.attention_error(err) == -6 and not err.any()
    for bad in (None, torch.zeros(3, dtype=torch.int32), torch.zeros(4)):
        with pytest.raises(TypeError):
            eqlin.attention_error(bad)
