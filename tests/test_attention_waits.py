"""Attention's bounded waits: a wait that runs out is recorded, the kernels give up and return, and the next call is
as ever.  Without polls every wait for a copy or a product runs out, since it is looked at once, as it begins."""
from __future__ import annotations

import pytest
import torch

from group_circulant_linear_b200 import eqlin

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
