"""What goes with the options of ``EQViTBlock``: what they refuse, empty batches."""
from __future__ import annotations

import pytest
import torch
import torch.nn as nn

from group_circulant_linear_b200 import ops
from group_circulant_linear_b200.block import DenseEQViTBlock, EQViTBlock, grid_positions


def bare(**kw):
    """A block without its layers, which need a GPU."""
    blk = EQViTBlock.__new__(EQViTBlock)
    nn.Module.__init__(blk)
    for name, value in {**dict(heads=4, kv_heads=4, rope=None, cap=0.0, slopes=None, native=True), **kw}.items():
        setattr(blk, name, value)
    return blk


@pytest.mark.parametrize("option", [dict(kv_heads=2), dict(rope=object()), dict(cap=5.0), dict(slopes=torch.ones(4))])
def test_dense_block_refuses_what_it_does_not_compute(option):
    with pytest.raises(ValueError, match="dense block"):
        DenseEQViTBlock(bare(**option))
    DenseEQViTBlock(bare())
    DenseEQViTBlock(bare(native=False))


def test_positions_of_an_empty_batch():
    grid = torch.zeros((49, 2))
    for pos in (grid, grid.expand(0, 49, 2), grid[:0]):
        assert ops._flat_pos(pos, 0, 2, 0).shape == (0, 2)
    with pytest.raises(ValueError, match="axes"):
        ops._flat_pos(grid, 0, 3, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead", [(0, 49), (3, 0), (0,)])
def test_an_empty_batch_runs_both_ways(lead, dtype):
    blk = EQViTBlock(32, 4, 4, dtype=dtype, native=True, kv_heads=2, rope_sections=(2, 2), cap=8.0, distance=True)
    x = torch.empty((*lead, 128), dtype=dtype, device="cuda", requires_grad=True)
    kw = dict(offsets=torch.zeros(1, dtype=torch.int32, device="cuda")) if len(lead) == 1 else {}
    y = blk(x, grid_positions(7, lead[-1] // 7) if len(lead) == 2 else torch.empty((0, 2), device="cuda"), **kw)
    assert y.shape == x.shape
    grads = torch.autograd.grad(y, [x, *blk.parameters()], torch.empty_like(y))
    assert grads[0].shape == x.shape and not any(g.any() for g in grads[1:])


def test_the_attention_record_is_kept_for_each_device(monkeypatch):
    import copy

    from group_circulant_linear_b200 import eqlin

    blk = bare(errs={})
    for name in ("qkv", "proj", "fc1", "fc2"):
        object.__setattr__(blk, name, type("Layer", (), {"h": None}))
    monkeypatch.setattr(eqlin, "get_error", lambda h: 0)
    cpu, meta = torch.device("cpu"), torch.device("meta")
    err = blk._err(cpu)
    assert blk._err(cpu) is err and blk._err(meta) is not err and blk._err(cpu) is err
    del blk.errs[meta]
    assert blk.get_error() == 0
    err[0] = 1
    twin = copy.deepcopy(blk.errs)
    assert blk.get_error() == -6 and blk.get_error() == 0 and int(twin[cpu][0]) == 1
