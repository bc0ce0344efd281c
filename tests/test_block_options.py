"""What goes with the options of ``EQViTBlock``: what they refuse, empty batches."""
from __future__ import annotations

import pytest
import torch
import torch.nn as nn

from group_circulant_linear_b200.block import DenseEQViTBlock, EQViTBlock


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
