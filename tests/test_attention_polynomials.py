"""The polynomials that stand for tanh below a cap: their coefficients, as the kernels have them, against the bounds
that the comments beside them state."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest

from group_circulant_linear_b200 import build


@pytest.mark.parametrize("name,start,limit", [("eqlin_attn_simt.cu", "float tanh_fast(", 0.7),
                                              ("eqlin_attn_tc.cuh", "uint64_t q_small2(", 0.6)])
def test_tanh_polynomials_keep_their_stated_bounds(name, start, limit):
    with open(os.path.join(build.CSRC, name)) as f:
        source = f.read()
    at = source.index(start)
    body = source[at:source.index("\n}", at)]
    c = [float(np.float32(v)) for v in dict.fromkeys(re.findall(r"-?\d\.\d{10,}(?=f)", body))]
    assert len(c) in (5, 6) and abs(c[-1] - 1) < 1e-6        # from the highest power down, in x^2
    note = re.sub(r"\n//", "", source[:at])
    stated, relative = (float(re.findall(p, note)[-1]) for p in
                        (r"(\d\.\de-\d) off at\s+most", r"with them (\d\.\de-\d)\s+relative"))
    x = np.linspace(1e-6, limit, 1000001)
    exact, q = np.tanh(x), np.full_like(x, c[0])
    for k in c[1:]:
        q = q * (x * x) + k
    assert np.abs(q * x - exact).max() <= stated
    # and as the GPU evaluates it: each step rounded to FP32 once
    f = x.astype(np.float32)
    z, q = f * f, np.full_like(f, c[0])
    for k in c[1:]:
        q = (q.astype(np.float64) * z + k).astype(np.float32)
    exact = np.tanh(f.astype(np.float64))
    assert (np.abs(q * f - exact) / exact).max() <= relative
