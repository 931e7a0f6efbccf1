"""Windowed attention over a bf16 cache whose values lie far from 1: the
weights of a bf16 cache are bf16 numbers of at most 1 (no f16 range to fit
into), so the weighted sum is no larger than the values' own sum."""
import numpy as np
import pytest
import torch

import view_ref as R
import workloads as W
from test_gpu_view import DEV, SCALE, Case

pytestmark = pytest.mark.gpu
# 300 values of at most 6 * 2^117 sum up to 2^128 at most: inside fp32
LENS = (1, 0, 17, 33, 100, 300)


@pytest.mark.parametrize("n,g,ps", [(1, 8, 16), (3, 4, 64), (9, 8, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
@pytest.mark.parametrize("power", [-100, 112, 117])
def test_values_of_a_bf16_cache(power, window, sinks, n, g, ps):
    c = Case("bf16", LENS, g, ps, n, window, sinks, seed=31)
    v = W.bf16_bits_to_f32(c.v).astype(np.float64) * 2.0 ** power
    v = np.where(np.isnan(v), np.nan, np.clip(v, -6 * 2.0 ** power, 6 * 2.0 ** power))
    with np.errstate(invalid="ignore"):
        c.v = W.f32_to_bf16_bits(v.astype(np.float32))      # what no query sees stays NaN
    c.d["v"] = torch.from_numpy(c.v.view(np.int16)).to(DEV).view(torch.bfloat16)
    for fp32 in (False, True):
        ref, bound = R.attention(c.q_bits, c.k, c.v, c.bt, c.lens, SCALE, window, sinks, fp32=fp32)
        assert np.all(np.isfinite(ref)) and np.abs(ref).max() > 2.0 ** power
        for s in (0, 1, 2, 5):
            R.assert_within(c.run(fp32, s), ref, bound, f"fp32={fp32} splits={s}")
