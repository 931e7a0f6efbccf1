"""The block-scaled attention over exponents outside the append's range: V's
are read as they are within [-48, 48] and as the nearer border outside, K's
from -126 on.  The softmax's denominator is a sum of weights of up to 2^15
times 2^-ev: further down it overflows, and weights of exponents further apart
are flushed before 2^-ev brings them back."""
import numpy as np
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
import view_ref as R
from test_gpu_view import DEV, LENS, SCALE, Case

pytestmark = pytest.mark.gpu
LOWEST, HIGHEST = -48, 48


def _check(c, splits, cut=2.0 ** -40):
    """Against the 64-bit form over the exponents that the header says count."""
    ke, ve = np.maximum(c.ke, -126), np.clip(c.ve, LOWEST, HIGHEST)
    for fp32 in (False, True):
        ref, bound = R.attention(c.q_bits, c.k, c.v, c.bt, c.lens, SCALE, c.window, c.sinks, ke=ke, ve=ve,
                                 fp32=fp32, cut=cut)
        assert np.any(ref != 0)
        for s in splits:
            R.assert_within(c.run(fp32, s), ref, bound, f"fp32={fp32} splits={s}")
    assert kvq.kvq_device_error() == 0


@pytest.mark.parametrize("n,g,ps", [(1, 4, 16), (3, 5, 32)])
@pytest.mark.parametrize("ev", [-128, -126, -120, -113, -112, -105, -99, -98, -97, -60])
def test_low_exponents_of_v(ev, n, g, ps):
    _check(Case("blocks", LENS, g, ps, n, 0, 0, seed=21, ev=(ev, ev)), (0, 1, 5, 12))


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 20)])
def test_low_exponents_among_others(window, sinks):
    _check(Case("blocks", LENS, 3, 16, 1, window, sinks, seed=22, ev=(-128, -90)), (0, 1, 5))
    _check(Case("blocks", LENS, 3, 16, 2, window, sinks, seed=23, ev=(-128, 60)), (0, 1, 5))


def test_low_exponents_shared_on_the_device():
    _check(Case("blocks", LENS, 4, 16, 1, 0, 0, seed=24, ev=(-128, -112), padded=True), (0,))


@pytest.mark.parametrize("ev", [(-128, -112), (-98, -98), (-128, 40)])
def test_low_exponents_in_tensor_memory(ev):
    c = Case("blocks", (5000, 0, 40, 4097, 1, 130, 2500, 9000), 8, 16, 8, 0, 0, hkv=8, seed=25, ev=ev)
    _check(c, (0, 1, 5), 2.0 ** -32)


@pytest.mark.parametrize("n,g,hkv", [(1, 8, 1), (2, 8, 1), (8, 8, 8)])
@pytest.mark.parametrize("ev", [-98, -128])
def test_a_full_split_of_the_largest_weights(ev, n, g, hkv):
    """8,192 tokens of one split whose scores are all but equal."""
    c = Case("blocks", [8192], g, 128, n, 0, 0, hkv=hkv, seed=26, ev=(ev, ev))
    c.ke = np.full_like(c.ke, -60)
    c.d["s0"] = torch.from_numpy(c.ke).to(DEV)
    _check(c, (1,), 2.0 ** -32 if n * g > 16 else 2.0 ** -40)


@pytest.mark.parametrize("n,g", [(1, 4), (3, 5)])
def test_low_exponents_of_k(n, g):
    c = Case("blocks", LENS, g, 16, n, 0, 0, seed=27)
    c.ke = np.random.default_rng(27).choice([-128, -127, -126, -125], c.ke.shape).astype(np.int8)
    c.d["s0"] = torch.from_numpy(c.ke).to(DEV)
    _check(c, (0, 1, 5))
