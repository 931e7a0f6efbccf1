"""Attention over shared prefixes where the scores' multiplier is zero, or underflows to it, and requests that share
less end between the others' tokens: the outputs are means of V, as kvq_decode_attn_window's are."""
import numpy as np
import pytest

import fp8_quantised_paged_kv_gb300 as kvq
from test_gpu_prefix import KINDS, SCALE, Case

pytestmark = pytest.mark.gpu


def case(kind, times, n=1, seed=0):
    """One prompt of which the requests share 900 tokens, 333, less than a tile, and as much as they hold."""
    kvq.kvq_device_error(clear=True)
    c = Case(kind, [(900, [20, 50, 29, 400, 22] * times)], 5, 16, n, poison_own=False, seed=seed)
    c.shared[:] = (16, 900, 2**31 - 1, 333, 15) * times
    return c


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("times,n", [(3, 1), (9, 1), (3, 4)])     # 75, 225 and 300 rows of a KV head
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-44])             # (1e-44 times a K scale of 0.02 is 0 in fp32)
def test_softmax_scales_of_nothing(kind, times, n, scale):
    c = case(kind, times, n)
    c.upload()
    c.check(scale=scale)


@pytest.mark.parametrize("times", [3, 9])
def test_a_head_whose_k_scale_is_zero(times):
    c = case("fp8", times)
    c.ks[0] = 0.0
    c.upload()
    c.check()


@pytest.mark.parametrize("times", [3, 9])
@pytest.mark.parametrize("exp,scale", [(-48, 1e-30), (-48, -1e-30), (-40, SCALE)])
def test_block_multipliers_that_underflow(times, exp, scale):
    """2^-48 of the keys' exponents, 2^-13 of the query rows' scaling and 1e-30: 0 in fp32."""
    c = case("blocks", times)
    c.ke = np.where(c.ke >= 127, c.ke, np.where(c.ke <= -128, c.ke, exp)).astype(np.int8)
    c.upload()
    c.check(scale=scale)
