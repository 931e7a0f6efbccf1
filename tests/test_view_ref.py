"""The plain implementations that the block-scaled and windowed operators are
tested against, pinned themselves: against the oracle's attention where the
two mean the same, against a dense softmax with the mask written as a loop,
and against closed forms."""
import numpy as np
import pytest

import oracle
import view_ref as R
import workloads as W


def _codes(rng, shape):
    return R.encode(rng.standard_normal(shape) * 60)


@pytest.mark.parametrize("n", [1, 3])
def test_no_window_and_equal_exponents_is_the_oracles_attention(n):
    rng = np.random.default_rng(n)
    lens = np.array([5, 40, 0, 1], np.int32)
    k, v = _codes(rng, (12, 2, 16, 128)), _codes(rng, (12, 2, 16, 128))
    bt = rng.permutation(12).astype(np.int32).reshape(4, 3)
    q = W.normal_bf16(rng, (4, n, 6, 128))
    ke, ve = np.full((12, 2, 1), -6, np.int8), np.full((12, 2, 1), -3, np.int8)
    scale = float(np.float32(0.09))                                  # the oracle takes the scale as fp32
    got, bound = R.attention(q, k, v, bt, lens, scale, 0, 0, ke=ke, ve=ve, fp32=True)
    ks, vs = np.full(2, 2.0 ** -6, np.float32), np.full(2, 2.0 ** -3, np.float32)
    ref = oracle.decode_attn_multi(q, k, v, ks, vs, bt, lens, scale)
    np.testing.assert_allclose(got, ref, rtol=1e-6, atol=1e-9)
    got, _ = R.attention(q, k, v, bt, lens, scale, 0, 0, ks=ks, vs=vs)
    np.testing.assert_allclose(got, ref, rtol=1e-6, atol=1e-9)
    assert np.all(bound >= 0) and np.all(bound[0] < 1e-2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (4, 2), (7, 20), (100, 1)])
def test_window_against_a_loop(window, sinks):
    rng = np.random.default_rng(window)
    L, n = 37, 3
    k, v = _codes(rng, (3, 1, 16, 128)), _codes(rng, (3, 1, 16, 128))
    bt = np.array([[2, 0, 1]], np.int32)
    q = W.normal_bf16(rng, (1, n, 2, 128))
    one = np.full(1, 2.0 ** -6, np.float32)
    got, _ = R.attention(q, k, v, bt, np.array([L]), 0.1, window, sinks, ks=one, vs=one)
    kk = oracle.e4m3_decode(k[[2, 0, 1], 0].reshape(48, 128)) / 64
    vv = oracle.e4m3_decode(v[[2, 0, 1], 0].reshape(48, 128)) / 64
    for i in range(n):
        p = L - n + i
        seen = [j for j in range(p + 1) if j < sinks or j > p - window]
        assert p in seen
        for h in range(2):
            s = np.array([kk[j] @ W.bf16_bits_to_f32(q[0, i, h]).astype(np.float64) * 0.1 for j in seen])
            w = np.exp(s - s.max())
            np.testing.assert_allclose(got[0, i, h], w @ vv[seen] / w.sum(), rtol=1e-12, atol=1e-12)


def test_exponents():
    assert R.exponent(448.0) == 0 and R.exponent(449.0) == 1 and R.exponent(224.0) == -1
    assert R.exponent(0.0) == -48 and R.exponent(1e-30) == -48 and R.exponent(1e30) == 48
    assert R.exponent(float("inf")) == 48 and R.exponent(1.0) == -8 and R.exponent(1.75) == -8
    assert R.exponent(1.76) == -7


def test_append_keeps_values_within_half_a_step_and_moves_old_rows():
    rng = np.random.default_rng(3)
    k, v = np.full((2, 1, 16, 128), 0x7E, np.uint8), np.zeros((2, 1, 16, 128), np.uint8)
    ke, ve = np.zeros((2, 1, 1), np.int8), np.zeros((2, 1, 1), np.int8)
    bt = np.array([[1, 0]], np.int32)
    small, large = W.normal_bf16(rng, (3, 1, 128)), W.f32_to_bf16_bits(rng.standard_normal((1, 1, 128)) * 50)
    R.append_blocks(k, v, ke, ve, small, small, [0, 3], bt, [3])
    assert ke[0, 0, 0] == 0 and np.all(k[0] == 0x7E) and np.all(k[1, 0, 3:] == 0x7E)
    e0 = ke[1, 0, 0]
    R.append_blocks(k, v, ke, ve, large, large, [0, 1], bt, [4])
    assert ke[1, 0, 0] > e0
    got = oracle.e4m3_decode(k[1, 0, :4]) * 2.0 ** float(ke[1, 0, 0])
    want = W.bf16_bits_to_f32(np.concatenate([small, large])[:, 0]).astype(np.float64)
    step = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * 2.0 ** float(ke[1, 0, 0])
    assert np.all(np.abs(got - want)[3] <= step[3])
    assert np.all(np.abs(got - want)[:3] <= 2 * step[:3])          # rounded twice
