"""kvq_append_blocks with token offsets that do not fit: ascending ones that
start below 0 or end past the tokens skip the requests concerned and no other;
where offsets descend, requests are lost, but every block is left as it was or
becomes what the request's own tokens make of it."""
import numpy as np
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
import view_ref as R
from test_gpu_blocks import _caches, _values, bf, t

pytestmark = pytest.mark.gpu


class Batch:
    def __init__(self, B, hkv, ps, most, seed):
        rng = np.random.default_rng([B, hkv, ps, seed])
        self.desc_of = lambda n: kvq.CacheDesc(n, ps, hkv)
        self.ps, self.hkv = ps, hkv
        self.counts = rng.integers(0, most + 1, B).astype(np.int32)
        self.lens = (self.counts + rng.integers(0, 40, B)).astype(np.int32)
        maxp = -(-int(self.lens.max()) // ps)
        self.N = B * maxp
        self.bt = rng.permutation(self.N).reshape(B, maxp).astype(np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(self.counts)]).astype(np.int64)
        self.T = int(self.offsets[-1])
        self.new = [_values(rng, (self.T, hkv, 128), "normal") for _ in range(2)]
        self.caches = _caches(rng, self.N, hkv, ps)

    def run(self, offsets):
        """(caches after the call, after view_ref's), numpy."""
        dev = [t(x) for x in self.caches]
        kvq.kvq_append_blocks(self.desc_of(self.N), *(bf(x) for x in self.new), t(offsets.astype(np.int32)),
                              t(self.bt), t(self.lens), None, *dev)
        torch.cuda.synchronize()
        ref = [x.copy() for x in self.caches]
        R.append_blocks(*ref, *self.new, offsets, self.bt, self.lens)
        out = [x.cpu().numpy() for x in dev]
        return [np.where(x == 0xFF, 0x7F, x) if x.dtype == np.uint8 else x for x in out], \
            [np.where(x == 0xFF, 0x7F, x) if x.dtype == np.uint8 else x for x in ref]


@pytest.mark.parametrize("B,hkv,ps,most", [(300, 1, 16, 9), (40, 2, 32, 60), (9, 5, 64, 200)])
def test_ascending_offsets_outside_the_tokens(B, hkv, ps, most):
    b = Batch(B, hkv, ps, most, 1)
    for offsets in (b.offsets - 3, b.offsets - b.T // 2, b.offsets + 7, b.offsets + b.T // 3, b.offsets * 1000,
                    b.offsets * 3 - b.T, np.full(B + 1, -2**31), np.full(B + 1, 2**31 - 1)):
        got, ref = b.run(offsets)
        for name, x, y in zip(("k", "v", "k_exp", "v_exp"), got, ref):
            assert np.array_equal(x, y), (name, int(offsets[0]), int(offsets[-1]))


@pytest.mark.parametrize("B,hkv,ps,most", [(300, 1, 16, 9), (40, 2, 32, 60), (9, 5, 64, 200)])
def test_descending_offsets_write_nothing_else(B, hkv, ps, most):
    """A block (16 rows and the exponent of a KV head) is as before or as the
    request's tokens make it; the requests whose own offsets descend keep
    everything."""
    b = Batch(B, hkv, ps, most, 2)
    rng = np.random.default_rng(B)
    for kind in range(4):
        offsets = b.offsets.copy()
        if kind == 0:                                       # one step back by a third of the tokens
            offsets[B // 2:] = np.maximum(offsets[B // 2:] - b.T // 3, 0)
        elif kind == 1:
            offsets = offsets[::-1].copy()
        elif kind == 2:
            offsets = rng.integers(-50, b.T + 50, B + 1)
        else:
            offsets[B // 3] = 2**31 - 1
        got, ref = b.run(offsets)
        old = [np.where(x == 0xFF, 0x7F, x) if x.dtype == np.uint8 else x for x in b.caches]
        for c, e in ((0, 2), (1, 3)):
            shape = (b.N, hkv, ps // 16, 16 * 128)
            same = lambda x: (np.all(got[c].reshape(shape) == x[c].reshape(shape), axis=3)  # noqa: E731
                              & (got[e] == x[e]))
            assert np.all(same(old) | same(ref)), kind
