"""kvq_copy_pages leaves alone what it is not given: exponent arrays that are
not listed, the pages of no pair, the memory around the arrays."""
import numpy as np
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = 4096


def _guarded(shape, dtype):
    """A tensor of random bytes inside a larger buffer of them, and the buffer."""
    size = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    whole = torch.randint(0, 256, (GUARD + size + GUARD,), dtype=torch.uint8, device=DEV)
    return whole[GUARD:GUARD + size].view(dtype).view(shape), whole


@pytest.mark.parametrize("ps,hkv,bf16,listed_exps", [(16, 1, False, 2), (16, 3, False, 1), (64, 5, True, 0),
                                                     (128, 8, False, 0), (32, 3, False, 2)])
@pytest.mark.parametrize("n", [0, 1, 33])
def test_copies_what_is_listed_only(ps, hkv, bf16, listed_exps, n):
    rng = np.random.default_rng([ps, hkv, n])
    N = 2 * n + 3
    desc = kvq.CacheDesc(N, ps, hkv, 128, kvq.KVQ_CACHE_BF16 if bf16 else kvq.KVQ_CACHE_FP8_E4M3)
    caches = [_guarded((N, hkv, ps, 128), torch.bfloat16 if bf16 else torch.uint8) for _ in range(3)]
    exps = [_guarded((N, hkv, ps // 16), torch.int8) for _ in range(3)]
    before = [whole.clone() for _, whole in caches + exps]
    perm = rng.permutation(N).astype(np.int32)
    src, dst = perm[:n].copy(), perm[n:2 * n].copy()
    kvq.kvq_copy_pages(desc, [x for x, _ in caches[:2]], [x for x, _ in exps[:listed_exps]],
                       torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV))
    torch.cuda.synchronize()
    for i, (old, (x, whole)) in enumerate(zip(before, caches + exps)):
        want = old.clone()
        if i < 2 or 3 <= i < 3 + listed_exps:
            page = x[0].numel() * x.element_size()
            rows = want[GUARD:-GUARD].view(N, page)
            rows[torch.from_numpy(dst).long().to(DEV)] = rows[torch.from_numpy(src).long().to(DEV)]
        assert torch.equal(whole, want), i
