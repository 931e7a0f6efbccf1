"""Page tables at the ends of their 32 bits."""
import pytest

torch = pytest.importorskip("torch")

import fp8_quantised_paged_kv_gb300 as kvq
from tests.test_gpu_tables import DEV, i32

pytestmark = pytest.mark.gpu


def test_a_length_stays_within_31_bits():
    """A table of 2^31 tokens and more: the last length that an int32 holds is reached, and not passed."""
    ps, maxp = 128, (1 << 24) + 4
    pool = kvq.PagePool.create(8, ps, device=DEV, tags=False)
    bt = torch.full((1, maxp), -1, dtype=torch.int32, device=DEV)
    seq, refused = i32([2**31 - 200]), torch.empty(1, dtype=torch.uint8, device=DEV)

    def extend(n):
        slots = torch.full((n,), -9, dtype=torch.int64, device=DEV)
        kvq.kvq_extend_tables(pool, None, n, seq, bt, None, slots, refused)
        return refused.item(), seq.item(), pool.free_count.item(), slots.tolist()

    assert extend(200) == (1, 2**31 - 200, 8, [-1] * 200)
    r, length, free, slots = extend(199)                    # 72 tokens of the page that is held, 127 of a new one
    assert (r, length, free) == (0, 2**31 - 1, 7) and slots[72:] == list(range(127))
    assert extend(1) == (1, 2**31 - 1, 7, [-1])


def test_the_largest_pool():
    """2^31 - 1 pages: those given back are found whatever their number."""
    n = 2**31 - 1
    free = torch.empty(n, dtype=torch.int32, device=DEV)
    pages = [7, 2**31 - 33, 2**31 - 2, 0]
    free[:4] = i32(pages)
    pool = kvq.PagePool(n, 16, free, i32([4]), torch.zeros(n, dtype=torch.int32, device=DEV))
    seq, bt = i32([0, 0]), torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    refused = torch.empty(2, dtype=torch.uint8, device=DEV)
    slots = torch.empty(64, dtype=torch.int64, device=DEV)
    kvq.kvq_extend_tables(pool, None, 64, seq, bt, None, slots, refused)
    assert bt[:, :2].flatten().tolist() == pages[::-1] and pool.free_count.item() == 0
    assert slots[16:32].tolist() == list(range((2**31 - 2) * 16, (2**31 - 1) * 16))
    kvq.kvq_trim_tables(pool, i32([0, 0]), seq, bt)
    assert pool.free_count.item() == 4 and free[:4].tolist() == sorted(pages)
    assert not pool.scratch.any() and pool.page_refs[pages].tolist() == [0] * 4
