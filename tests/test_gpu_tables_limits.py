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
