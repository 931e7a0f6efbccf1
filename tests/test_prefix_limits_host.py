"""The largest calls over shared prefixes, as include/kvq.h states them: no GPU is needed."""
import pytest

import fp8_quantised_paged_kv_gb300 as kvq

DESC = kvq.CacheDesc(4104, 64, 8, 128)


@pytest.mark.parametrize("batch,n,max_pages", [(2048, 16, 16384), (4096, 16, 8192)])
def test_lines_of_work_that_pass_31_bits_are_refused(batch, n, max_pages):
    """batch x 8 KV heads x 8 blocks of 16 rows x the table's 64-token units, and six more per line."""
    lines = batch * 8 * 8
    assert lines * (max_pages + 6) > 2**31 - 1
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_decode_plan_prefix(DESC, batch, n, 64, max_pages)
    assert e.value.status == 2
    fits = (2**31 - 1) // lines - 200                       # with room for what the SMs hold at a time
    assert lines * (fits + 6) < 2**31
    assert kvq.kvq_decode_plan_prefix(DESC, batch, n, 64, fits) > 0


def test_the_workspace_has_places_for_every_row_twice():
    rows = 65535 * 64
    assert kvq.kvq_decode_plan_prefix(DESC, 65535, 1, 64, 64) > 2 * rows * 516
