"""From how many requests on the other row is read, as include/kvq.h states it for one query token: at that number a
request's own entries of the shared pages are never looked at, one below it the leader's are looked at for itself
alone."""
import pytest

import fp8_quantised_paged_kv_gb300 as kvq
import view_ref as R
from test_gpu_prefix import Case

pytestmark = pytest.mark.gpu

# (cache, fp32 output, heads per group, query tokens, requests)
BORDERS = [("fp8", False, 1, 1, 3), ("fp8", False, 8, 1, 3), ("fp8", True, 4, 1, 4), ("fp8", True, 5, 1, 5),
           ("blocks", False, 6, 1, 3), ("blocks", False, 7, 1, 4), ("blocks", True, 1, 1, 5), ("blocks", True, 8, 1, 5),
           ("bf16", False, 1, 1, 2), ("bf16", False, 8, 1, 2), ("bf16", True, 1, 1, 3), ("bf16", True, 8, 1, 3),
           ("fp8", False, 8, 4, 2), ("bf16", True, 8, 4, 2)]  # 32 query rows: own rows are read twice


@pytest.mark.parametrize("kind,fp32,g,n,border", BORDERS)
def test_where_the_other_row_begins_to_serve(kind, fp32, g, n, border):
    kvq.kvq_device_error(clear=True)
    for count in (border, border - 1):
        c = Case(kind, [(320, [20, 21, 19, 40, 9][:count]), (None, [300])], g, 16, n, poison_own=False)
        if count == 1:                                      # a run of its own row is apart whatever is read
            continue
        bad = c.desc.num_pages + 7
        if count == border:
            c.given[1:count, :20] = bad
        else:
            c.given[0, 3] = bad
        c.upload()
        ref, bound = c.ref(fp32)
        got = c.run(fp32)
        right = list(range(len(c.lens)))
        if count < border:
            right.remove(0)
            assert not got[0].any()
        R.assert_within(got[right], ref[right], bound[right], f"{count} requests")
        assert got[right].any(axis=(1, 2, 3)).all()
    assert kvq.kvq_device_error() == 0
