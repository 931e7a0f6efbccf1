"""Page tables: the plain model against counts worked by hand, and the calls' refusals, which need no GPU."""
import ctypes

import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
from tests.tables_ref import Tables


def test_the_model_by_hand():
    t = Tables(8, 16, 3, 4)
    slots, refused = t.extend([0, 17, 17, 20], 20)          # 17, 0 and 3 tokens: pages 0, 1 and 2
    assert refused == [0, 0, 0] and t.seq == [17, 0, 3] and t.count == 5
    assert t.rows[0][:2] == [0, 1] and t.rows[2][0] == 2
    assert slots[:2] == [0, 1] and slots[16] == 16 and slots[17:] == [32, 33, 34]
    src, dst, refused = t.fork([-1, 0, -1], [0, 17, 0])     # shares page 0, a page of its own for one token
    assert (src, dst, refused) == ([-1, 1, -1], [-1, 3, -1], [0, 0, 0])
    assert t.refs[:5] == [2, 1, 1, 1, 0] and t.rows[1][:2] == [0, 3]
    t.trim([0, -1, 3])                                      # page 0 is still the fork's
    assert t.count == 5 and t.free[:5] == [7, 6, 5, 4, 1] and t.refs[0] == 1
    t.trim([0, 16, 0])
    assert t.free[:7] == [7, 6, 5, 4, 1, 2, 3] and t.count == 7
    t.extend([0, 0, 0, 100], 100)                           # more than the row holds
    assert t.seq == [0, 16, 0]


class _Pool(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("free_pages", ctypes.c_void_p),
                ("free_count", ctypes.c_void_p), ("page_refs", ctypes.c_void_p), ("page_tags", ctypes.c_void_p),
                ("scratch", ctypes.c_void_p)]


P = ctypes.c_void_p(0x10000)
GOOD = dict(num_pages=64, page_size=16, free_pages=P, free_count=P, page_refs=P, page_tags=P, scratch=P)


def _calls(pool, batch=2, maxp=4, tokens=2, missing=None):
    """The three calls' statuses; `missing`: the position of a device pointer that is NULL."""
    lib, pool = kvq.load(), ctypes.byref(pool) if pool is not None else None
    a = [P] * 8
    if missing is not None:
        a[missing] = None
    return [lib.kvq_extend_tables(pool, None, tokens, a[0], batch, a[1], maxp, a[2], None, a[3], None),
            lib.kvq_fork_tables(pool, a[4], a[5], a[0], batch, a[1], maxp, a[2], a[6], a[7], a[3], None),
            lib.kvq_trim_tables(pool, a[4], a[0], batch, a[1], maxp, None)]


def test_bad_pools_are_refused():
    assert _calls(None) == [1, 1, 1]
    for name in ("free_pages", "free_count", "page_refs", "scratch"):
        assert _calls(_Pool(**{**GOOD, name: None})) == [1, 1, 1], name
    assert _calls(_Pool(**{**GOOD, "num_pages": 0})) == [1, 1, 1]
    for ps in (0, 8, 24, 256):
        assert _calls(_Pool(**{**GOOD, "page_size": ps})) == [2, 2, 2]


def test_bad_arguments_are_refused():
    pool = _Pool(**GOOD)
    assert _calls(pool, batch=65536, tokens=65536) == [2, 2, 2]
    assert _calls(pool, batch=-1) == [1, 1, 1] and _calls(pool, maxp=0) == [1, 1, 1]
    assert _calls(pool, tokens=3)[0] == 1                   # no offsets, and not as many each
    assert _calls(pool, tokens=-2)[0] == 1
    assert _calls(pool, batch=0, tokens=1)[0] == 1
    assert _calls(pool, batch=0, tokens=0) == [0, 0, 0]     # nothing to do
    for i, want in {0: [1, 1, 1], 1: [1, 1, 1], 2: [1, 1], 3: [1, 1]}.items():
        assert _calls(pool, missing=i)[:len(want)] == want, i
    for i in (4, 5, 6, 7):
        assert _calls(pool, missing=i)[1] == 1, i
    assert _calls(_Pool(**{**GOOD, "page_tags": None}))[:2] == [1, 1]     # expected tags without live ones


def test_the_binding_checks_tensors():
    pool = kvq.PagePool.create(8, 16, device="cpu")
    i32 = dict(dtype=torch.int32)
    seq, bt = torch.zeros(2, **i32), torch.zeros((2, 4), **i32)
    flags = torch.zeros(2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="expected CUDA tensors"):
        kvq.kvq_extend_tables(pool, None, 2, seq, bt, bt, None, flags)
    with pytest.raises(ValueError, match="shape"):
        kvq.kvq_extend_tables(pool, None, 2, torch.zeros(3, **i32), bt, bt, None, flags)
    with pytest.raises(TypeError, match="slot_mapping"):
        kvq.kvq_extend_tables(pool, None, 2, seq, bt, bt, torch.zeros(2, **i32), flags)
    with pytest.raises(TypeError, match="parents"):
        kvq.kvq_fork_tables(pool, None, seq, seq, bt, bt, seq, seq, flags)
    with pytest.raises(ValueError, match="contiguous"):
        kvq.kvq_trim_tables(pool, torch.zeros((2, 2), **i32)[:, 0], seq, bt)
    with pytest.raises(AttributeError):
        kvq.kvq_trim_tables(object(), seq, seq, bt)
    pool.scratch = torch.zeros(3, **i32)
    with pytest.raises(ValueError, match="scratch"):
        kvq.kvq_trim_tables(pool, seq, seq, bt)
