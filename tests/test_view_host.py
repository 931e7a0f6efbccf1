"""Refusals of the block-scaled, windowed and page-copy calls, on the host:
plans and argument checks that need no GPU."""
import ctypes

import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq

P = ctypes.c_void_p(0x10000)
F = ctypes.c_float(0.1)
BIG = 1 << 30


def desc(ps=16, hkv=8, dtype=0, pages=4104, head_dim=128):
    return kvq.CacheDesc(pages, ps, hkv, head_dim, dtype)


@pytest.mark.parametrize("plan", [kvq.kvq_decode_plan_window, kvq.kvq_decode_plan_blocks])
def test_plans_count_what_a_request_can_show(plan):
    # without a window: the whole context
    st, ms, ws = plan(desc(), 8, 1, 64, 513, 0, 0, 4)
    assert st * ms >= 513 * 16
    # window 100 from position p - 99, 3 sinks, 5 query tokens: 104 positions
    # on at most 103 // 16 + 2 = 8 pages, and one page of sinks
    st, ms, ws = plan(desc(), 8, 5, 64, 513, 100, 3, 64)
    assert st == 32 and ms == -(-9 * 16 // 32)
    # a window of one position: one page of it at most twice, no sinks
    assert plan(desc(), 1, 1, 8, 100000, 1, 0, 0)[:2] == (32, 1)
    # a window or sinks beyond the table's row: the row, whatever the sum is
    for w, s in ((2**31 - 1, 2**31 - 1), (1 << 20, 0), (5, 1 << 20)):
        assert plan(desc(), 8, 16, 64, 513, w, s, 12) == plan(desc(), 8, 16, 64, 513, 0, 0, 12)
    # one wave's planning goes by the shown tokens: no 8,192-token splits of a long row
    assert plan(desc(64), 4, 1, 16, 16384, 4096, 4)[0] < 8192


def test_plans_of_large_tables_share_on_the_device():
    """From 256 MB of cache that the tables allow: a workspace slot (8 query rows,
    16 with several query tokens) for every (CTA, pair) that can meet, the
    grid in whole waves of the resident CTAs (152 SMs x 3 on a host without a
    GPU), and no more splits of a pair than the combine takes."""
    below = kvq.kvq_decode_plan_blocks(desc(64), 16, 1, 32, 127)
    at = kvq.kvq_decode_plan_blocks(desc(64), 16, 1, 32, 128)
    assert below[0] < 8192 and at[0] == 8192
    pairs = 16 * 8
    slots = 152 * 3 + pairs
    counters = (pairs * 4 + 255) // 256 * 256
    assert at[2] == counters + (slots * 8 * 4 + 255) // 256 * 256 + slots * 8 * 512
    mt = kvq.kvq_decode_plan_window(desc(64), 16, 5, 32, 128, 0, 0)          # 20 rows: two row blocks
    slots = 152 * 3 + 2 * pairs
    assert mt[2] == (2 * pairs * 4 + 255) // 256 * 256 + (slots * 16 * 4 + 255) // 256 * 256 + slots * 16 * 512
    # a window that shows little of a large table
    assert kvq.kvq_decode_plan_window(desc(64), 16, 1, 32, 4096, 500, 4)[0] < 8192
    # 64 x 8 pairs of 1M tokens: several waves, at most 1,024 splits a pair
    st, ms, _ = kvq.kvq_decode_plan_blocks(desc(64), 64, 1, 32, 16384)
    assert st == 8192 and 900 < ms <= 1024
    # an explicit split count keeps the grid
    assert kvq.kvq_decode_plan_blocks(desc(64), 16, 1, 32, 128, 0, 0, 4)[:2] == (2048, 4)


@pytest.mark.parametrize("plan", [kvq.kvq_decode_plan_window, kvq.kvq_decode_plan_blocks])
def test_plans_refuse(plan):
    for args, status in [((desc(), 8, 0, 64, 513, 0, 0), 1), ((desc(), 8, 17, 64, 513, 0, 0), 2),
                         ((desc(), 8, 1, 64, 513, -1, 0), 1), ((desc(), 8, 1, 64, 513, 1, -1), 1),
                         ((desc(), 8, 1, 63, 513, 1, 0), 1), ((desc(), 8, 1, 128, 513, 1, 0), 2),
                         ((desc(ps=8), 8, 1, 64, 513, 1, 0), 2), ((desc(head_dim=64), 8, 1, 64, 513, 1, 0), 2),
                         ((desc(), 65536, 1, 64, 513, 1, 0), 2), ((desc(), 8, 1, 64, 0, 1, 0), 1)]:
        with pytest.raises(kvq.KvqError) as e:
            plan(*args)
        assert e.value.status == status, args


def test_numbers_past_32_bits_are_refused():
    for plan in (kvq.kvq_decode_plan_window, kvq.kvq_decode_plan_blocks):
        with pytest.raises(OverflowError):
            plan(desc(), 8, 1, 64, 513, 2**32 + 5, 0)
        with pytest.raises(OverflowError):
            plan(desc(), 8, 1, 64, 513, 5, 2**31)


def test_the_block_scaled_cache_is_an_fp8_cache():
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_decode_plan_blocks(desc(dtype=1), 8, 1, 64, 513)
    assert e.value.status == 1
    assert kvq.kvq_decode_plan_window(desc(dtype=1), 8, 1, 64, 513, 100)[1] >= 1


def _attn(fn, d, q=P, B=2, n=1, Hq=8, k=P, v=P, s0=P, s1=P, bt=P, maxp=8, seq=P, scale=F, window=16, sinks=1,
          out=P, dtype=0, ws=P, ws_bytes=BIG):
    return getattr(kvq.load(), fn)(ctypes.byref(d.c()), q, B, n, Hq, k, v, s0, s1, bt, maxp, seq, scale, window,
                                   sinks, None, out, dtype, ws, ws_bytes, 0, None)


@pytest.mark.parametrize("fn", ["kvq_decode_attn_window", "kvq_decode_attn_blocks"])
def test_attention_refuses(fn):
    d = desc()
    odd = ctypes.c_void_p(0x10008)
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(s0=None), dict(s1=None), dict(bt=None),
                dict(seq=None), dict(out=None), dict(q=odd), dict(k=odd), dict(v=odd), dict(out=odd), dict(ws=odd),
                dict(window=-1), dict(sinks=-1), dict(dtype=2), dict(n=0), dict(B=-1),
                dict(scale=ctypes.c_float(float("nan")))):
        assert _attn(fn, d, **bad) == 1, bad
    assert _attn(fn, d, n=17) == 2
    assert _attn(fn, d, ws_bytes=16) == 3 and _attn(fn, d, ws=None) == 3
    assert _attn(fn, d, B=0) == 0                          # nothing to do


def _append(d, k=P, v=P, T=4, off=P, bt=P, maxp=8, seq=P, B=2, kc=P, vc=P, ke=P, ve=P):
    return kvq.load().kvq_append_blocks(ctypes.byref(d.c()), k, v, T, off, bt, maxp, seq, B, None, kc, vc, ke, ve,
                                        None)


def test_append_refuses():
    odd = ctypes.c_void_p(0x10008)
    for bad in (dict(k=None), dict(v=None), dict(bt=None), dict(seq=None), dict(kc=None), dict(vc=None),
                dict(ke=None), dict(ve=None), dict(k=odd), dict(v=odd), dict(kc=odd), dict(vc=odd), dict(T=-1),
                dict(B=-1), dict(B=0), dict(maxp=0), dict(T=5, off=None)):
        assert _append(desc(), **bad) == 1, bad
    assert _append(desc(dtype=1)) == 1
    assert _append(desc(), B=65536) == 2 and _append(desc(ps=48)) == 2
    assert _append(desc(), T=0) == 0 and _append(desc(), T=0, B=0) == 0


def test_tag_check_refuses():
    def call(B=2, maxp=8, ps=16, pages=64, window=4, sinks=0, n=1, flags=P, bt=P):
        return kvq.load().kvq_tag_check_window(bt, P, P, B, maxp, ps, P, pages, window, sinks, n, flags, None)
    for bad in (dict(window=-1), dict(sinks=-1), dict(n=0), dict(ps=0), dict(pages=0), dict(maxp=0), dict(B=-1),
                dict(flags=None), dict(bt=None)):
        assert call(**bad) == 1, bad
    assert call(n=17) == 2
    assert call(B=0) == 0


def test_copy_refuses():
    arr = lambda *p: (ctypes.c_void_p * len(p))(*p)  # noqa: E731

    def call(d=desc(), caches=arr(0x10000, 0x20000), nc=2, exps=arr(0x30001), ne=1, src=P, dst=P, n=3):
        return kvq.load().kvq_copy_pages(ctypes.byref(d.c()), caches, nc, exps, ne, src, dst, n, None)
    for bad in (dict(nc=-1), dict(ne=-1), dict(n=-1), dict(caches=None), dict(exps=None), dict(src=None),
                dict(dst=None), dict(caches=arr(0x10000, None)), dict(caches=arr(0x10000, 0x20008)),
                dict(exps=arr(None)), dict(d=desc(dtype=1))):
        assert call(**bad) == 1, bad
    assert call(d=desc(ps=8)) == 2
    assert call(n=0) == 0 and call(nc=0, ne=0, caches=None, exps=None) == 0


def test_binding_refuses_host_tensors_and_shapes():
    d = desc(pages=4, hkv=1)
    cache = torch.zeros((4, 1, 16, 128), dtype=torch.uint8)
    exps = torch.zeros((4, 1, 1), dtype=torch.int8)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    new = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    q = torch.zeros((2, 1, 1, 128), dtype=torch.bfloat16)
    ok = [d, new, new, None, i32(2, 2), i32(2), None, cache, cache, exps, exps]
    with pytest.raises(ValueError):                        # tensors not on a GPU
        kvq.kvq_append_blocks(*ok)
    for at, wrong, err in [(1, new.float(), TypeError), (2, new[:1], ValueError), (3, i32(2), ValueError),
                           (5, i32(3), ValueError), (7, cache[:3], ValueError), (9, exps.int(), TypeError),
                           (10, exps[:, :, :0], ValueError)]:
        args = list(ok)
        args[at] = wrong
        with pytest.raises(err):
            kvq.kvq_append_blocks(*args)
    out = torch.zeros_like(q)
    for fn, s in ((kvq.kvq_decode_attn_window, torch.ones(1)), (kvq.kvq_decode_attn_blocks, exps)):
        args = [d, q, cache, cache, s, s, i32(2, 2), i32(2), 0.1, 4, 1, None, out, cache]
        with pytest.raises(ValueError):
            fn(*args)
        for at, wrong, err in [(1, q.half(), TypeError), (2, cache[:3], ValueError), (4, s[:0], ValueError),
                               (6, i32(3, 2), ValueError), (12, out.half(), ValueError)]:
            bad = list(args)
            bad[at] = wrong
            with pytest.raises(err):
                fn(*bad)
    with pytest.raises(ValueError):
        kvq.kvq_copy_pages(d, [cache], [exps], i32(2), i32(2))
    with pytest.raises(ValueError):
        kvq.kvq_copy_pages(d, [cache], [], i32(2), i32(3))
    with pytest.raises(TypeError):
        kvq.kvq_copy_pages(d, [cache.char()], [], i32(2), i32(2))
    with pytest.raises(ValueError):
        kvq.kvq_tag_check_window(i32(2, 2), i32(2, 2), i32(2), 16, i32(4), 4, 0, 1,
                                 torch.zeros(2, dtype=torch.uint8))
