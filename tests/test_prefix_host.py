"""Plans and refusals of the attention over shared prefixes, on the host: no GPU is needed."""
import ctypes

import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq

P = ctypes.c_void_p(0x10000)
F = ctypes.c_float(0.1)
BIG = 1 << 34


def desc(ps=64, hkv=8, dtype=0, pages=4104, head_dim=128):
    return kvq.CacheDesc(pages, ps, hkv, head_dim, dtype)


def test_plans():
    plan = kvq.kvq_decode_plan_prefix
    # below 512 MB of cache that the tables allow: the unshared call's own size
    small = plan(desc(), 4, 1, 32, 16)
    assert small == kvq.kvq_decode_plan_window(desc(), 4, 1, 32, 16, 0, 0)[2]
    assert plan(desc(), 64, 1, 32, 63) < 152 * 256 * 512 <= plan(desc(), 64, 1, 32, 64)      # 64 x 8 x 4,096 x 256 B
    assert plan(desc(dtype=1), 64, 1, 32, 31) < 152 * 256 * 512 <= plan(desc(dtype=1), 64, 1, 32, 32)
    # each 16 query rows read the pages again
    assert plan(desc(), 64, 5, 32, 31) < 152 * 256 * 512 <= plan(desc(), 64, 5, 32, 32)       # 20 rows
    # the unshared call's, places for 256 rows of each of 152 SMs and twice the rows (a log-sum-exp
    # and 128 values each), a record of 16 bytes per row, the rest small
    n = kvq.kvq_decode_plan_window(desc(), 64, 1, 32, 4096, 0, 0)[2] + (152 * 256 + 2 * 64 * 32) * 516 + 64 * 32 * 16
    assert abs(plan(desc(), 64, 1, 32, 4096) - n) <= 8192
    assert plan(desc(), 0, 1, 32, 16) > 0


@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("batch,n,hq,maxp", [(1, 1, 8, 1), (3, 2, 32, 16), (64, 1, 64, 30), (16, 16, 64, 64), (200, 1, 8, 9)])
def test_one_plan_serves_the_block_scaled_call_too(ps, batch, n, hq, maxp):
    assert (kvq.kvq_decode_plan_blocks(desc(ps), batch, n, hq, maxp, 0, 0)[2]
            <= kvq.kvq_decode_plan_prefix(desc(ps), batch, n, hq, maxp))


@pytest.mark.parametrize("status,change", [
    (2, dict(head_dim=64)), (2, dict(ps=8)), (1, dict(pages=0)), (1, dict(hkv=0)), (1, dict(dtype=7))])
def test_plans_refuse_caches(status, change):
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_decode_plan_prefix(desc(**change), 4, 1, 32, 16)
    assert e.value.status == status


@pytest.mark.parametrize("status,args", [
    (1, (-1, 1, 32, 16)), (1, (4, 0, 32, 16)), (2, (4, 17, 32, 16)), (1, (4, 1, 33, 16)), (2, (4, 1, 128, 16)),
    (1, (4, 1, 32, 0)), (2, (65536, 1, 32, 16)), (2, (60000, 16, 64, 4096))])
def test_plans_refuse_shapes(status, args):
    with pytest.raises(kvq.KvqError) as e:
        kvq.kvq_decode_plan_prefix(desc(), *args)
    assert e.value.status == status
    with pytest.raises(OverflowError):
        kvq.kvq_decode_plan_prefix(desc(), 4, 1, 32, 2**31)


def _call(blocks, d=None, batch=64, n=1, hq=32, maxp=64, ptrs=None, scale=0.1, out_dtype=0, ws=P, ws_bytes=BIG):
    lib = kvq.load()
    fn = lib.kvq_decode_attn_prefix_blocks if blocks else lib.kvq_decode_attn_prefix
    p = [P] * 10                                            # q, k, v, s0, s1, table, lens, prefix_of, prefix_lens, out
    for i, v in (ptrs or {}).items():
        p[i] = v
    d = d or desc()
    return fn(ctypes.byref(d.c()), p[0], batch, n, hq, p[1], p[2], p[3], p[4], p[5], maxp, p[6], p[7], p[8],
              ctypes.c_float(scale), None, p[9], out_dtype, ws, ws_bytes, None)


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("maxp", [4, 64])                   # apart, and shared
def test_calls_are_refused_before_they_reach_a_gpu(blocks, maxp):
    for i in range(10):
        assert _call(blocks, maxp=maxp, ptrs={i: None}) == 1, i
    for i in (0, 1, 2, 9):
        assert _call(blocks, maxp=maxp, ptrs={i: ctypes.c_void_p(0x10008)}) == 1, i
    assert _call(blocks, maxp=maxp, out_dtype=2) == 1
    for scale in (float("nan"), float("inf")):
        assert _call(blocks, maxp=maxp, scale=scale) == 1
    need = kvq.kvq_decode_plan_prefix(desc(), 64, 1, 32, maxp)
    assert _call(blocks, maxp=maxp, ws_bytes=need - 1) == 3 and _call(blocks, maxp=maxp, ws=None) == 3
    assert _call(blocks, maxp=maxp, ws=ctypes.c_void_p(0x10008)) == 1
    assert _call(blocks, maxp=maxp, n=17) == 2 and _call(blocks, maxp=maxp, batch=-1) == 1
    assert _call(blocks, maxp=maxp, batch=0, ptrs={i: None for i in range(10)}) == 0
    if blocks:
        assert _call(True, desc(dtype=1), maxp=maxp) == 1   # exponents with a bf16 cache


def test_the_binding_checks_tensors():
    d = desc(pages=8, hkv=2)
    q = torch.zeros((2, 1, 4, 128), dtype=torch.bfloat16)
    k = torch.zeros((8, 2, 64, 128), dtype=torch.uint8)
    s = torch.ones(2)
    i32 = torch.zeros(2, dtype=torch.int32)
    bt = torch.zeros((2, 4), dtype=torch.int32)
    ws = torch.empty(1 << 20, dtype=torch.uint8)
    call = lambda **x: kvq.kvq_decode_attn_prefix(**{**dict(  # noqa: E731
        desc=d, q=q, k_cache=k, v_cache=k, k_scale=s, v_scale=s, block_table=bt, seq_lens=i32, prefix_of=i32,
        prefix_lens=i32, softmax_scale=0.1, abort_flags=None, out=q, workspace=ws), **x})
    with pytest.raises(ValueError, match="expected CUDA tensors"):
        call()
    with pytest.raises(TypeError, match="prefix_of"):
        call(prefix_of=i32.long())
    with pytest.raises(ValueError, match="prefix_lens"):
        call(prefix_lens=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError, match="prefix_of"):
        call(prefix_of=None)
    with pytest.raises(ValueError, match="rows"):
        call(block_table=bt[:1])
    with pytest.raises(ValueError, match="contiguous"):
        call(seq_lens=torch.zeros((2, 2), dtype=torch.int32)[:, 0])
    e = torch.zeros((8, 2, 4), dtype=torch.int8)
    with pytest.raises(ValueError, match="k_exp"):
        kvq.kvq_decode_attn_prefix_blocks(d, q, k, k, e[:, :1].contiguous(), e, bt, i32, i32, i32, 0.1, None, q, ws)
