"""Where the arrival counters of the windowed and block-scaled calls end, on the
host: calls of one batch, head count and n share a workspace whatever their
windows, sinks and table widths are, so no plan may put anything else where
another of them keeps a counter."""
import pytest

import fp8_quantised_paged_kv_gb300 as kvq

PLANS = (kvq.kvq_decode_plan_window, kvq.kvq_decode_plan_blocks)


def _up256(x):
    return -(-x // 256) * 256


def kind_of(plan, desc, batch, n, hq, maxp, window, splits, counters):
    """Which form of launch asks for as many bytes as the plan says, with that
    many of counters in front: equal splits (their partials by rows), a launch
    shared on the device (a slot of 8 or 16 rows per (CTA, pair), and a record
    per pair where there are few pairs), or one split, or on a host with a GPU
    a cluster of splits (nothing else)."""
    split_tokens, most, total = plan(desc, batch, n, hq, maxp, window, 4 if window else 0, splits)
    if total == counters:
        return "one"
    rows = batch * n * hq * most
    if total == counters + _up256(rows * 4) + rows * 512:
        return "grid"
    # 152 SMs of three CTAs, which a host without a GPU plans for too
    pairs = batch * desc.num_kv_heads * (1 if n == 1 else -(-n * (hq // desc.num_kv_heads) // 16))
    for waves in range(1, 100):
        rows = (456 * waves + pairs) * (8 if n == 1 else 16)
        if total == counters + _up256(rows * 4) + rows * 512 + (8 * pairs if 456 >= 8 * pairs else 0):
            return "shared"
    return None


@pytest.mark.parametrize("plan", PLANS)
@pytest.mark.parametrize("batch,hkv,g", [(8, 8, 8), (40, 4, 4), (3, 8, 6)])
@pytest.mark.parametrize("n", [1, 3, 5, 8, 16])
def test_counters_go_by_batch_heads_and_query_tokens(plan, batch, hkv, g, n):
    """Tables from 64 tokens to 128 K, no window and windows on both sides of
    every border of the planner's."""
    counters = _up256(batch * hkv * (1 if n == 1 else -(-n * g // 16)) * 4)
    desc = kvq.CacheDesc(1 << 16, 64, hkv)
    seen = set()
    for maxp in (1, 16, 100, 128, 256, 512, 2048):
        for window in (0, 1, 500, 2000, 4000, 8000, 8192, 16000, 2**31 - 1):
            for splits in (0, 3):
                kind = kind_of(plan, desc, batch, n, hkv * g, maxp, window, splits, counters)
                assert kind is not None, (maxp, window, splits)
                seen.add(kind)
    assert "grid" in seen and ("shared" in seen) == (n == 1 or n * g <= 32)


@pytest.mark.parametrize("plan", PLANS)
def test_window_and_full_layers_in_turn(plan):
    """8 requests, 8 KV heads, 24 query rows each, tables of 16,384 tokens: a
    window of 8,000 plans equal splits, no window a launch that shares its work
    out and joins the splits by the counters."""
    desc = kvq.CacheDesc(4096, 64, 8)
    assert kind_of(plan, desc, 8, 3, 64, 256, 8000, 0, 512) == "grid"
    assert kind_of(plan, desc, 8, 3, 64, 256, 0, 0, 512) == "shared"
