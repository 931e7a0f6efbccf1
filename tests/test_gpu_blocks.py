"""GPU parity of the block-scaled append (codes and exponents bit for bit) and
of the page copy, and a decode run that uses them together: prompts appended,
requests forked by copying their last page, windowed tag check, append and
attention step by step."""
import numpy as np
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
import view_ref as R
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128


def t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def bf(x):
    return t(x.view(np.int16)).view(torch.bfloat16)


def _caches(rng, N, hkv, ps):
    k, v = (rng.integers(0, 256, (N, hkv, ps, D)).astype(np.uint8) for _ in range(2))
    ke, ve = (rng.integers(-12, -4, (N, hkv, ps // 16)).astype(np.int8) for _ in range(2))
    far = rng.random(ke.shape) < 0.2
    ke[far] = rng.integers(-128, 128, far.sum())
    return k, v, ke, ve


def _append(desc, k_new, v_new, offsets, bt, lens, abort, k, v, ke, ve):
    """The GPU's caches after the call, and view_ref's (numpy)."""
    dev = [t(x) for x in (k, v, ke, ve)]
    kvq.kvq_append_blocks(desc, bf(k_new), bf(v_new), None if offsets is None else t(offsets), t(bt), t(lens),
                          None if abort is None else t(abort), *dev)
    torch.cuda.synchronize()
    ref = [x.copy() for x in (k, v, ke, ve)]
    if offsets is None:
        offsets = np.arange(len(lens) + 1) * (k_new.shape[0] // len(lens))
    R.append_blocks(*ref, k_new, v_new, offsets, bt, lens, abort)
    for name, a, b in zip(("k", "v", "k_exp", "v_exp"), dev, ref):
        got = a.cpu().numpy()
        if got.dtype == np.uint8:                           # a NaN stays NaN, of either sign
            got, b = (np.where(x == 0xFF, 0x7F, x) for x in (got, b))
        if not np.array_equal(got, b):
            at = tuple(np.argwhere(got != b)[0])
            raise AssertionError(f"{name}: {(got != b).sum()} differ, first at {at}: {got[at]} for {b[at]}")
    return ref


def _values(rng, shape, kind):
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-8, 9, shape[:2] + (1,)))
    if kind == "ties":                                      # halves of e4m3 steps, both sides of a border
        x = np.ldexp(rng.integers(0, 64, shape).astype(np.float64) + 0.5, rng.integers(-6, 6, shape))
        x *= rng.choice([-1, 1], shape)
    bits = W.f32_to_bf16_bits(x.astype(np.float32))
    if kind == "special":
        some = rng.random(shape) < 0.01
        bits[some] = rng.choice([0x7F80, 0xFF80, 0x7FC0, 0xFFFF, 0, 0x8000, 1, 0x7F7F, 0xFF7F, 0x0080], some.sum())
        bits[rng.random(shape[:2]) < 0.1] = 0               # whole rows of zeros
        bits[rng.random(shape[:2]) < 0.1] = 0x0003          # of the smallest subnormals
    return bits


@pytest.mark.parametrize("kind", ["normal", "ties", "special"])
@pytest.mark.parametrize("hkv,ps", [(1, 16), (8, 32), (3, 64), (5, 128)])
def test_append_ragged(hkv, ps, kind):
    rng = np.random.default_rng([hkv, ps, len(kind)])
    counts = np.array([1, 0, 2, 16, 15, 17, 33, 100, 1, 48, 5, 1, 31, 18], np.int32)
    starts = np.array([0, 5, 15, 0, 1, 16, 31, 7, 31, 16, 300, 129, 17, 14], np.int32)
    lens = counts + starts
    B = len(lens)
    maxp = -(-int(lens.max()) // ps) + 1
    N = B * maxp + 2
    bt = rng.permutation(N)[:B * maxp].reshape(B, maxp).astype(np.int32)
    bt[7, 1 if ps < 128 else 0] = -1                        # a bad page among good ones
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    T = int(offsets[-1])
    new = [_values(rng, (T, hkv, D), kind) for _ in range(2)]
    _append(kvq.CacheDesc(N, ps, hkv), *new, offsets, bt, lens, None, *_caches(rng, N, hkv, ps))
    abort = (np.arange(B) % 3 == 1).astype(np.uint8)
    _append(kvq.CacheDesc(N, ps, hkv), *new, offsets, bt, lens, abort, *_caches(rng, N, hkv, ps))


@pytest.mark.parametrize("n", [1, 2, 16, 17, 40])
def test_append_equal_counts(n):
    rng = np.random.default_rng(n)
    lens = np.array([n, n + 1, n + 15, n + 16, n + 37, n - 1, 0, 64 + n, 640], np.int32)   # two have too few positions
    B, ps, hkv = len(lens), 32, 2
    maxp = 20
    N = B * maxp
    bt = rng.permutation(N).reshape(B, maxp).astype(np.int32)
    new = [_values(rng, (B * n, hkv, D), "normal") for _ in range(2)]
    _append(kvq.CacheDesc(N, ps, hkv), *new, None, bt, lens, None, *_caches(rng, N, hkv, ps))


def test_append_many_requests_and_bad_offsets():
    """More requests than one round of the search tests; then offsets that
    descend, start below 0 or end past the tokens: those requests are skipped
    (and whatever work items the bad numbering loses write nothing)."""
    rng = np.random.default_rng(4)
    B, ps, hkv = 1500, 16, 1
    counts = rng.integers(0, 5, B).astype(np.int32)
    lens = (counts + rng.integers(0, 40, B)).astype(np.int32)
    N = B * 3
    bt = rng.permutation(N).reshape(B, 3).astype(np.int32)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    new = [_values(rng, (int(offsets[-1]), hkv, D), "normal") for _ in range(2)]
    caches = _caches(rng, N, hkv, ps)
    _append(kvq.CacheDesc(N, ps, hkv), *new, offsets, bt, lens, None, *caches)
    too_long = lens.copy()
    too_long[::7] = 49 + counts[::7]
    _append(kvq.CacheDesc(N, ps, hkv), *new, offsets, bt, too_long, None, *caches)
    # a prefix that does not start at 0: the rows before it belong to no request
    shifted = [np.concatenate([x[:5], x]) for x in new]
    _append(kvq.CacheDesc(N, ps, hkv), *shifted, offsets + 5, bt, lens, None, *caches)
    dev = [t(x) for x in caches]
    for bad in (offsets - 3, offsets[::-1].copy(), offsets * 1000, np.full(B + 1, -2**31, np.int32),
                np.full(B + 1, 2**31 - 1, np.int32)):
        k2 = [x.clone() for x in dev]
        kvq.kvq_append_blocks(kvq.CacheDesc(N, ps, hkv), bf(new[0]), bf(new[1]), t(bad.astype(np.int32)), t(bt),
                              t(lens), None, *k2)
        torch.cuda.synchronize()
        if bad is not offsets and bad[0] >= 0 and np.all(np.diff(bad) <= 0):
            assert all(torch.equal(a, b) for a, b in zip(dev, k2))


def test_append_without_tokens_or_requests():
    d = kvq.CacheDesc(4, 16, 1)
    k = torch.zeros((4, 1, 16, D), dtype=torch.uint8, device=DEV)
    e = torch.zeros((4, 1, 1), dtype=torch.int8, device=DEV)
    none = torch.zeros((0, 1, D), dtype=torch.bfloat16, device=DEV)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)  # noqa: E731
    kvq.kvq_append_blocks(d, none, none, i32(4), i32(3, 1), i32(3), None, k, k.clone(), e, e.clone())
    kvq.kvq_append_blocks(d, none, none, None, i32(0, 1), i32(0), None, k, k.clone(), e, e.clone())
    torch.cuda.synchronize()
    assert not k.any() and not e.any()


# ------------------------------------------------------------- page copy

@pytest.mark.parametrize("ps,hkv,bf16,layers,n", [(16, 1, False, 1, 1), (16, 8, False, 3, 40), (128, 8, False, 1, 7),
                                                  (64, 5, True, 2, 33), (32, 3, False, 100, 9), (16, 3, True, 1, 0)])
def test_copy_pages(ps, hkv, bf16, layers, n):
    """100 layers make more arrays than one launch takes; exponent arrays of
    odd page sizes lie at odd addresses."""
    rng = np.random.default_rng([ps, hkv, n])
    N = 2 * n + 5
    desc = kvq.CacheDesc(N, ps, hkv, D, kvq.KVQ_CACHE_BF16 if bf16 else kvq.KVQ_CACHE_FP8_E4M3)
    caches = torch.randint(0, 256, (2 * layers, N, hkv, ps, D * (2 if bf16 else 1)), dtype=torch.uint8, device=DEV)
    exps = torch.randint(-128, 128, (2 * layers, N, hkv, ps // 16), dtype=torch.int8, device=DEV)
    perm = rng.permutation(N).astype(np.int32)
    src, dst = perm[:n].copy(), perm[n:2 * n].copy()
    if n > 6:
        src[1] = src[0]                                     # one source, two destinations
        src[2], dst[3], src[4] = -1, N, 2**31 - 1           # skipped
        dst[5] = src[5]                                     # onto itself
    want_c, want_e = caches.clone(), exps.clone()
    for a, b in zip(src, dst):
        if 0 <= a < N and 0 <= b < N:
            want_c[:, b] = want_c[:, a]
            want_e[:, b] = want_e[:, a]
    view = caches.view(torch.bfloat16) if bf16 else caches
    kvq.kvq_copy_pages(desc, list(view), [] if bf16 else list(exps), t(src), t(dst))
    torch.cuda.synchronize()
    assert torch.equal(caches, want_c)
    assert torch.equal(exps, exps if bf16 else want_e)


# ---------------------------------------------------- the set as it is used

@pytest.mark.parametrize("window,sinks", [(0, 0), (48, 5)])
def test_a_decode_run(window, sinks):
    """Four prompts appended; two requests forked from the first (full pages
    shared, the last page copied); then steps of tag check, append and
    attention with growing values, so that blocks change their exponents while
    forks share their parent's pages.  Pages that leave the window are given
    back (-1, their tags changed).  Caches and outputs against view_ref."""
    rng = np.random.default_rng(window)
    ps, hkv, g, N, maxp = 16, 2, 4, 64, 12
    desc = kvq.CacheDesc(N, ps, hkv)
    scale = float(np.float32(1 / np.sqrt(D)))
    ref = list(_caches(rng, N, hkv, ps))
    dev = [t(x) for x in ref]
    free = list(rng.permutation(N))
    bt = np.full((6, maxp), -1, np.int32)
    lens = np.array([70, 16, 33, 1, 0, 0], np.int32)
    tags = rng.integers(0, 2**31, N).astype(np.int32)
    expected = np.zeros((6, maxp), np.int32)

    def give(r, i):
        page = int(free.pop())
        bt[r, i], expected[r, i] = page, tags[page]

    for r in range(4):
        for i in range(-(-int(lens[r]) // ps)):
            give(r, i)
    counts = lens.copy()
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    new = [W.normal_bf16(rng, (int(offsets[-1]), hkv, D)) for _ in range(2)]
    kvq.kvq_append_blocks(desc, bf(new[0]), bf(new[1]), t(offsets), t(bt), t(lens), None, *dev)
    R.append_blocks(*ref, *new, offsets, bt, lens)
    # fork request 0 twice
    last = (int(lens[0]) - 1) // ps
    for child in (4, 5):
        lens[child] = lens[0]
        bt[child, :last], expected[child, :last] = bt[0, :last], expected[0, :last]
        give(child, last)
    src, dst = np.full(2, bt[0, last], np.int32), bt[4:6, last].copy()
    kvq.kvq_copy_pages(desc, dev[:2], dev[2:], t(src), t(dst))
    for x in ref:
        x[dst] = x[src]
    ws = kvq.workspace_for_blocks(desc, 6, 1, hkv * g, maxp, window, sinks)
    for step in range(40):
        lens += 1
        for r in range(6):
            if (lens[r] - 1) % ps == 0:
                give(r, (int(lens[r]) - 1) // ps)
        if window:
            for r in range(4):                              # forks' parents keep shared pages alive
                gone = (int(lens[r]) - window) // ps
                for i in range(-(-sinks // ps), max(gone, 0)):
                    page = bt[r, i]
                    if page >= 0 and r:
                        tags[page] += 1
                        free.append(page)
                    bt[r, i] = -1
        new = [W.f32_to_bf16_bits((rng.standard_normal((6, hkv, D)) * 2.0 ** (step % 12 - 4)).astype(np.float32))
               for _ in range(2)]
        q = W.normal_bf16(rng, (6, 1, hkv * g, D))
        abort = torch.empty(6, dtype=torch.uint8, device=DEV)
        out = torch.empty((6, 1, hkv * g, D), dtype=torch.float32, device=DEV)
        kvq.kvq_tag_check_window(t(bt), t(expected), t(lens), ps, t(tags), window, sinks, 1, abort)
        kvq.kvq_append_blocks(desc, bf(new[0]), bf(new[1]), None, t(bt), t(lens), abort, *dev)
        kvq.kvq_decode_attn_blocks(desc, bf(q), *dev, t(bt), t(lens), scale, window, sinks, abort, out, ws)
        R.append_blocks(*ref, *new, np.arange(7), bt, lens)
        assert not abort.any()
        for a, b in zip(dev, ref):
            assert np.array_equal(a.cpu().numpy(), b), step
        want, bound = R.attention(q, ref[0], ref[1], bt, lens, scale, window, sinks, ke=ref[2], ve=ref[3],
                                  fp32=True)
        R.assert_within(out.cpu().numpy().astype(np.float64), want, bound, f"step {step}")
    assert kvq.kvq_device_error() == 0
