"""GPU parity of the windowed and the block-scaled decode attention and of the
windowed tag check against plain fp64 implementations, with bounds derived
from the kernels' roundings (view_ref).  Whatever a query does not see --
table entries, tags, K, V and exponents outside the window -- is poisoned."""
import numpy as np
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
import view_ref as R
import workloads as W

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 128
SCALE = float(np.float32(1 / np.sqrt(D)))
LENS = (1, 0, 2, 15, 16, 17, 31, 33, 64, 100, 129, 257, 1000, 2049)
KINDS = ("fp8", "bf16", "blocks")


@pytest.fixture(autouse=True)
def _no_device_errors():
    kvq.kvq_device_error(clear=True)
    yield
    torch.cuda.synchronize()
    assert kvq.kvq_device_error() == 0


class Case:
    """Caches of random values, shuffled pages, everything unseen poisoned."""

    def __init__(self, kind, lens, g, ps, n, window, sinks, hkv=2, seed=0, ev=(-10, 3), padded=False):
        rng = np.random.default_rng([seed, n, g, ps, window, sinks])
        self.kind, self.n, self.window, self.sinks, self.ps = kind, n, window, sinks, ps
        self.lens = np.asarray(lens, np.int32)
        B = len(lens)
        counts = [max(1, -(-int(x) // ps)) for x in lens]
        maxp = max(counts)
        if padded:                                          # a table padded until the work is shared on the device
            maxp += -(-(256 << 20) // (256 * B * hkv * ps))
        N = sum(counts) + 3
        perm = rng.permutation(N).astype(np.int32)
        self.bt = np.full((B, maxp), -1, np.int32)
        at = 0
        for r, c in enumerate(counts):
            self.bt[r, :c] = perm[at:at + c]
            at += c
        shape = (N, hkv, ps, D)
        nan = 0x7FC0 if kind == "bf16" else R.NAN_CODE
        values = [rng.standard_normal(shape) for _ in range(2)]
        if kind == "bf16":
            full = [W.f32_to_bf16_bits(x.astype(np.float32)) for x in values]
        else:
            full = [R.encode(x * 90) for x in values]
        self.k, self.v = (np.full(shape, nan, x.dtype) for x in full)
        self.ks, self.vs = (rng.uniform(0.006, 0.02, hkv).astype(np.float32) for _ in range(2))
        self.ke = self.ve = None
        if kind == "blocks":
            e = [rng.integers(-11, -5, (N, hkv, ps // 16)), rng.integers(ev[0], ev[1] + 1, (N, hkv, ps // 16))]
            self.ke, self.ve = (np.where(rng.random(x.shape) < .5, 127, -128).astype(np.int8) for x in e)
        for r in range(B):                                  # only what some query sees is real
            L = int(self.lens[r])
            pos = np.flatnonzero(R.view_mask(L, n, window, sinks).any(axis=0)) if L > 0 else np.zeros(0, int)
            pages = self.bt[r][pos // ps]
            for dst, src in ((self.k, full[0]), (self.v, full[1])):
                dst[pages, :, pos % ps] = src[pages, :, pos % ps]
            if kind == "blocks":
                for dst, src in ((self.ke, e[0]), (self.ve, e[1])):
                    dst[pages, :, pos % ps // 16] = src[pages, :, pos % ps // 16]
            held = np.zeros(maxp, bool)
            held[pos // ps] = True
            self.bt[r, ~held] = rng.choice([-1, N, 2**31 - 1, -2**31])
        self.q_bits = W.normal_bf16(rng, (B, n, hkv * g, D))
        self.desc = kvq.CacheDesc(N, ps, hkv, D, kvq.KVQ_CACHE_BF16 if kind == "bf16" else kvq.KVQ_CACHE_FP8_E4M3)
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        bf = lambda x: t(x.view(np.int16)).view(torch.bfloat16)  # noqa: E731
        self.d = dict(k=bf(self.k) if kind == "bf16" else t(self.k), v=bf(self.v) if kind == "bf16" else t(self.v),
                      bt=t(self.bt), seq=t(self.lens), q=bf(self.q_bits))
        if kind == "blocks":
            self.d.update(s0=t(self.ke), s1=t(self.ve))
        else:
            self.d.update(s0=t(self.ks), s1=t(self.vs))

    def workspace(self, splits):
        make = kvq.workspace_for_blocks if self.kind == "blocks" else kvq.workspace_for_window
        return make(self.desc, len(self.lens), self.n, self.q_bits.shape[2], self.bt.shape[1], self.window,
                    self.sinks, splits)

    def call(self, out, ws, splits=0, abort=None, stream=None, **other):
        d = {**self.d, **other}
        fn = kvq.kvq_decode_attn_blocks if self.kind == "blocks" else kvq.kvq_decode_attn_window
        return fn(self.desc, d["q"], d["k"], d["v"], d["s0"], d["s1"], d["bt"], d["seq"], SCALE, self.window,
                  self.sinks, abort, out, ws, splits, stream)

    def out(self, fp32):
        return torch.full(self.q_bits.shape, 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV)

    def run(self, fp32, splits=0, abort=None):
        out = self.call(self.out(fp32), self.workspace(splits), splits, abort)
        torch.cuda.synchronize()
        return out.float().cpu().numpy().astype(np.float64)

    def ref(self, fp32, abort=None):
        # 33 and more query rows per KV head of an FP8 cache can take the tensor-memory kernel
        rows = self.n * self.q_bits.shape[2] // self.k.shape[1]
        cut = 2.0 ** -32 if self.kind != "bf16" and self.n > 1 and rows >= 33 else 2.0 ** -40
        return R.attention(self.q_bits, self.k, self.v, self.bt, self.lens, SCALE, self.window, self.sinks,
                           ks=self.ks, vs=self.vs, ke=self.ke, ve=self.ve, abort=abort, fp32=fp32, cut=cut)

    def check(self, splits=(0, 1, 5, 12), kinds=(False, True), abort=None, what=""):
        t = None if abort is None else torch.from_numpy(abort).to(DEV)
        for fp32 in kinds:
            ref, bound = self.ref(fp32, abort)
            for s in splits:
                R.assert_within(self.run(fp32, s, t), ref, bound, f"{what} fp32={fp32} splits={s}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (2, 1), (16, 4), (33, 17), (100, 200), (1000, 3),
                                          (5000, 4), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("ps,g", [(16, 8), (64, 3)])
def test_one_query_token(kind, window, sinks, ps, g):
    Case(kind, LENS, g, ps, 1, window, sinks).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,g,ps", [(2, 1, 32), (4, 4, 16), (5, 8, 128), (16, 8, 16), (11, 7, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (7, 3), (40, 20), (1000, 65)])
def test_several_query_tokens(kind, n, g, ps, window, sinks):
    Case(kind, LENS, g, ps, n, window, sinks).check()


@pytest.mark.parametrize("kind", KINDS)
def test_long_contexts_and_many_splits(kind):
    Case(kind, [70001, 9000, 33], 4, 64, 1, 20000, 70, hkv=1).check(splits=(0, 3, 40))
    Case(kind, [70001, 9000, 33], 4, 16, 3, 0, 0, hkv=1).check(splits=(0, 100), kinds=(True,))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ps,g,n", [(16, 8, 1), (128, 3, 1), (32, 5, 3), (64, 8, 16), (16, 7, 7)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 20), (1000, 65), (2**30, 0)])
def test_work_shared_on_the_device(kind, ps, g, n, window, sinks):
    """Tables padded to 256 MB of cache and more: requests of every length in one
    call, empty ones between (a window far larger than any context does not
    shorten the tables' reach, one of 1,000 does, and such a call runs a grid)."""
    c = Case(kind, LENS + (0, 0, 513, 0), g, ps, n, window, sinks, padded=True)
    shared = window == 0 or window == 2**30
    make = kvq.kvq_decode_plan_blocks if kind == "blocks" else kvq.kvq_decode_plan_window
    plan = make(c.desc, len(c.lens), n, 2 * g, c.bt.shape[1], window, sinks)
    tensor_memory = kind != "bf16" and n > 1 and n * g >= 33   # grids of its own
    assert (plan[0] == 8192) == (shared and not tensor_memory)
    abort = (np.arange(len(c.lens)) % 5 == 3).astype(np.uint8)
    c.check(splits=(0,), abort=abort)


# Few requests of many heads: enough work for the tensor-memory kernel (cache
# bytes x query rows of 2e9 and more, 33 rows and more per KV head)
TM_LENS = (5000, 0, 40, 4097, 1, 130, 2500, 9000)


@pytest.mark.parametrize("kind", ["fp8", "blocks"])
@pytest.mark.parametrize("n,g,ps", [(5, 8, 16), (8, 8, 64), (11, 6, 32), (16, 8, 128), (16, 3, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (4000, 70), (2**31 - 1, 3)])
def test_tensor_memory_kernel(kind, n, g, ps, window, sinks):
    c = Case(kind, TM_LENS, g, ps, n, window, sinks, hkv=8, ev=(-20, 10))
    assert 256 * n * g * 8 * len(TM_LENS) * min(9000, window or 9000) >= 2e9
    c.check(splits=(0, 1, 3, 12))


class FewRows(Case):
    """17 to 32 query rows per KV head, enough work and less than 256 MB of cache
    that the tables allow: the tensor-memory kernel, which holds weights 2^7
    times and so cuts them at 2^-32 of the largest."""

    def ref(self, fp32, abort=None):
        return R.attention(self.q_bits, self.k, self.v, self.bt, self.lens, SCALE, self.window, self.sinks,
                           ks=self.ks, vs=self.vs, ke=self.ke, ve=self.ve, abort=abort, fp32=fp32, cut=2.0 ** -32)


@pytest.mark.parametrize("kind", ["fp8", "blocks"])
@pytest.mark.parametrize("n,g,ps", [(3, 8, 16), (5, 4, 64), (16, 2, 32), (4, 8, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (8000, 70)])
def test_tensor_memory_kernel_few_rows(kind, n, g, ps, window, sinks):
    c = FewRows(kind, TM_LENS, g, ps, n, window, sinks, hkv=8, ev=(-20, 10))
    table = 256 * 8 * len(TM_LENS) * 9000
    assert table * n * g * min(1, (window or 9000) / 9000) >= 1.4e9 and 1.05 * table < 256 << 20 and 17 <= n * g <= 32
    abort = (np.arange(len(TM_LENS)) == 5).astype(np.uint8)
    c.check(splits=(0, 1, 7), abort=abort)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 2])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2**30, 3)])
def test_one_long_request_shared_on_the_device(kind, n, window, sinks):
    """Over a hundred splits of a pair in a launch that shares its work out, joined
    by a launch behind it; the other requests fit one split, show nothing or
    name a page that is not there."""
    c = Case(kind, (70001, 0, 33, 1, 200), 5, 64, n, window, sinks, padded=True, hkv=1)
    c.bt[4, 1] = c.desc.num_pages
    c.d["bt"] = torch.from_numpy(c.bt).to(DEV)
    c.check(splits=(0,))


@pytest.mark.parametrize("kind", ["fp8", "blocks"])
def test_tensor_memory_kernel_edges(kind):
    """Scores that rise along the context (the stale maximum is raised tile after
    tile), exponents far apart, a NaN in K and in V, requests that get zeros,
    and a copy wait that gives up."""
    n, g, ps = 8, 8, 16
    c = Case(kind, TM_LENS, g, ps, n, 0, 0, hkv=8, ev=(-48, 48), seed=3)
    big = np.arange(9000)                                   # K of request 7 grows along its positions
    pages = c.bt[7][big // ps]
    grow = R.encode((W.bf16_bits_to_f32(c.q_bits[7, 0, 0]).astype(np.float64)[None, :] * np.linspace(-60, 60, 9000)[:, None]))
    c.k[pages, :, big % ps] = grow[:, None, :]
    c.d["k"] = torch.from_numpy(c.k).to(DEV)
    c.check(splits=(0, 1, 5))
    abort = np.array([0, 0, 0, 1, 0, 0, 0, 0], np.uint8)
    c.bt[0, 7], c.lens[6] = c.desc.num_pages, c.bt.shape[1] * ps + 1
    c.d["bt"], c.d["seq"] = torch.from_numpy(c.bt).to(DEV), torch.from_numpy(c.lens).to(DEV)
    for s in (0, 1, 5):
        got = c.run(True, s, torch.from_numpy(abort).to(DEV))
        for r in (0, 1, 3, 6):
            assert np.all(got[r] == 0.0), (s, r)
        assert np.any(got[7] != 0)
    c = Case(kind, TM_LENS, g, ps, n, 4000, 70, hkv=8)
    c.k[c.bt[0, 4000 // ps], 2, 4000 % ps, 5] = R.NAN_CODE  # seen by every query of request 0
    c.v[c.bt[3, 4000 // ps], 1, 4000 % ps, 9] = R.NAN_CODE
    c.d["k"], c.d["v"] = torch.from_numpy(c.k).to(DEV), torch.from_numpy(c.v).to(DEV)
    for s in (0, 1, 5):
        got = c.run(True, s)
        assert np.isnan(got[0, :, 16:24]).all() and np.isnan(got[0]).sum() == n * 8 * D
        assert np.isnan(got[3, :, 8:16, 9]).all() and np.isnan(got[3]).sum() == n * 8
        assert not np.isnan(got[[1, 2, 4, 5, 6, 7]]).any()
    c = Case(kind, TM_LENS, g, ps, n, 4000, 70, hkv=8)
    ref, bound = c.ref(True)
    try:
        kvq.kvq_diag_set_copy_wait_ns(0)
        got = c.run(True, 3)
    finally:
        kvq.kvq_diag_set_copy_wait_ns(-1)
    bits = kvq.kvq_device_error(clear=True)
    assert bits & 1 and not bits & 2
    assert np.all(got == 0.0)
    R.assert_within(c.run(True, 3), ref, bound, kind)


def test_tensor_memory_kernel_many_splits():
    """More (row, split) weights than the combine's table holds: rows in groups."""
    c = Case("blocks", [70000, 3000], 8, 16, 16, 0, 0, hkv=1, seed=9)
    plan = kvq.kvq_decode_plan_blocks(c.desc, 2, 16, 8, c.bt.shape[1], 0, 0, 128)
    assert plan[1] * 128 > 8192 and 256 * 128 * 2 * 70000 >= 2e9
    c.check(splits=(128, 0), kinds=(True,))


@pytest.mark.parametrize("kind", KINDS)
def test_shared_work_of_many_or_few_requests(kind):
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 200, 700)                        # more requests than threads in a block
    lens[100:300] = 0
    Case(kind, lens, 4, 16, 1, 0, 0, hkv=1, padded=True).check(splits=(0,), kinds=(True,))
    Case(kind, [5], 4, 16, 1, 0, 0, hkv=1, padded=True).check(splits=(0,))
    Case(kind, [0, 0], 4, 16, 2, 0, 0, hkv=1, padded=True).check(splits=(0,))
    # more than one wave of 8,192-token shares would need gigabytes; shares
    # that cross no border, one, and many
    Case(kind, [60000, 1, 1, 30000], 2, 64, 1, 0, 0, hkv=2, padded=True).check(splits=(0,), kinds=(True,))
    Case(kind, [33] * 40 + [20000], 2, 16, 4, 0, 0, hkv=3, padded=True).check(splits=(0,), kinds=(True,))


def test_exponents_far_apart():
    """V exponents over the whole range the append makes, K's chosen so that
    every block keeps some weight: the running maximum of score + exponent, the
    weights' f16 range and the undone sum."""
    Case("blocks", LENS, 4, 16, 1, 0, 0, seed=5, ev=(-48, 48)).check()
    Case("blocks", LENS, 4, 32, 3, 50, 20, seed=6, ev=(-48, 48)).check()
    Case("blocks", LENS, 2, 16, 1, 0, 0, seed=7, ev=(40, 48)).check()
    Case("blocks", LENS, 2, 16, 1, 0, 0, seed=8, ev=(-48, -40)).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,padded", [(1, False), (4, False), (1, True), (4, True)])
def test_requests_that_get_zeros(kind, n, padded):
    c = Case(kind, [300, 0, 77, 500, 40, -5], 4, 16, n, 64 if not padded else 0, 3, padded=padded)
    c.bt[2, 0] = c.desc.num_pages + 3                       # a sink's page out of range
    c.lens[3] = c.bt.shape[1] * 16 + 1                      # longer than its row
    abort = np.array([0, 0, 0, 0, 1, 0], np.uint8)
    c.d["bt"], c.d["seq"] = (torch.from_numpy(x).to(DEV) for x in (c.bt, c.lens))
    for s in (0, 1, 2, 12):
        got = c.run(True, s, torch.from_numpy(abort).to(DEV))
        assert np.all(got[1:] == 0.0) and np.all(np.isfinite(got[0])) and np.any(got[0] != 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [1, 3, 12, 0])
def test_a_nan_that_a_query_sees_reaches_its_output_only(kind, splits):
    """One request with a NaN in K, one with a NaN in one dim of V, one clean."""
    c = Case(kind, [200, 200, 200], 2, 16, 1, 0 if splits == 0 else 100, 3, padded=splits == 0)
    nan = 0x7FC0 if kind == "bf16" else R.NAN_CODE
    for r, name in ((0, "k"), (1, "v")):
        cache = getattr(c, name)
        cache[c.bt[r, 150 // 16], 0, 150 % 16, 5] = nan
        c.d[name] = torch.from_numpy(cache.view(np.int16) if kind == "bf16" else cache).to(DEV)
        if kind == "bf16":
            c.d[name] = c.d[name].view(torch.bfloat16)
    got = c.run(True, splits)
    assert np.isnan(got[0, 0, :2]).all() and not np.isnan(got[0, 0, 2:]).any()     # KV head 0's two heads
    assert np.isnan(got[1, 0, :2, 5]).all() and np.isnan(got[1]).sum() == 2
    assert not np.isnan(got[2]).any()


def test_no_window_agrees_with_the_plain_entry_points():
    c = Case("fp8", LENS, 8, 16, 3, 0, 0)
    d = c.d
    ws = kvq.workspace_for_mt(c.desc, len(LENS), 3, 16, c.bt.shape[1], 4)
    ref = c.out(True)
    kvq.kvq_decode_attn_mt(c.desc, d["q"], d["k"], d["v"], d["s0"], d["s1"], d["bt"], d["seq"], SCALE, None, ref,
                           ws, 4)
    got = c.call(c.out(True), c.workspace(4), 4)
    # not bit for bit: the windowed build keeps its weights 2^15 times larger, so
    # it cuts the small ones elsewhere; both are within the entry points' tolerance
    err = (got - ref).abs()
    assert torch.all(err <= 2e-4 + 2e-4 * ref.abs())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("splits", [12, 0])
def test_captured_replayed_and_on_another_stream(kind, splits):
    """One workspace, a captured graph replayed over new lengths and queries,
    eager calls between; then a stream of its own.  (0: shared on the device,
    where the lengths of the replay count.)"""
    c = Case(kind, [500, 33, 1200], 4, 32, 2, 0 if splits == 0 else 300, 4, padded=splits == 0)
    ws, out = c.workspace(splits), c.out(True)
    c.call(out, ws, splits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(out, ws, splits)
    first, bound = c.ref(True)
    for _ in range(3):
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        R.assert_within(out.cpu().numpy().astype(np.float64), first, bound, "replay")
        eager = c.call(c.out(True), ws, splits)
        torch.cuda.synchronize()
        assert torch.equal(eager, out)
    c.d["seq"].copy_(torch.tensor([0, 33, 900], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.all(out[0] == 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(c.out(True), c.workspace(splits), splits, stream=side)
    side.synchronize()
    assert torch.equal(got, out)


@pytest.mark.parametrize("kind", KINDS)
def test_refusals_with_tensors_on_the_gpu(kind):
    """Tensors that the library cannot take as they are: not contiguous, off a
    16-byte border, on the host, of another shape; a workspace that is too
    small.  Nothing is launched: the output keeps what it held."""
    c = Case(kind, [40, 20], 2, 16, 2, 16, 3)
    ws, out = c.workspace(0), c.out(True)
    q = c.d["q"]
    wide = torch.zeros((*q.shape[:3], 2 * D), dtype=q.dtype, device=DEV)[..., :D]
    shifted = torch.zeros(q.numel() + 1, dtype=q.dtype, device=DEV)[1:].view(q.shape)
    for other, err in ((dict(q=wide), ValueError), (dict(seq=c.d["seq"].cpu()), ValueError),
                       (dict(bt=c.d["bt"][:1]), ValueError), (dict(k=c.d["k"].cpu()), ValueError),
                       (dict(seq=c.d["seq"].long()), TypeError), (dict(q=shifted), kvq.KvqError),
                       (dict(q=None), TypeError), (dict(bt=c.d["bt"][0]), ValueError)):
        with pytest.raises(err):
            c.call(out, ws, **other)
    with pytest.raises(kvq.KvqError) as e:
        c.call(out, ws[:16])
    assert e.value.status == 3
    with pytest.raises(kvq.KvqError):
        c.call(out, None)
    with pytest.raises(OverflowError):
        c.call(out, ws, splits=2**31)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)
    # a stream given as a handle
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(c.out(True), ws, stream=side.cuda_stream)
    side.synchronize()
    ref, bound = c.ref(True)
    R.assert_within(got.cpu().numpy().astype(np.float64), ref, bound, "handle")


def test_two_calls_at_once_with_workspaces_of_their_own():
    a = Case("blocks", [3000, 700, 41], 8, 16, 1, 0, 0, hkv=2, padded=True)
    b = Case("fp8", [9000, 33], 4, 16, 4, 2000, 5)
    wa, wb = a.workspace(0), b.workspace(12)
    ra, ba = a.ref(True)
    rb, bb = b.ref(True)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        oa = a.call(a.out(True), wa, 0, stream=streams[0])
        ob = b.call(b.out(True), wb, 12, stream=streams[1])
    torch.cuda.synchronize()
    R.assert_within(oa.cpu().numpy().astype(np.float64), ra, ba, "first")
    R.assert_within(ob.cpu().numpy().astype(np.float64), rb, bb, "second")


def test_one_workspace_under_changing_lengths_windows_and_graphs():
    """Two graphs captured over one workspace (as documented: the same batch,
    heads and query tokens) and replayed in turn with an eager call between."""
    c = Case("fp8", [5000, 64, 900], 4, 16, 1, 0, 0)
    ws = torch.zeros(max(c.workspace(0).numel(), 1 << 22), dtype=torch.uint8, device=DEV)
    outs, graphs, refs = [], [], []
    for window, splits in ((0, 12), (700, 12), (700, 0), (0, 0)):
        c.window = window
        refs.append(R.attention(c.q_bits, c.k, c.v, c.bt, c.lens, SCALE, window, 0, ks=c.ks, vs=c.vs, fp32=True))
        out = c.call(c.out(True), ws, splits)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(out, ws, splits)
        outs.append(out)
        graphs.append(g)
    for order in ((0, 1, 2, 3), (3, 1, 0, 2)):
        for i in order:
            outs[i].fill_(5.0)
            graphs[i].replay()
            torch.cuda.synchronize()
            R.assert_within(outs[i].cpu().numpy().astype(np.float64), *refs[i], f"graph {i}")


def test_wait_limit_of_the_new_builds():
    """A copy wait that gives up at once: the bit, zeros, and the next call is right."""
    for kind in KINDS:
        for splits in (4, 0):
            c = Case(kind, [4096, 300], 4, 16, 1, 0 if splits == 0 else 3000, 4, padded=splits == 0)
            ref, bound = c.ref(True)
            try:
                kvq.kvq_diag_set_copy_wait_ns(0)
                got = c.run(True, splits)
            finally:
                kvq.kvq_diag_set_copy_wait_ns(-1)
            bits = kvq.kvq_device_error(clear=True)
            assert bits & 1 and not bits & 2
            assert np.all(got == 0.0)
            R.assert_within(c.run(True, splits), ref, bound, kind)


# ------------------------------------------------------------- tag check

@pytest.mark.parametrize("ps", [16, 128])
@pytest.mark.parametrize("window,sinks,n", [(0, 0, 1), (1, 0, 1), (40, 5, 3), (5000, 200, 16), (2**31 - 1, 2**31 - 1, 1)])
def test_tag_check_window(ps, window, sinks, n):
    rng = np.random.default_rng([ps, window, n])
    lens = np.array(list(LENS) * 12 + [70000, 100001, -3], np.int32)
    B, N = len(lens), 9000
    maxp = 100000 // ps                                     # the last long request does not fit
    bt = rng.integers(0, N, (B, maxp)).astype(np.int32)
    tags = rng.integers(0, 2**32, N, dtype=np.uint64).astype(np.uint32)
    exp = tags[bt]
    for r in range(B):                                      # unseen entries poisoned; a wrong one somewhere in half
        L = max(int(lens[r]), 0)
        used = -(-L // ps)
        see = R.view_mask(L, n, window, sinks).any(axis=0)
        held = np.zeros(max(maxp, used), bool)
        held[np.flatnonzero(see) // ps] = True
        # pages of the sinks and the window whose positions no query sees are still looked at
        held = held[:maxp]
        unseen = ~held
        first = -(-min(L, sinks) // ps) if window else 0
        last = max(0, L - n + 1 - window) // ps if window else 0
        unseen[:first] = False
        unseen[last:used] = False
        exp[r, unseen] ^= 1
        bt[r, unseen & (rng.random(maxp) < .5)] = -7
        if r % 2 and used:
            i = rng.integers(0, min(used, maxp))
            if r % 4 == 1:
                exp[r, i] ^= 4
            else:
                bt[r, i] = N
    want = R.tag_check(bt, exp, lens, ps, tags, window, sinks, n)
    assert 0 < want.sum() < B
    t = lambda x: torch.from_numpy(x.view(np.int32)).to(DEV)  # noqa: E731
    got = torch.full((B,), 9, dtype=torch.uint8, device=DEV)
    kvq.kvq_tag_check_window(t(bt), t(exp), t(lens), ps, t(tags), window, sinks, n, got)
    assert np.array_equal(got.cpu().numpy(), want)
    if window == 0:
        got2 = torch.full((B,), 9, dtype=torch.uint8, device=DEV)
        kvq.kvq_tag_check(t(bt), t(exp), t(lens), ps, t(tags), got2)
        assert torch.equal(got, got2)
