"""GPU parity of the attention over shared prefixes against plain fp64, with the bounds of view_ref: every request over
its own row.  Whatever no request sees -- K, V and exponents of other slots, table entries -- is poisoned.

Small calls run each request apart; tables padded past the border (``pad=WIDE``) make the call share.  Of those the
entries of a request's own shared pages are poisoned too, where so many share that the other row is read."""
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
KINDS = ("fp8", "bf16", "blocks")
WIDE = "wide"                                               # tables that allow 512 MB of cache


@pytest.fixture(autouse=True)
def _no_device_errors():
    kvq.kvq_device_error(clear=True)
    yield
    torch.cuda.synchronize()
    assert kvq.kvq_device_error() == 0


class Case:
    """Groups of requests that share whole pages: (prefix, [own tokens of each request]).  Request r of a group holds
    prefix + own[r] tokens; a group of one, or a prefix of None, shares nothing."""

    def __init__(self, kind, groups, g, ps, n, hkv=2, seed=0, ev=(-10, 3), pad=WIDE, poison_own=True,
                 q_scale=1.0):
        rng = np.random.default_rng([seed, n, g, ps])
        self.kind, self.n, self.ps, self.g, self.hkv = kind, n, ps, g, hkv
        lens, lead, shared, rows, used = [], [], [], [], 0
        for prefix, own in groups:
            first, alone = len(lens), len(own) == 1 or prefix is None
            whole = 0 if alone else prefix // ps
            common = list(range(used, used + whole))
            used += whole
            copy_of = None
            for o in own:
                L = (prefix or 0) + o
                mine = max(0, -(-L // ps) - whole)
                row = common[:max(0, -(-L // ps))] + list(range(used, used + mine))
                if not alone and prefix % ps and copy_of is None and mine:
                    copy_of = (row[whole], prefix % ps)
                rows.append((row, whole, copy_of))
                used += mine
                lens.append(L)
                lead.append(first if not alone else rng.choice([-1, -7, len(groups) * 1000]))
                shared.append(prefix if not alone else rng.choice([0, -3, 5]))
        B, N = len(lens), used + 3
        if pad == WIDE:
            pad = -(-(512 << 20) // (256 * B * hkv * ps))
        self.sharing = pad > 0
        self.lens, self.lead, self.shared = (np.asarray(x, np.int32) for x in (lens, lead, shared))
        perm = rng.permutation(N).astype(np.int32)
        maxp = max(1, max(len(r[0]) for r in rows)) + pad
        self.bt = rng.choice([-1, N, 2**31 - 1, -2**31], (B, maxp)).astype(np.int32)
        for r, (row, _, _) in enumerate(rows):
            self.bt[r, :len(row)] = perm[row]
        shape = (N, hkv, ps, D)
        nan = 0x7FC0 if kind == "bf16" else R.NAN_CODE
        values = [rng.standard_normal(shape) for _ in range(2)]
        if kind == "bf16":
            full = [W.f32_to_bf16_bits(x.astype(np.float32)) for x in values]
        else:
            full = [R.encode(x * 90) for x in values]
        e = [rng.integers(-11, -5, (N, hkv, ps // 16)), rng.integers(ev[0], ev[1] + 1, (N, hkv, ps // 16))]
        for r, (row, whole, copy_of) in enumerate(rows):    # a copied page's first tokens are its origin's
            if copy_of is not None and len(row) > whole:
                to, src, m = perm[row[whole]], perm[copy_of[0]], copy_of[1]
                for x in full:
                    x[to, :, :m] = x[src, :, :m]
                for x in e:
                    x[to] = x[src]
        self.k, self.v = (np.full(shape, nan, x.dtype) for x in full)
        self.ks, self.vs = (rng.uniform(0.006, 0.02, hkv).astype(np.float32) for _ in range(2))
        self.ke = self.ve = None
        if kind == "blocks":
            self.ke, self.ve = (np.where(rng.random(x.shape) < .5, 127, -128).astype(np.int8) for x in e)
        for r in range(B):
            pos = np.arange(max(0, int(self.lens[r])))
            pages = self.bt[r][pos // ps]
            for dst, src in ((self.k, full[0]), (self.v, full[1])):
                dst[pages, :, pos % ps] = src[pages, :, pos % ps]
            if kind == "blocks":
                for dst, src in ((self.ke, e[0]), (self.ve, e[1])):
                    dst[pages, :, pos % ps // 16] = src[pages, :, pos % ps // 16]
        self.q_bits = W.normal_bf16(rng, (B, n, hkv * g, D))
        if q_scale != 1.0:
            self.q_bits = W.f32_to_bf16_bits(W.bf16_bits_to_f32(self.q_bits) * np.float32(q_scale))
        self.desc = kvq.CacheDesc(N, ps, hkv, D, kvq.KVQ_CACHE_BF16 if kind == "bf16" else kvq.KVQ_CACHE_FP8_E4M3)
        # what the call is given: own entries of shared pages may hold anything
        self.given = self.bt.copy()
        if poison_own and self.sharing:
            for r in range(B):
                if 0 <= self.lead[r] < B and self.lead[r] != r and (self.lead == self.lead[r]).sum() >= 8:
                    w = min(int(self.shared[r]), int(self.lens[self.lead[r]]), int(self.lens[r]) - n + 1)
                    self.given[r, :max(0, w) // max(ps, 64) * max(ps, 64) // ps] = N + 7
        self.upload()

    def upload(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        bf = lambda x: t(x.view(np.int16)).view(torch.bfloat16)  # noqa: E731
        bf16 = self.kind == "bf16"
        self.d = dict(k=bf(self.k) if bf16 else t(self.k), v=bf(self.v) if bf16 else t(self.v), bt=t(self.given),
                      seq=t(self.lens), q=bf(self.q_bits), lead=t(self.lead), shared=t(self.shared))
        blocks = self.kind == "blocks"
        self.d.update(s0=t(self.ke if blocks else self.ks), s1=t(self.ve if blocks else self.vs))

    def workspace(self):
        return kvq.workspace_for_prefix(self.desc, len(self.lens), self.n, self.q_bits.shape[2], self.bt.shape[1])

    def call(self, out, ws, abort=None, stream=None, scale=SCALE, **other):
        d = {**self.d, **other}
        fn = kvq.kvq_decode_attn_prefix_blocks if self.kind == "blocks" else kvq.kvq_decode_attn_prefix
        return fn(self.desc, d["q"], d["k"], d["v"], d["s0"], d["s1"], d["bt"], d["seq"], d["lead"], d["shared"],
                  scale, abort, out, ws, stream)

    def out(self, fp32):
        return torch.full(self.q_bits.shape, 7.0, dtype=torch.float32 if fp32 else torch.bfloat16, device=DEV)

    def run(self, fp32, abort=None, scale=SCALE):
        ws = self.workspace()
        ws.fill_(255)                                       # no contents are needed: NaN, ids of -1
        out = self.call(self.out(fp32), ws, abort, scale=scale)
        torch.cuda.synchronize()
        return out.float().cpu().numpy().astype(np.float64)

    def ref(self, fp32, abort=None, scale=SCALE):
        return R.attention(self.q_bits, self.k, self.v, self.bt, self.lens, scale, 0, 0, ks=self.ks, vs=self.vs,
                           ke=self.ke, ve=self.ve, abort=abort, fp32=fp32, cut=2.0 ** -32)

    def check(self, kinds=(False, True), abort=None, what="", scale=SCALE):
        t = None if abort is None else torch.from_numpy(abort).to(DEV)
        for fp32 in kinds:
            R.assert_within(self.run(fp32, t, scale), *self.ref(fp32, abort, scale), f"{what} fp32={fp32}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ps,g", [(16, 8), (64, 3), (128, 1)])
@pytest.mark.parametrize("pad", [0, WIDE])
def test_one_query_token(kind, ps, g, pad):
    """Prefixes of every kind of end, own parts from none to several pages, groups of one, two and more, empty
    requests."""
    Case(kind, [(5 * ps, [1, 2, ps, 3 * ps + 1, 0, 9, 1, 1, ps - 1]), (None, [0]), (ps - 1, [1, 3] * 5),
                (7 * ps + 5, [1, 40, 0, 300, 5, 5, 5, ps]), (1000, [17]), (33 * ps, [0, 0, 1] * 3), (64, [7, 8]),
                (0, [5, 0])], g, ps, 1, pad=pad).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,g,ps", [(2, 1, 32), (4, 4, 16), (5, 8, 128), (16, 8, 16), (11, 7, 64)])
@pytest.mark.parametrize("pad", [0, WIDE])
def test_several_query_tokens(kind, n, g, ps, pad):
    """Own parts shorter than the drafts, so that queries stand inside the shared pages; contexts shorter than them."""
    Case(kind, [(5 * ps, [n, 1, 0, n - 1, 2 * ps, n, n, n + 1, 3]), (None, [1, n - 1, n, 100]), (400, [n, n + 1, 70])],
         g, ps, n, pad=pad).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,g", [(15, 8), (16, 8), (17, 8), (32, 8), (33, 8), (70, 7), (128, 3), (130, 1)])
def test_rows_around_the_tiles(kind, m, g):
    """120 to 512 rows of a KV head: one row tile, both, and more pairs of them."""
    rng = np.random.default_rng(m)
    Case(kind, [(700, [int(x) for x in rng.integers(1, 50, m)])], g, 16, 1, hkv=1).check()


@pytest.mark.parametrize("kind", KINDS)
def test_long_prefixes(kind):
    """Shares of many tiles, so that fp32 sums leave tensor memory on the way, and several CTAs per row pair."""
    Case(kind, [(70000, [1, 300] + [7] * 6), (20000, [5, 5, 9000, 1, 1, 1, 1, 1])], 2, 64, 1, hkv=1).check()
    Case(kind, [(160000, [3] * 9)], 2, 16, 4, hkv=1).check(kinds=(True,))


@pytest.mark.parametrize("kind", KINDS)
def test_many_small_groups(kind):
    """Runs that cross every 128th request, among them."""
    rng = np.random.default_rng(5)
    groups = [(int(rng.integers(0, 300)), [int(x) for x in rng.integers(0, 60, rng.integers(1, 12))]) for _ in range(100)]
    Case(kind, groups, 2, 16, 1).check()


@pytest.mark.parametrize("kind", KINDS)
def test_requests_with_prefixes_of_their_own_lengths(kind):
    """One row serves requests that share more and less of it, and more than it or they hold."""
    c = Case(kind, [(900, [1, 50, 9, 400, 2] * 3)], 5, 16, 1, poison_own=False)
    c.shared[:] = (16, 900, 2**31 - 1, 333, 15) * 3
    c.upload()
    c.check()
    c.lead[:] = [0] * 5 + [12] * 9 + [-1]                   # two runs
    c.upload()
    c.check()
    c.lead[:] = 2**31 - 1
    c.upload()
    c.check()


@pytest.mark.parametrize("kind", KINDS)
def test_aborted_requests_and_leaders(kind):
    """An aborted request gets zeros; requests whose leader is aborted read their own rows."""
    groups = [(200, [3, 40, 7] * 3), (100, [1, 20] * 4)]
    for which in ([1, 5], [0, 16], [0, 9, 10], range(17)):
        abort = np.zeros(17, np.uint8)
        abort[list(which)] = 3
        Case(kind, groups, 4, 16, 1, poison_own=False).check(abort=abort)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_are_too_short_and_bad_pages(kind):
    c = Case(kind, [(640, [5, 70, 5, 30] * 3), (300, [9, 9] * 4)], 4, 16, 2, poison_own=False)
    c.given[0, 20] = -1                                     # a shared page of the first group
    c.lens[13] = 10**7                                      # longer than its row
    c.given[3, 41] = c.desc.num_pages                       # a page of request 3's own
    c.shared[3] = 300                                       # 18 pages: below the bad one
    c.upload()
    ref, bound = c.ref(True)
    right = [12] + list(range(14, 20))
    got = c.run(True)
    R.assert_within(got[right], ref[right], bound[right])
    assert not got[:12].any() and not got[13].any()
    c.given[3, 41] = c.bt[3, 41]
    c.upload()
    right.append(3)
    got = c.run(True)
    R.assert_within(got[right], ref[right], bound[right])
    assert not np.delete(got, right, axis=0).any()


@pytest.mark.parametrize("kind", KINDS)
def test_nan_reaches_those_who_see_it(kind):
    c = Case(kind, [(320, [20] * 9), (160, [30, 1] * 4)], 2, 16, 1)
    nan = 0x7FC0 if kind == "bf16" else R.NAN_CODE
    c.v[c.bt[0, 3], 0, 5, 7] = nan                          # a shared V row of the first group
    c.v[c.bt[9, 10], 1, 0, 100] = nan                       # request 9's own
    c.upload()
    for fp32 in (False, True):
        ref, bound = c.ref(fp32)
        assert np.isnan(ref[:9, :, :2, 7]).all() and np.isnan(ref).sum() == 9 * 2 + 2
        R.assert_within(c.run(fp32), ref, bound, f"fp32={fp32}")
    c.k[c.bt[0, 4], 1, 2, 3] = nan                          # a shared K row: every weight of the other head's rows
    c.upload()
    got, (ref, bound) = c.run(True), c.ref(True)
    assert np.isnan(got[:9, :, 2:]).all()
    for at in ((slice(9), slice(None), slice(2)), (slice(9, 17),)):
        R.assert_within(got[at], ref[at], bound[at])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ps,m,g,n", [(16, 1, 3, 1), (64, 2, 8, 1), (128, 1, 5, 4)])
def test_no_request_meets_what_stands_behind_its_end(kind, ps, m, g, n):
    """Requests that end inside the others' prefix, one and two row tiles: NaN and infinities in V past their ends."""
    own = ([10] * 4 + [-100, -700, -1500, -2000, 0, -2100]) * m
    c = Case(kind, [(2112, own)], g, ps, n)
    nan, inf = (0x7FC0, 0x7F80) if kind == "bf16" else (R.NAN_CODE, R.NAN_CODE)
    for x, places in ((nan, ((2105, 0, 5), (2050, 1, 9), (1999, 0, 77), (1000, 1, 3), (100, 0, 2))),
                      (inf, ((2100, 0, 6), (1200, 1, 8)))):
        for pos, h, d in places:
            c.v[c.bt[0, pos // ps], h, pos % ps, d] = x
    c.upload()
    for fp32 in (False, True):
        got, (ref, bound) = c.run(fp32), c.ref(fp32)
        spoilt = ~np.isfinite(ref)
        # (a page that the prefix does not fill is request 0's alone)
        seen = [7] + [7 if 2112 % ps == 0 else 4] * 3
        assert spoilt[:4].any(axis=(1, 2)).sum(axis=1).tolist() == seen and not spoilt[9].any()
        assert not np.isfinite(got[spoilt]).any()
        R.assert_within(got[~spoilt], ref[~spoilt], bound[~spoilt], f"fp32={fp32}")


@pytest.mark.parametrize("kind", KINDS)
def test_sums_that_leave_tensor_memory(kind):
    """1,024 rows over one prefix, 37 tiles of both row tiles a CTA: fp32 sums go out on the way, and some rows' for good."""
    own = [20, 40, -30000, 17, -60000, 20, -100, 33]
    c = Case(kind, [(90000, own)], 8, 16, 16, hkv=1)
    for pos in (89990, 80001, 59950, 45000):
        c.v[c.bt[0, pos // 16], 0, pos % 16, pos % 128] = 0x7FC0 if kind == "bf16" else R.NAN_CODE
    c.upload()
    got, (ref, bound) = c.run(True), c.ref(True)
    assert [np.isnan(x).any(axis=(0, 1)).sum() for x in ref] == [4, 4, 2, 4, 0, 4, 3, 4]
    R.assert_within(got, ref, bound)


def test_large_values_over_a_bf16_cache():
    """Values near bf16's largest, of one sign: sums of weights do not leave fp32."""
    c = Case("bf16", [(3000, [10, 600] * 4)], 4, 16, 1, hkv=1)
    big = W.f32_to_bf16_bits(np.full(c.v.shape, 2.0 ** 120, np.float32))
    seen = c.v != 0x7FC0
    c.v = np.where(seen, big, c.v)
    c.upload()
    for fp32 in (False, True):
        got = c.run(fp32)
        assert np.allclose(got, 2.0 ** 120, rtol=2.0 ** -8)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale,q_scale", [(-SCALE, 1.0), (0.0, 1.0), (SCALE, 300.0), (SCALE * 40, 1.0), (SCALE, 2.0 ** -100)])
def test_scales(kind, scale, q_scale):
    """Negative and zero softmax scales, peaked and flat softmaxes (the maximum rises by thousands), tiny queries."""
    Case(kind, [(1500, [3, 200, 50] * 3)], 3, 32, 1, q_scale=q_scale).check(scale=scale)


@pytest.mark.parametrize("ev", [(-48, 48), (-128, 127)])
def test_far_value_exponents(ev):
    c = Case("blocks", [(900, [3, 200, 50] * 3)], 3, 16, 1, ev=ev)
    c.ve = np.clip(c.ve, -48, 48)                           # how they are read
    for fp32 in (False, True):
        R.assert_within(c.run(fp32), *c.ref(fp32), f"fp32={fp32}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [0, WIDE])
@pytest.mark.parametrize("n", [1, 4])
def test_calls_repeat_bit_for_bit_and_need_no_workspace_contents(kind, pad, n):
    c = Case(kind, [(3000, [10, 600, 4] * 3), (700, [5, 5])], 8, 16, n, pad=pad)
    ws = c.workspace()
    a = c.call(c.out(True), ws).clone()
    b = c.call(c.out(True), ws)
    ws.fill_(255)
    d = c.call(c.out(True), ws)
    assert torch.equal(a, b) and torch.equal(a, d)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pad", [0, WIDE])
def test_a_graph_follows_lengths_and_another_stream(kind, pad):
    """A captured call replayed after the lengths, flags and tables changed in place."""
    c = Case(kind, [(640, [5, 70, 300] * 3), (200, [9, 9, 400] * 3)], 4, 16, 1, poison_own=False, pad=pad)
    ws, out = c.workspace(), c.out(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.call(out, ws)
    c.call(out, ws, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(out, ws)
    for lens, shared in (([100, 30, 1] * 3 + [0, 209, 600] * 3, [90, 16, 0] * 3 + [50, 48, 200] * 3),
                         ([645, 710, 940] * 3 + [209, 209, 1] * 3, [640] * 9 + [200] * 9)):
        c.lens[:], c.shared[:] = lens, shared
        c.d["seq"].copy_(torch.from_numpy(c.lens))
        c.d["shared"].copy_(torch.from_numpy(c.shared))
        graph.replay()
        torch.cuda.synchronize()
        R.assert_within(out.cpu().numpy().astype(np.float64), *c.ref(True))


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_two_calls_at_once(kind):
    """On two streams with a workspace each."""
    cs = [Case(kind, [(2000 + 100 * i, [10, 60, 1] * 3)], 4, 16, 1, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cs]
    ws, outs = [c.workspace() for c in cs], [c.out(True) for c in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, w, o in zip(cs, streams, ws, outs):
            c.call(o, w, stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cs, outs):
        R.assert_within(o.cpu().numpy().astype(np.float64), *c.ref(True))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(9, 1), (40, 4)])
def test_copy_wait_timeout_zeroes_and_recovers(kind, m, n):
    """Every wait for a copy gives up at once: zeros for what was served, no copy left in flight, and the next call
    is right."""
    c = Case(kind, [(9000, [5] * m)], 4, 16, n)
    try:
        kvq.kvq_diag_set_copy_wait_ns(0)
        got = c.run(True)
    finally:
        kvq.kvq_diag_set_copy_wait_ns(-1)
    bits = kvq.kvq_device_error(clear=True)
    assert bits & 1 and not bits & 2
    assert not got.any()
    c.check()


@pytest.mark.parametrize("pad", [0, WIDE])
def test_an_empty_batch_and_no_sharing_at_all(pad):
    c = Case("fp8", [(None, [100]), (None, [1]), (None, [0])], 4, 16, 1, pad=pad)
    c.check()
    c.lens[:] = 0
    c.upload()
    assert not c.run(True).any()
    c2 = Case("fp8", [(64, [3, 3])], 1, 16, 1, hkv=1, pad=pad)
    e = lambda *s: torch.empty(s, dtype=torch.int32, device=DEV)  # noqa: E731
    q = torch.empty((0, 1, 1, D), dtype=torch.bfloat16, device=DEV)
    kvq.kvq_decode_attn_prefix(c2.desc, q, c2.d["k"], c2.d["v"], c2.d["s0"], c2.d["s1"], e(0, 4), e(0), e(0), e(0),
                               SCALE, None, q.clone(), c2.workspace())


def _against_the_unshared_call(desc, q, k, v, bt, lens, lead, shared, sample):
    """All rows against kvq_decode_attn_window (both are within 2e-4 + 2e-4 |o|), some against 64 bits."""
    n, hq = q.shape[1], q.shape[2]
    s = torch.full((desc.num_kv_heads,), 0.011, device=DEV)
    out, plain = (torch.full(q.shape, 7.0, dtype=torch.float32, device=DEV) for _ in range(2))
    ws = kvq.workspace_for_prefix(desc, len(lens), n, hq, bt.shape[1])
    kvq.kvq_decode_attn_prefix(desc, q, k, v, s, s, bt, lens, lead, shared, SCALE, None, out, ws)
    ws = kvq.workspace_for_window(desc, len(lens), n, hq, bt.shape[1], 0)
    kvq.kvq_decode_attn_window(desc, q, k, v, s, s, bt, lens, SCALE, 0, 0, None, plain, ws)
    assert ((out - plain).abs() <= 4e-4 * (1 + plain.abs())).all()
    bits = lambda x: x.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    for r in sample:
        pages = bt[r, :-(-int(lens[r]) // desc.page_size)].long()
        kc, vc = k[pages], v[pages]
        kc, vc = (bits(x) if x.dtype == torch.bfloat16 else x.cpu().numpy() for x in (kc, vc))
        ref, bound = R.attention(bits(q[r:r + 1]), kc, vc, np.arange(len(pages), dtype=np.int32)[None],
                                 lens[r:r + 1].cpu().numpy(), SCALE, 0, 0, ks=s.cpu().numpy(), vs=s.cpu().numpy(),
                                 fp32=True, cut=2.0 ** -32)
        R.assert_within(out[r:r + 1].cpu().numpy().astype(np.float64), ref, bound, f"request {r}")


def test_the_largest_batch():
    """65,535 requests in runs of 1,000, 64 shared tokens and up to 48 of their own each."""
    B, N = 65535, 65535 * 3 + 4
    g = torch.Generator(device=DEV).manual_seed(3)
    desc = kvq.CacheDesc(N, 16, 1, D, kvq.KVQ_CACHE_FP8_E4M3)
    k, v = (torch.randint(0, 120, (N, 1, 16, D), dtype=torch.uint8, device=DEV, generator=g) +
            torch.randint(0, 2, (N, 1, 16, D), dtype=torch.uint8, device=DEV, generator=g) * 128 for _ in range(2))
    q = torch.randn((B, 1, 2, D), device=DEV, generator=g).bfloat16() * 0.02
    r = torch.arange(B, dtype=torch.int32, device=DEV)
    bt = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    bt[:, :4] = torch.arange(4, dtype=torch.int32, device=DEV)
    bt[:, 4:7] = 4 + 3 * r[:, None] + torch.arange(3, dtype=torch.int32, device=DEV)
    lens = 64 + r % 49
    assert kvq.kvq_decode_plan_prefix(desc, B, 1, 2, 8) > 152 * 256 * 512       # shared
    _against_the_unshared_call(desc, q, k, v, bt, lens, r // 1000 * 1000, torch.full_like(r, 64), (0, 999, 1000, 33333, 65534))


@pytest.mark.parametrize("kind", ["fp8", "bf16"])
def test_pages_past_four_gigabytes_of_a_cache(kind):
    """Wide table rows, and pages whose places in the caches pass 32 bits."""
    ps, hkv, B = 64, 2, 40
    page_bytes = hkv * ps * D * (2 if kind == "bf16" else 1)
    N = (5 << 30) // page_bytes
    desc = kvq.CacheDesc(N, ps, hkv, D, kvq.KVQ_CACHE_BF16 if kind == "bf16" else kvq.KVQ_CACHE_FP8_E4M3)
    g = torch.Generator(device=DEV).manual_seed(4)
    dtype = torch.bfloat16 if kind == "bf16" else torch.uint8
    k, v = (torch.empty((N, hkv, ps, D), dtype=dtype, device=DEV) for _ in range(2))
    used = 30 + 2 * B
    for x in (k, v):
        shape = (used, hkv, ps, D)
        x[N - used:] = (torch.randn(shape, device=DEV, generator=g).bfloat16() if kind == "bf16" else
                        torch.randint(0, 120, shape, dtype=torch.uint8, device=DEV, generator=g))
    q = torch.randn((B, 1, 2 * hkv, D), device=DEV, generator=g).bfloat16() * 0.1
    r = torch.arange(B, dtype=torch.int32, device=DEV)
    bt = torch.full((B, 1 << 16), -1, dtype=torch.int32, device=DEV)
    bt[:, :30] = N - 1 - torch.arange(30, dtype=torch.int32, device=DEV)
    bt[:, 30:32] = N - used + 2 * r[:, None] + torch.arange(2, dtype=torch.int32, device=DEV)
    _against_the_unshared_call(desc, q, k, v, bt, 30 * ps + 1 + r, r // 20 * 20, torch.full_like(r, 30 * ps), (0, 19, 20, 39))
