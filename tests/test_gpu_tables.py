"""Page tables kept on the GPU against the plain model: whole state after each call, so every number is compared."""
import random

import pytest

torch = pytest.importorskip("torch")

import fp8_quantised_paged_kv_gb300 as kvq
from tests.tables_ref import Tables

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """The model and the GPU's state, put through the same calls."""

    def __init__(self, num_pages, ps, batch, maxp, tags=True):
        self.ref = Tables(num_pages, ps, batch, maxp)
        self.pool = kvq.PagePool.create(num_pages, ps, device=DEV, tags=tags)
        self.seq = torch.zeros(batch, dtype=torch.int32, device=DEV)
        self.bt = torch.full((batch, maxp), -1, dtype=torch.int32, device=DEV)
        self.expected = torch.zeros((batch, maxp), dtype=torch.int32, device=DEV) if tags else None
        self.refused = torch.full((batch,), 7, dtype=torch.uint8, device=DEV)
        self.src, self.dst = (torch.full((batch,), 7, dtype=torch.int32, device=DEV) for _ in range(2))

    def push(self):
        """The model's state onto the GPU."""
        self.seq.copy_(i32(self.ref.seq))
        self.bt.copy_(i32(self.ref.rows))

    def check(self):
        torch.cuda.synchronize()
        r = self.ref
        assert self.seq.tolist() == r.seq
        assert self.bt.tolist() == r.rows
        assert self.pool.free_count.item() == r.count
        assert self.pool.free_pages.tolist() == r.free
        assert self.pool.page_refs.tolist() == r.refs
        if self.expected is not None:
            assert self.pool.page_tags.tolist() == r.tags and self.expected.tolist() == r.expected
        assert not self.pool.scratch.any()

    def extend(self, lens, stream=None, even=False):
        offsets = [0]
        for n in lens:
            offsets.append(offsets[-1] + n)
        return self.extend_at(offsets, offsets[-1], stream, even)

    def extend_at(self, offsets, total, stream=None, even=False):
        slots = torch.full((total,), -99, dtype=torch.int64, device=DEV)
        kvq.kvq_extend_tables(self.pool, None if even else i32(offsets), total, self.seq, self.bt, self.expected,
                              slots, self.refused, stream)
        want, refused = self.ref.extend(offsets, total)
        assert slots.tolist() == [-99 if w is None else w for w in want]
        assert self.refused.tolist() == refused
        self.check()
        return refused

    def fork(self, parents, lens):
        kvq.kvq_fork_tables(self.pool, i32(parents), i32(lens), self.seq, self.bt, self.expected, self.src, self.dst,
                            self.refused)
        src, dst, refused = self.ref.fork(parents, lens)
        assert (self.src.tolist(), self.dst.tolist(), self.refused.tolist()) == (src, dst, refused)
        self.check()
        return refused

    def trim(self, keep):
        kvq.kvq_trim_tables(self.pool, i32(keep), self.seq, self.bt)
        self.ref.trim(keep)
        self.check()


@pytest.mark.parametrize("batch,ps,tags", [(1, 16, True), (5, 16, True), (37, 32, False), (300, 64, True), (700, 128, True)])
def test_a_random_run(batch, ps, tags):
    """Prompts, forks, decode steps, drafts and finished requests; the pool runs out now and then."""
    rng = random.Random(batch)
    maxp = 12
    b = Both(batch * 5 + 1, ps, batch, maxp, tags)
    refusals = 0
    for step in range(12):
        kind = rng.randrange(5)
        if kind == 0:                                       # prompts and chunks of them
            refusals += sum(b.extend([rng.choice([0, 1, ps, ps + 1, rng.randint(0, 4 * ps)]) for _ in range(batch)]))
        elif kind == 1:
            b.extend([1] * batch, even=True)
        elif kind == 2:
            parents = [rng.choice([-1, rng.randrange(batch + 1)]) for _ in range(batch)]
            lens = [rng.randint(0, max(b.ref.seq[p], 0)) if 0 <= p < batch else 3 for p in parents]
            refusals += sum(b.fork(parents, lens))
        else:                                               # finished ones, and a few tokens of others
            b.trim([rng.choice([-1, 0, 0, max(0, b.ref.seq[r] - rng.randint(0, ps)), 10 ** 6]) for r in range(batch)])
    b.trim([0] * batch)
    assert b.ref.count == b.ref.n and sorted(b.ref.free) == list(range(b.ref.n))
    assert refusals or batch == 1


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 63, 64, 65, 4095, 4096, 20001])
def test_one_request(tokens):
    b = Both(4000, 16, 1, 1300)
    b.extend([tokens])
    b.extend([tokens % 700])
    b.trim([tokens // 2])
    b.extend([3], even=True)


@pytest.mark.parametrize("batch", [255, 256, 257, 3001])
def test_many_requests(batch):
    """Several CTAs, each with several requests."""
    b = Both(2 * batch, 16, batch, 6)
    rng = random.Random(3)
    b.extend([1] * batch, even=True)
    b.extend([rng.randint(0, 40) for _ in range(batch)])    # more than the pool holds
    b.fork([(r - 1) // 2 if b.ref.seq[r] == 0 else -1 for r in range(batch)], [17] * batch)
    b.trim([rng.choice([0, 1, 17, -1]) for _ in range(batch)])
    b.fork([0 if r and b.ref.seq[r] == 0 else -1 for r in range(batch)], [b.ref.seq[0]] * batch)
    b.trim([0] * batch)
    assert b.ref.count == b.ref.n


def test_long_prompts_in_parts():
    """Few requests of many tokens: several CTAs share a request."""
    b = Both(5000, 64, 3, 2000)
    b.extend([100000, 7, 60001])
    b.extend([1, 50000, 0])
    b.trim([5, 0, 60000])


def test_refused_requests_keep_what_they_have():
    b = Both(10, 16, 4, 8)
    assert b.extend([40, 0, 0, 30]) == [0, 0, 0, 0]         # 3 and 2 pages of 10
    assert b.extend([8, 96, 1, 2]) == [0, 1, 1, 0]          # room without a page; 6 of 5; the next one's want is past it
    assert b.extend([8, 80, 1, 1]) == [0, 1, 1, 1]          # 1 + 5 of 5, and more after them
    assert b.extend([0, 64, 129, 0]) == [0, 0, 1, 0]        # a row of 8 pages
    assert b.fork([-1, -1, 1, -1], [0, 0, 64, 0]) == [0, 0, 0, 0]
    assert b.extend([9, 0, 0, 0]) == [1, 0, 0, 0]           # nothing is left
    b.trim([0, 0, -1, 0])
    assert b.ref.count == 6


def test_forks_that_are_refused():
    b = Both(6, 16, 6, 4)
    b.extend([33, 5, 0, 0, 0, 0])
    #          itself, holds tokens, longer than the parent, past the batch, negative length, not asked
    assert b.fork([0, 0, 1, 6, 0, -1], [1, 1, 6, 0, -1, 0]) == [1, 1, 1, 1, 1, 0]
    assert b.fork([-1, -1, 0, 0, 0, 0], [0, 0, 33, 32, 17, 1]) == [0, 0, 0, 0, 0, 1]     # two pages of the three are left
    assert b.fork([-1, -1, -1, -1, -1, 4], [0, 0, 0, 0, 0, 0]) == [0, 0, 0, 0, 0, 0]     # of no tokens


def test_descending_offsets_and_offsets_outside_are_refused():
    b = Both(50, 16, 5, 4)
    assert b.extend_at([3, 1, 4, 9, 30, -5], 20) == [1, 0, 0, 1, 1]
    assert b.extend_at([-2, 0, 5, 5, 20, 20], 20) == [1, 0, 0, 0, 0]


def test_bad_rows_do_not_reach_the_pool():
    """Ids outside the pool, a page named twice and lengths outside the row."""
    b = Both(20, 16, 5, 4)
    b.extend([40, 40, 16, 0, 0])
    b.ref.rows[0][1] = 999
    b.ref.rows[1][2] = b.ref.rows[1][0]
    b.ref.seq[2], b.ref.seq[3] = 1000, -4
    b.push()
    assert b.extend([0, 0, 1, 1, 0]) == [0, 0, 1, 1, 0]
    assert b.fork([-1, -1, -1, -1, 0], [0, 0, 0, 0, 35]) == [0] * 5
    b.trim([0, 0, 5, 0, 0])


def test_tags_wrap_around():
    b = Both(3, 16, 1, 3)
    b.pool.page_tags.fill_(-1)
    b.ref.tags = [2 ** 32 - 1] * 3
    slots = torch.empty(20, dtype=torch.int64, device=DEV)
    kvq.kvq_extend_tables(b.pool, None, 20, b.seq, b.bt, b.expected, slots, b.refused)
    b.ref.extend([0, 20], 20)
    assert b.pool.page_tags.tolist() == [0, 0, -1] and b.expected.tolist() == [[0, 0, 0]]


def test_a_captured_step_and_another_stream():
    """Extend and trim replayed from a graph walk the same states as eager calls."""
    a, b = Both(400, 16, 9, 40), Both(400, 16, 9, 40)
    lens = [0, 1, 17, 30, 16, 5, 2, 40, 9]
    slots = torch.empty(sum(lens), dtype=torch.int64, device=DEV)
    off = i32([sum(lens[:i]) for i in range(10)])
    keep = i32([-1, 0, 10, -1, 5, 300, -1, 33, 1])

    def step(x):
        kvq.kvq_extend_tables(x.pool, off, slots.numel(), x.seq, x.bt, x.expected, slots, x.refused)
        kvq.kvq_trim_tables(x.pool, keep, x.seq, x.bt)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(b)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for _ in range(3):
        graph.replay()
    for _ in range(4):
        a.ref.extend(off.tolist(), slots.numel())
        a.ref.trim(keep.tolist())
    b.ref = a.ref
    b.check()


def test_a_pool_of_many_pages():
    """The bitmap's scan over several passes."""
    n = 300001
    pool = kvq.PagePool.create(n, 16, device=DEV, tags=False)
    B, maxp = 10, 40000
    seq = torch.zeros(B, dtype=torch.int32, device=DEV)
    bt = torch.full((B, maxp), -1, dtype=torch.int32, device=DEV)
    refused = torch.empty(B, dtype=torch.uint8, device=DEV)
    kvq.kvq_extend_tables(pool, None, B * 480000, seq, bt, None, None, refused)
    assert not refused.any() and pool.free_count.item() == 1
    assert torch.equal(bt[:, :30000].flatten().long(), torch.arange(300000, device=DEV))
    kvq.kvq_trim_tables(pool, torch.zeros_like(seq), seq, bt)
    assert pool.free_count.item() == n
    want = torch.cat([torch.tensor([n - 1], device=DEV), torch.arange(n - 1, device=DEV)])
    assert torch.equal(pool.free_pages.long(), want) and not pool.scratch.any() and not pool.page_refs.any()
