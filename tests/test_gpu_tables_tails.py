"""kvq_extend_tables of rows whose partly filled last page other rows hold too, as kvq_trim_tables can leave them
behind a fork: such a row gets nothing, so that no slot lies in a page that another row reads.  Whole states against
the plain model with that rule."""
import random

import pytest

torch = pytest.importorskip("torch")

import fp8_quantised_paged_kv_gb300 as kvq
from tests.tables_ref import Tables
from tests.test_gpu_tables import DEV, Both, i32

pytestmark = pytest.mark.gpu


class Model(Tables):
    """The plain model; a row that may not write its last page is put past its table while the rest is extended."""

    def tail_is_shared(self, r, n):
        old = self.seq[r]
        if not (n > 0 and 0 < old < self.maxp * self.ps and old % self.ps):
            return False
        page = self.rows[r][old // self.ps]
        return 0 <= page < self.n and self.refs[page] > 1

    def extend(self, offsets, total):
        shared = {r: self.seq[r] for r in range(len(self.seq))
                  if self.tail_is_shared(r, offsets[r + 1] - offsets[r])}
        for r in shared:
            self.seq[r] = self.maxp * self.ps
        slots, refused = super().extend(offsets, total)
        assert all(refused[r] for r in shared)
        for r, old in shared.items():
            self.seq[r] = old
        for s in slots:                                     # what the rule is for
            assert s is None or s < 0 or self.refs[s // self.ps] == 1
        return slots, refused


class Tails(Both):
    def __init__(self, num_pages, ps, batch, maxp, tags=True):
        super().__init__(num_pages, ps, batch, maxp, tags)
        self.ref = Model(num_pages, ps, batch, maxp)


@pytest.mark.parametrize("ps", [16, 64, 128])
@pytest.mark.parametrize("more", [1, 40, 3000])             # a thread, a warp and a CTA on a request
def test_a_fork_trimmed_into_shared_pages(ps, more):
    b = Tails(400, ps, 4, 220)
    b.extend([5 * ps + 6, 0, 3, 0])
    b.fork([-1, 0, -1, -1], [0, 4 * ps, 0, 0])              # four whole pages shared
    b.trim([-1, 3 * ps + 2, -1, -1])                        # into the last of them
    assert b.extend([1, more, 1, 0]) == [0, 1, 0, 0]
    assert b.extend([0, 0, 0, 0]) == [0, 0, 0, 0]           # of no tokens: nothing to refuse
    b.trim([-1, 3 * ps, -1, -1])                            # to a page's end
    assert b.extend([0, more, 0, more]) == [0, 0, 0, 0]


@pytest.mark.parametrize("ps", [16, 128])
def test_the_parent_trimmed_behind_the_branch(ps):
    b = Tails(60, ps, 4, 8)
    b.extend([4 * ps, 0, 0, 0])
    b.fork([-1, 0, -1, -1], [0, 4 * ps, 0, 0])
    b.trim([3 * ps + 1, -1, -1, -1])
    assert b.extend([1, 1, 1, 1]) == [1, 0, 0, 0]
    b.trim([-1, 4 * ps - 1, -1, -1])                        # both end in the page
    assert b.extend([1, 1, 1, 1]) == [1, 1, 0, 0]
    # a row of its own: forked onto an empty one, which copies the page, and the old one given back
    b.trim([-1, -1, 0, -1])
    assert b.fork([-1, -1, 0, -1], [0, 0, 3 * ps + 1, 0]) == [0, 0, 0, 0]
    assert b.src[2].item() == b.ref.rows[0][3] and b.dst[2].item() == b.ref.rows[2][3]
    b.trim([0, -1, -1, -1])
    assert b.extend([0, 1, 1, 0]) == [0, 0, 0, 0]           # and the other row is the page's only holder now
    b.trim([0] * 4)
    assert b.ref.count == b.ref.n


def test_a_refused_row_wants_no_pages():
    """The pool's last pages go to the requests after it."""
    b = Tails(8, 16, 4, 8)
    b.extend([48, 0, 0, 0])
    b.fork([-1, 0, -1, -1], [0, 48, 0, 0])
    b.trim([-1, 40, -1, -1])
    assert b.extend([0, 60, 70, 0]) == [0, 1, 0, 0]         # 5 pages are left, and 5 wanted
    assert b.ref.count == 0


def branch_step(rng, model, ps, step):
    """(parents, lengths forked, lengths kept, new tokens) of a step: empty rows forked from others, mostly at a page's
    end, tokens taken back past the branch points, and one or a few tokens each."""
    batch = len(model.seq)
    held = [r for r in range(batch) if model.seq[r] > 0]
    parents = [rng.choice(held) if n == 0 and rng.random() < 0.8 else -1 for n in model.seq]
    lens = [rng.choice([model.seq[p] // ps * ps, model.seq[p]]) if p >= 0 else 0 for p in parents]
    after = [n if p >= 0 else m for p, n, m in zip(parents, lens, model.seq)]
    keep = [rng.choice([-1, -1, -1, max(0, n - rng.randint(1, ps)), max(0, n - rng.randint(1, ps))]) if r and
            rng.random() < 0.9 else -1 if r == 0 else 0 for r, n in enumerate(after)]
    return parents, lens, keep, [1] * batch if step % 2 == 0 else [rng.choice([0, 1, 2, ps]) for _ in range(batch)]


@pytest.mark.parametrize("batch,ps", [(9, 16), (41, 32), (300, 64), (700, 16)])
def test_a_random_run_of_branches(batch, ps):
    rng = random.Random(batch)
    b = Tails(batch * 6, ps, batch, 10)
    b.extend([5 * ps] + [rng.choice([0, 4 * ps, rng.randint(1, 5 * ps)]) for _ in range(batch - 1)])
    met = 0
    for step in range(12):
        parents, lens, keep, new = branch_step(rng, b.ref, ps, step)
        b.fork(parents, lens)
        b.trim(keep)
        met += sum(b.ref.tail_is_shared(r, n) for r, n in enumerate(new))
        b.extend(new, even=step % 2 == 0)
    assert met >= batch // 3
    b.trim([0] * batch)
    assert b.ref.count == b.ref.n


def test_a_captured_step_follows_the_holders():
    """Refused while the page is shared, served once it is not."""
    b = Tails(40, 16, 2, 8)
    b.extend([64, 0])
    b.fork([-1, 0], [0, 64])
    b.trim([-1, 50])
    slots = torch.empty(2, dtype=torch.int64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_extend_tables(b.pool, None, 2, b.seq, b.bt, b.expected, slots, b.refused)
    for keep in ([-1, -1], [0, -1], [-1, -1]):
        b.trim(keep)
        graph.replay()
        want, refused = b.ref.extend([0, 1, 2], 2)
        assert slots.tolist() == want and b.refused.tolist() == refused
        b.check()
    assert refused == [0, 0]
