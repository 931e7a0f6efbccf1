"""A serving run whose tables, prefixes and steps never leave the GPU: prompts admitted (kvq_extend_tables, the append),
samples forked from one (kvq_fork_tables, kvq_copy_pages), steps of one token as one CUDA graph (extend, tag check,
append, attention over the shared prefix), finished requests and rejected tokens given back (kvq_trim_tables) and
others forked in their place.  Tables against the plain model, caches and outputs against oracle and view_ref."""
import numpy as np
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
import oracle
import view_ref as R
import workloads as W
from tables_ref import Tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, PS, HKV, G, B, N = 128, 16, 2, 4, 12, 220
SCALE = float(np.float32(1 / np.sqrt(D)))


def t(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def bf(bits):
    return t(bits.view(np.int16)).view(torch.bfloat16)


class Run:
    def __init__(self, kind, wide):
        self.kind, self.rng = kind, np.random.default_rng(wide)
        self.maxp = (512 << 20) // (256 * B * HKV * PS) + 1 if wide else 40
        self.model = Tables(N, PS, B, 40)                   # columns past 40 stay unused
        self.desc = kvq.CacheDesc(N, PS, HKV)
        self.pool = kvq.PagePool.create(N, PS)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.seq = torch.zeros(B, **i32)
        self.bt = torch.full((B, self.maxp), -1, **i32)
        self.expected = torch.zeros((B, self.maxp), **i32)
        self.slots = torch.empty(B, dtype=torch.int64, device=DEV)
        self.refused, self.abort = (torch.empty(B, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.src, self.dst, self.lead, self.shared = (torch.full((B,), -1, **i32) for _ in range(4))
        self.ref = [R.encode(self.rng.standard_normal((N, HKV, PS, D)) * 90) for _ in range(2)]
        self.dev = [t(x) for x in self.ref]
        self.scales = [self.rng.uniform(0.006, 0.02, HKV).astype(np.float32) for _ in range(2)]
        if kind == "blocks":
            self.ref += [self.rng.integers(-9, -5, (N, HKV, PS // 16)).astype(np.int8) for _ in range(2)]
            self.dev += [t(x) for x in self.ref[2:]]
        self.scale = [t(x) for x in self.scales]
        self.ws = kvq.workspace_for_prefix(self.desc, B, 1, HKV * G, self.maxp)
        self.k_new, self.v_new = (torch.empty((B, HKV, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.q = torch.empty((B, 1, HKV * G, D), dtype=torch.bfloat16, device=DEV)
        self.out = torch.empty(self.q.shape, dtype=torch.float32, device=DEV)

    def check_tables(self):
        torch.cuda.synchronize()
        m = self.model
        assert self.seq.tolist() == m.seq and self.bt[:, :40].tolist() == m.rows
        assert self.pool.free_count.item() == m.count and self.pool.free_pages[:m.count].tolist() == m.free[:m.count]
        assert self.pool.page_refs.tolist() == m.refs and self.expected[:, :40].tolist() == m.expected
        for x, y in zip(self.dev, self.ref):
            assert np.array_equal(x.cpu().numpy(), y)

    def append(self, k, v, slots, offsets, abort, dev_slots, dev_offsets, dev_abort, dk, dv):
        if self.kind == "blocks":
            kvq.kvq_append_blocks(self.desc, dk, dv, dev_offsets, self.bt, self.seq, dev_abort, *self.dev)
        else:
            kvq.kvq_append(self.desc, dk, dv, dev_slots, *self.scale, dev_abort, *self.dev)
        if k is not None:
            self.ref_append(k, v, slots, offsets, abort)

    def ref_append(self, k, v, slots, offsets, abort):
        if self.kind == "blocks":
            R.append_blocks(*self.ref, k, v, offsets, np.asarray(self.model.rows), self.model.seq, abort)
        else:
            s = np.asarray(slots, np.int64).copy()
            if abort is not None:
                s[np.asarray(abort) != 0] = -1
            oracle.append(*self.ref, k, v, s, *self.scales, page_size=PS)

    def admit(self, lens):
        offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        T = int(offsets[-1])
        slots = torch.empty(T, dtype=torch.int64, device=DEV)
        off = t(offsets)
        kvq.kvq_extend_tables(self.pool, off, T, self.seq, self.bt, self.expected, slots, self.refused)
        want, refused = self.model.extend(offsets.tolist(), T)
        k, v = (W.normal_bf16(self.rng, (T, HKV, D)) for _ in range(2))
        self.append(k, v, want, offsets, None, slots, off, None, bf(k), bf(v))
        assert slots.tolist() == want and self.refused.tolist() == refused == [0] * B
        self.check_tables()

    def fork(self, parents, lens):
        parents, lens = np.asarray(parents, np.int32), np.asarray(lens, np.int32)
        kvq.kvq_fork_tables(self.pool, t(parents), t(lens), self.seq, self.bt, self.expected, self.src, self.dst,
                            self.refused)
        kvq.kvq_copy_pages(self.desc, self.dev[:2], self.dev[2:], self.src, self.dst)
        src, dst, refused = self.model.fork(parents.tolist(), lens.tolist())
        for a, b in zip(src, dst):
            if b >= 0:
                for x in self.ref:
                    x[b] = x[a]
        forked = parents >= 0
        lead = np.where(forked, parents, self.lead.cpu().numpy())
        lead[parents[forked]] = parents[forked]             # a parent leads the row of its own prefix
        shared = np.where(forked, lens, self.shared.cpu().numpy())
        shared[parents[forked]] = np.asarray(self.model.seq)[parents[forked]]
        self.lead.copy_(t(lead.astype(np.int32)))
        self.shared.copy_(t(shared.astype(np.int32)))
        assert self.refused.tolist() == refused == [0] * B
        self.check_tables()

    def trim(self, keep):
        kvq.kvq_trim_tables(self.pool, t(np.asarray(keep, np.int32)), self.seq, self.bt)
        self.model.trim(keep)
        self.shared[torch.tensor([k == 0 for k in keep], device=DEV)] = 0       # whoever comes next shares nothing yet
        self.check_tables()

    def calls(self):
        """The step, as it is captured."""
        kvq.kvq_extend_tables(self.pool, None, B, self.seq, self.bt, self.expected, self.slots, self.refused)
        kvq.kvq_tag_check(self.bt, self.expected, self.seq, PS, self.pool.page_tags, self.abort)
        self.append(None, None, None, None, None, self.slots, None, self.abort, self.k_new, self.v_new)
        blocks = self.kind == "blocks"
        call = kvq.kvq_decode_attn_prefix_blocks if blocks else kvq.kvq_decode_attn_prefix
        call(self.desc, self.q, *self.dev[:2], *(self.dev[2:] if blocks else self.scale), self.bt, self.seq, self.lead,
             self.shared, SCALE, self.abort, self.out, self.ws)

    def step(self, replay, stale=None):
        k, v = (W.normal_bf16(self.rng, (B, HKV, D)) for _ in range(2))
        q = W.normal_bf16(self.rng, (B, 1, HKV * G, D))
        self.k_new.copy_(bf(k))
        self.v_new.copy_(bf(v))
        self.q.copy_(bf(q))
        m = self.model
        slots, refused = m.extend(list(range(B + 1)), B)
        abort = np.zeros(B, np.uint8)
        if stale is not None:                               # a page of this request changed owner
            page = m.rows[stale][0]
            self.pool.page_tags[page] += 1
            m.tags[page] += 1
            abort[[r for r in range(B) if page in m.rows[r]]] = 1
        replay()
        self.ref_append(k, v, slots, np.arange(B + 1), abort)
        self.check_tables()
        assert self.slots.tolist() == slots and self.refused.tolist() == refused
        assert self.abort.tolist() == abort.tolist()
        exps = dict(zip(("ke", "ve"), self.ref[2:])) if self.kind == "blocks" else dict(zip(("ks", "vs"), self.scales))
        ref, bound = R.attention(q, *self.ref[:2], np.asarray(m.rows), m.seq, SCALE, 0, 0, abort=abort, fp32=True,
                                 cut=2.0 ** -32, **exps)
        R.assert_within(self.out.cpu().numpy().astype(np.float64), ref, bound)
        if stale is not None:
            self.pool.page_tags[page] -= 1
            m.tags[page] -= 1


@pytest.mark.parametrize("kind", ["fp8", "blocks"])
@pytest.mark.parametrize("wide", [False, True])
def test_a_run_with_shared_prefixes(kind, wide):
    kvq.kvq_device_error(clear=True)
    r = Run(kind, wide)
    r.admit([300, 45] + [0] * 10)
    r.fork([-1, -1] + [0] * 9 + [-1], [0, 0, 300, 299, 288, 17, 300, 1, 300, 272, 300, 0])
    r.step(r.calls)                                         # before the capture
    graph = torch.cuda.CUDAGraph()
    state = [x.clone() for x in (r.seq, r.bt, r.expected, r.pool.free_count, r.pool.page_refs, r.pool.page_tags)]
    with torch.cuda.graph(graph):
        r.calls()
    for x, y in zip((r.seq, r.bt, r.expected, r.pool.free_count, r.pool.page_refs, r.pool.page_tags), state):
        assert torch.equal(x, y)                            # a capture runs nothing
    for i in range(6):
        r.step(graph.replay, stale={2: 1, 4: 0}.get(i))
    keep = [-1] * B
    keep[4], keep[6], keep[9] = 0, 0, r.model.seq[9] - 5    # two finished, five tokens of one rejected
    r.trim(keep)
    r.step(graph.replay)
    r.trim([-1] * 4 + [0, -1, 0] + [-1] * 5)
    r.fork([-1] * 4 + [0, -1, 0] + [-1] * 5, [0] * 4 + [296, 0, r.model.seq[0], 0, 0, 0, 0, 0])
    for _ in range(3):
        r.step(graph.replay)
    r.trim([0] * B)
    assert r.model.count == N and kvq.kvq_device_error() == 0
