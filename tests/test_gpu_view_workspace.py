"""One workspace under windowed and block-scaled calls of one batch, head count
and n, as layers with a window and layers without one use it in turn, and as
tables that grow do: whichever kernel a call takes, it finds the arrival
counters at zero and leaves them there."""
import numpy as np
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
import view_ref as R
from test_gpu_view import DEV, KINDS, SCALE, Case

pytestmark = pytest.mark.gpu
PS, WIDE = 64, 256
LENS = (5000, 0, 700, 33, 6000, 1, 9000, 2500)
# (window, table entries per request): a window that shows less than 256 MB of
# cache, every token of 16,384-token tables (268 MB), tables as long as the
# longest request, a short window
CALLS = ((8000, WIDE), (0, WIDE), (0, 141), (2000, WIDE))


class Layers(Case):
    """A case whose positions all hold values, with tables of WIDE entries."""

    def __init__(self, kind, n, g):
        super().__init__(kind, LENS, g, PS, n, 0, 0, hkv=8)
        pad = np.full((len(LENS), WIDE - self.bt.shape[1]), -1, np.int32)
        self.bt = np.concatenate([self.bt, pad], axis=1)
        self.tables = {w: torch.from_numpy(np.ascontiguousarray(self.bt[:, :w])).to(DEV) for w in (WIDE, 141)}
        self.refs = {}

    def plan(self, window, width):
        make = kvq.kvq_decode_plan_blocks if self.kind == "blocks" else kvq.kvq_decode_plan_window
        return make(self.desc, len(LENS), self.n, self.q_bits.shape[2], width, window, 0)

    def attend(self, out, ws, window, width):
        self.window = window
        return self.call(out, ws, bt=self.tables[width])

    def compare(self, out, window, what):
        if window not in self.refs:
            self.window = window
            rows = self.n * self.q_bits.shape[2] // self.k.shape[1]
            cut = 2.0 ** -32 if self.kind != "bf16" and rows >= 17 else 2.0 ** -40
            self.refs[window] = R.attention(self.q_bits, self.k, self.v, self.bt, self.lens, SCALE, window, 0,
                                            ks=self.ks, vs=self.vs, ke=self.ke, ve=self.ve, fp32=True, cut=cut)
        torch.cuda.synchronize()
        R.assert_within(out.cpu().numpy().astype(np.float64), *self.refs[window], what)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,g", [(1, 8), (3, 8), (8, 8)])
def test_windows_and_table_widths_in_turn(kind, n, g):
    c = Layers(kind, n, g)
    plans = [c.plan(*call) for call in CALLS]
    assert len(set(plans)) >= 3
    if kind != "bf16" and n * g == 24:                      # equal splits for the window, shared without
        assert plans[0][0] < 8192 and plans[1][0] == 8192 and plans[0][1] > 1
    ws = torch.zeros(max(p[2] for p in plans), dtype=torch.uint8, device=DEV)
    counters = ws[:8 * 8 * (1 if n == 1 else -(-n * g // 16)) * 4]
    for order in ((0, 1, 0, 1), (1, 3, 1, 2, 1), (2, 1, 0)):
        for i in order:
            out = c.attend(c.out(True), ws, *CALLS[i])
            c.compare(out, CALLS[i][0], f"call {i} of {order}")
            assert not counters.any(), (i, order)
    outs, graphs = [], []
    for call in CALLS:
        out, graph = c.out(True), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.attend(out, ws, *call)
        outs.append(out)
        graphs.append(graph)
    for i in (0, 1, 2, 1, 3, 1, 0):
        outs[i].fill_(5.0)
        graphs[i].replay()
        c.compare(outs[i], CALLS[i][0], f"replay {i}")
    assert not counters.any()


def test_a_window_of_layers_in_one_graph():
    """Four layers, every other one behind a window, on one workspace in one
    graph (nothing between the calls but the stream's order)."""
    c = Layers("blocks", 3, 8)
    calls = [CALLS[0], CALLS[1]] * 2
    ws = torch.zeros(max(c.plan(*call)[2] for call in calls), dtype=torch.uint8, device=DEV)
    outs = [c.out(True) for _ in calls]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out, call in zip(outs, calls):
            c.attend(out, ws, *call)
    for _ in range(2):
        for out in outs:
            out.fill_(5.0)
        graph.replay()
        for i, (out, call) in enumerate(zip(outs, calls)):
            c.compare(out, call[0], f"layer {i}")
