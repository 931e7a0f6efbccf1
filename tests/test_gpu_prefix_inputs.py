"""Attention over shared prefixes right behind the kernels that write its inputs: every input is rewritten in place
between two calls on one stream, and each call must see what was written last.  (The launch over the requests' own
pages starts beside the one over the shared pages, without a wait of its own for the kernels before the call.)"""
import pytest
import torch

import fp8_quantised_paged_kv_gb300 as kvq
from test_gpu_prefix import KINDS, Case

pytestmark = pytest.mark.gpu
SETS, ROUNDS = 4, 8


def words(x):
    return x.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[x.element_size()])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,graph", [(1, False), (1, True), (4, False), (4, True)])
def test_each_call_sees_the_inputs_written_before_it(kind, n, graph):
    kvq.kvq_device_error(clear=True)
    groups = [(640, [30, 70, 300] * 3), (None, [500, 40]), (200, [19, 29, 400] * 3)]
    cases = [Case(kind, groups, 4, 16, n, seed=i) for i in range(SETS)]
    for i, c in enumerate(cases):                           # lengths and flags differ too
        c.lens -= i
        c.upload()
        c.d["abort"] = (torch.arange(len(c.lens), device="cuda") % 7 == i).to(torch.uint8)
    live = cases[0]
    mine = {k: x.clone() for k, x in live.d.items()}
    ws = live.workspace()

    def write(c):                                           # by kernels that run on the SMs
        for k, x in mine.items():
            torch.bitwise_xor(words(c.d[k]), 0, out=words(x))

    def call(out):
        live.call(out, ws, mine["abort"], **{k: x for k, x in mine.items() if k != "abort"})

    want, got = ([live.out(True) for _ in cases] for _ in range(2))
    for c, out in zip(cases, want):
        write(c)
        torch.cuda.synchronize()
        call(out)
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])

    def all_sets():
        for c, out in zip(cases, got):
            write(c)
            call(out)

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_sets()
    for _ in range(ROUNDS):
        for out in got:
            out.fill_(7.0)
        g.replay() if graph else all_sets()
        torch.cuda.synchronize()
        for i in range(SETS):
            assert torch.equal(got[i], want[i]), i
    assert kvq.kvq_device_error() == 0
