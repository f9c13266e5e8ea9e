"""CUDA graphs and the library's scratch: a captured call keeps working whatever is called between capture and replay, its
scratch is no other graph's, and it goes when the graph goes."""
import gc

import pytest

import workloads as wl
from gpu_util import upload
from test_gpu_mla import filled, gen, setup

pytestmark = pytest.mark.gpu


class Attend:
    """One attention over the cache: sequences long enough to be split, so that its partial results go through scratch."""

    def __init__(self, torch, coli, seed, lens, H, columns=0, e4m3=False):
        g = gen(torch, seed)
        self.coli = coli
        self.cache, table = filled(torch, coli, e4m3, 256, 32, 64, lens, g, columns=columns)
        self.table, self.lens = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.ql = torch.randn(len(lens), 1, H, 256, generator=g).to(torch.bfloat16).cuda()
        self.qr = torch.randn(len(lens), 1, H, 32, generator=g).to(torch.bfloat16).cuda()
        self.out = torch.zeros(len(lens), 1, H, 256, device="cuda")

    def __call__(self):
        self.coli.mla_attend(self.cache, self.ql, self.qr, self.table, self.lens, 0.06, self.out)
        return self.out


def captured(torch, st, *calls):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        for c in calls:
            c()
    return graph


def test_replay_after_larger_calls():
    """Larger calls on the captured stream outgrow its scratch; what they freed belongs to others by the time of the replay."""
    torch, coli = setup()
    st = torch.cuda.Stream()
    small, large = Attend(torch, coli, 1, [2000, 300], 16), Attend(torch, coli, 2, [9000, 5000, 40], 128)
    q, kv = torch.randn(3000, 16, 192, device="cuda"), torch.randn(3000, 16, 256, device="cuda")
    kr, cu = torch.randn(3000, 64, device="cuda"), torch.tensor([0, 3000], dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        want = small().clone()
    graph = captured(torch, st, small)
    with torch.cuda.stream(st):
        want_large = large().clone()
        coli.mla_prefill(q, kv, kr, cu, cu, 0.07, torch.empty(3000, 16, 128, device="cuda"))
    torch.cuda.synchronize()
    others = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(32)]
    small.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    coli.sync_check(st)
    assert torch.equal(small.out, want)
    assert all(bool((o == 3).all()) for o in others)
    with torch.cuda.stream(st):
        assert torch.equal(large(), want_large)
    torch.cuda.synchronize()


def test_first_call_under_capture():
    """A stream's first call, with no scratch yet, and a larger one after it, within one capture."""
    torch, coli = setup()
    small, large = Attend(torch, coli, 3, [2000, 300], 16, e4m3=True), Attend(torch, coli, 4, [9000, 5000, 40], 128, e4m3=True)
    want = small().clone(), large().clone()
    torch.cuda.synchronize()
    graph = captured(torch, torch.cuda.Stream(), small, large, small)
    for _ in range(2):
        small.out.zero_()
        large.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(small.out, want[0]) and torch.equal(large.out, want[1])
    coli.sync_check()


def test_two_graphs_of_one_stream_side_by_side():
    """Captured on one stream, replayed on two at once, with eager calls on a third: each has scratch of its own."""
    torch, coli = setup()
    a, b, c = (Attend(torch, coli, 5 + i, [3000, 2000, 500], 64) for i in range(3))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        want = [x().clone() for x in (a, b, c)]
    ga, gb = captured(torch, st, *[a] * 8), captured(torch, st, *[b] * 8)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for x in (a, b, c):
            x.out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
        with torch.cuda.stream(st):
            for _ in range(8):
                c()
        torch.cuda.synchronize()
        assert all(torch.equal(x.out, w) for x, w in zip((a, b, c), want))
    coli.sync_check()


def test_scratch_goes_with_the_graph():
    torch, coli = setup()
    st = torch.cuda.Stream()
    a = Attend(torch, coli, 8, [9000, 5000, 40], 128)          # some 20 MB of partial results
    torch.cuda.synchronize()
    free = []
    for _ in range(40):
        graph = captured(torch, st, a)
        graph.replay()
        torch.cuda.synchronize()
        del graph
        gc.collect()
        free.append(torch.cuda.mem_get_info()[0])
    assert free[3] - free[-1] < 64 << 20


def test_products_and_expert_block_after_larger_calls():
    """The products' planes, the router's logits, the decode block's counters and the prefill block's buffers likewise."""
    torch, coli = setup()
    g = wl.rng(9)
    H, F, E, K = 512, 256, 8, 4
    W = upload(coli, wl.random_matrix(g, 4, 640, H, 64))
    router = upload(coli, wl.random_matrix(g, 2, E, H, 0))
    table = coli.ExpertTable([tuple(upload(coli, m) for m in wl.expert(g, H, F, 4, 64)) for _ in range(E)])
    x = {S: torch.randn(S, H, device="cuda") for S in (1, 20, 400)}
    st = torch.cuda.Stream()

    def block(S):
        y, z = torch.empty(S, 640, device="cuda"), torch.empty(S, H, device="cuda")
        ids, w = torch.empty(S, K, dtype=torch.int32, device="cuda"), torch.empty(S, K, device="cuda")

        def run():
            coli.matmul(W, x[S], y)
            coli.moe_router(x[S], router, K, ids, w, norm_topk=True)
            coli.moe_block(x[S], table, ids, w, z)
        return run, (y, z, ids, w)
    runs = {S: block(S) for S in (1, 20, 400)}
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for S in (1, 20):
            runs[S][0]()
    torch.cuda.synchronize()
    want = {S: [t.clone() for t in runs[S][1]] for S in (1, 20)}
    graphs = [captured(torch, st, runs[S][0]) for S in (1, 20)]
    with torch.cuda.stream(st):
        runs[400][0]()
    torch.cuda.synchronize()
    others = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(16)]
    for _ in range(3):
        for S in (1, 20):
            for t in runs[S][1]:
                t.zero_()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for S in (1, 20):
            for t, v in zip(runs[S][1], want[S]):
                assert torch.equal(t, v)
    assert all(bool((o == 3).all()) for o in others)
    coli.sync_check(st)
