"""Grouped-head attention as a program calls it: captured and replayed, on several streams, with many sequences, with more
query rows than a unit holds, in caches past 2^32 bytes, with waits that run out.  Values are compared with plain 64-bit
computations as in test_gpu_gqa.py, or with the bits of the same call made alone."""
import ctypes

import pytest

from test_gpu_gqa import filled, gen, packed_qkv, reference_prompt, reference_step, run_step, setup, stays

pytestmark = pytest.mark.gpu


def i32(torch, x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Steps:
    """A step whose segments are split, so that its partial results go through scratch, and an eviction of what it weighed."""

    def __init__(self, torch, coli, seed, lens, weigh=True):
        g = gen(torch, seed)
        self.coli, self.weigh = coli, weigh
        self.s, table, spare = filled(torch, coli, lens, 2, 64, 128, 32, g, spare=len(lens) * 2)
        self.table, self.lens, self.dst = table.cuda(), i32(torch, lens), spare.view(len(lens), 2).contiguous().cuda()
        self.q = torch.randn(len(lens), 1, 16, 128, generator=g).to(torch.bfloat16).cuda()
        self.out = torch.zeros(len(lens), 1, 16, 128, device="cuda")
        self.kept, self.new = torch.zeros(len(lens), 2, 100, dtype=torch.int32, device="cuda"), torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        self.w0 = self.s.w.clone()

    def __call__(self):
        self.coli.gqa_attend(self.s.c, self.q, self.table, self.lens, 0.06, self.out, weigh=self.weigh)
        if self.weigh:
            self.coli.gqa_evict(self.s.c, self.table, self.lens, 100, 10, self.dst, self.kept, self.new)

    def clear(self):
        self.s.w.copy_(self.w0)
        self.out.zero_()
        self.kept.zero_()

    def result(self):
        return [t.clone() for t in (self.out, self.s.w, self.kept, self.new)]


class Prompt:
    def __init__(self, torch, coli, seed, n, f32):
        g = gen(torch, seed)
        q, kv = packed_qkv(torch, [n], [n], 8, 2, 128, g, torch.float32 if f32 else torch.bfloat16)
        self.coli, self.q, self.kv, self.cu = coli, q.cuda(), kv.cuda(), i32(torch, [0, n])
        self.out = torch.zeros(n, 8, 128, device="cuda")

    def __call__(self):
        self.coli.gqa_prefill(self.q, self.kv[:, :2], self.kv[:, 2:4], self.cu, self.cu, 0.09, self.out)

    def clear(self):
        self.out.zero_()

    def result(self):
        return [self.out.clone()]


def same(torch, a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def captured(torch, st, *calls):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        for c in calls:
            c()
    return graph


def test_graphs_of_one_stream_side_by_side():
    """Captured on one stream, replayed on two at once, eager calls on a third: each has scratch of its own."""
    torch, coli = setup()
    work = [Steps(torch, coli, 1, [3000, 70, 900]), Prompt(torch, coli, 2, 700, True), Steps(torch, coli, 3, [2500, 400], weigh=False)]
    want = []
    for w in work:
        w.clear()
        w()
        want.append(w.result())
        w.clear()
    coli.sync_check()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = [captured(torch, st, w) for w in work[:2]]
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for w in work:
            w.clear()
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        with torch.cuda.stream(st):
            work[2]()
        torch.cuda.synchronize()
        assert all(same(torch, w.result(), x) for w, x in zip(work, want))
    coli.sync_check()


def test_replay_after_larger_calls():
    """Larger calls on the captured stream outgrow its scratch; what they freed belongs to others by the time of the replay."""
    torch, coli = setup()
    st = torch.cuda.Stream()
    small, large = Prompt(torch, coli, 4, 300, True), Prompt(torch, coli, 5, 3000, True)
    steps = Steps(torch, coli, 6, [3000, 100])
    torch.cuda.synchronize()
    want = []
    with torch.cuda.stream(st):
        for w in (small, steps):
            w.clear()
            w()
            want.append(w.result())
            w.clear()
    torch.cuda.synchronize()
    graph = captured(torch, st, small, steps)
    with torch.cuda.stream(st):
        large()
    torch.cuda.synchronize()
    others = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(32)]
    graph.replay()
    torch.cuda.synchronize()
    coli.sync_check(st)
    assert same(torch, small.result(), want[0]) and same(torch, steps.result(), want[1])
    assert all(bool((o == 3).all()) for o in others)


def test_streams_of_their_own():
    """Two streams at once, given by the argument rather than as the current one."""
    torch, coli = setup()
    a, b = Steps(torch, coli, 7, [3000, 70]), Steps(torch, coli, 8, [2000, 1500])
    want = []
    for w in (a, b):
        w.clear()
        w()
        want.append(w.result())
        w.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for w, s in zip((a, b), streams):
        coli.gqa_attend(w.s.c, w.q, w.table, w.lens, 0.06, w.out, weigh=True, stream=s)
        coli.gqa_evict(w.s.c, w.table, w.lens, 100, 10, w.dst, w.kept, w.new, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert same(torch, a.result(), want[0]) and same(torch, b.result(), want[1])


@pytest.mark.parametrize("n", [257, 700])
def test_many_sequences(n):
    """More sequences than a CTA has threads, most of them short or empty."""
    torch, coli = setup()
    g = gen(torch, n)
    lens = [int(x) for x in torch.randint(0, 3, (n,), generator=g) * torch.randint(0, 60, (n,), generator=g)]
    s, table, _ = filled(torch, coli, lens, 1, 16, 64, 32, g)
    q = torch.randn(n, 1, 4, 64, generator=g).to(torch.bfloat16)
    before = s.w.cpu().double()
    out, _ = run_step(torch, coli, s, table, lens, q, 0.1, "f32", weigh=True)
    ref, tol, _, weights, w_tol = reference_step(torch, s, table, lens, q, 0.1, "bf16", "f32")
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    got = s.w.cpu().double()
    for b, m in enumerate(lens):
        for i in range(-(-m // 16)):
            k = min(16, m - 16 * i)
            p = int(table[b, i])
            assert ((got[p, 0, :k] - before[p, 0, :k] - weights[b][0, 16 * i:16 * i + k]).abs() <= w_tol[b][0, 16 * i:16 * i + k] + 2.0 ** -23).all()


@pytest.mark.parametrize("n_q,H,K,lens", [(40, 8, 1, [300, 30]), (33, 6, 6, [50]), (7, 40, 2, [7, 6, 200])])
def test_many_query_rows(n_q, H, K, lens):
    """More rows of a head than one unit has; a window of queries longer than the sequence."""
    torch, coli = setup()
    g = gen(torch, n_q)
    s, table, _ = filled(torch, coli, lens, K, 32, 64, 32, g)
    before = s.w.cpu().double()
    q = torch.randn(len(lens), n_q, H, 64, generator=g).to(torch.bfloat16)
    out, lse = run_step(torch, coli, s, table, lens, q, 0.1, "f32", weigh=True)
    ref, tol, ref_lse, weights, w_tol = reference_step(torch, s, table, lens, q, 0.1, "bf16", "f32")
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(ref_lse))
    for b, m in enumerate(lens):
        for i in range(-(-m // 32)):
            k = min(32, m - 32 * i)
            p = int(table[b, i])
            got = s.w.cpu().double()[p, :, :k] - before[p, :, :k]
            # f32 additions of sets of 8 rows to a weight of up to n_q times the group
            slack = w_tol[b][:, 32 * i:32 * i + k] + 2.0 ** -23 * (2 + n_q * H // K / 8) * (1 + weights[b][:, 32 * i:32 * i + k])
            assert ((got - weights[b][:, 32 * i:32 * i + k]).abs() <= slack).all()


def test_wide_page_tables():
    """Tables far wider than in use plan for lengths that they could hold; the result is that of the narrow ones."""
    torch, coli = setup()
    g = gen(torch, 51)
    lens = [500, 40]
    s, table, _ = filled(torch, coli, lens, 2, 16, 128, 64, g)
    q = torch.randn(2, 1, 8, 128, generator=g).to(torch.bfloat16)
    want, _ = run_step(torch, coli, s, table, lens, q, 0.1, "f32")
    wide = torch.full((2, 200000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    got, _ = run_step(torch, coli, s, wide, lens, q, 0.1, "f32")
    ref, tol, *_ = reference_step(torch, s, table, lens, q, 0.1, "bf16", "f32")
    assert ((got.cpu().double() - ref).abs() <= tol).all() and ((want.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("seqs,K,H,n_q,D,gs", [(1, 8, 32, 1, 128, 32), (2, 8, 24, 2, 64, 64), (9, 4, 28, 1, 128, 64), (8, 8, 16, 2, 128, 128), (20, 5, 5, 1, 64, 32),
                                               (38, 8, 16, 1, 128, 32), (39, 8, 16, 1, 64, 32)])
def test_clusters_and_shares(seqs, K, H, n_q, D, gs):
    """Segments shared by clusters of 8, 4, 2 CTAs and by none, and the same dealt out as a wide table has them, against 64 bits: outputs,
    lse, weights."""
    torch, coli = setup()
    g = gen(torch, seqs + D)
    lens = [int(x) for x in torch.randint(0, 230, (seqs,), generator=g)]
    lens[0] = 231
    s, table, _ = filled(torch, coli, lens, K, 16, D, gs, g)
    q = torch.randn(seqs, n_q, H, D, generator=g).to(torch.bfloat16)
    ref, tol, ref_lse, weights, w_tol = reference_step(torch, s, table, lens, q, 0.1, "bf16", "f32")
    wide = torch.full((seqs, 5000), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    none = torch.isinf(ref_lse)
    for t in (table, wide):
        before = s.w.cpu().double()
        out, lse = run_step(torch, coli, s, t, lens, q, 0.1, "f32", weigh=True)
        assert ((out.cpu().double() - ref).abs() <= tol).all()
        got = lse.cpu().double()
        assert torch.equal(torch.isinf(got), none) and ((got - ref_lse)[~none].abs() <= 1e-4 * (1 + ref_lse[~none].abs())).all()
        after = s.w.cpu().double()
        for b, m in enumerate(lens):
            for i in range(-(-m // 16)):
                k, p = min(16, m - 16 * i), int(table[b, i])
                off = (after[p, :, :k] - before[p, :, :k] - weights[b][:, 16 * i:16 * i + k]).abs()
                # f32 additions to what the first call has left
                assert (off <= w_tol[b][:, 16 * i:16 * i + k] + 2.0 ** -23 * (1 + before[p, :, :k].abs() + weights[b][:, 16 * i:16 * i + k])).all()


def test_far_pages():
    """Codes past 2^32 bytes, rows past 2^26: writes, reads, steps with weights and an eviction at both ends of the cache."""
    torch, coli = setup()
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    n_pages, kv, page, dim = 140000, 8, 64, 128                          # 71.7 M rows of 64 bytes
    k, v = (torch.zeros(n_pages, kv, page, dim // 2, dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.zeros(n_pages, kv, page, 4, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    w = torch.zeros(n_pages, kv, page, device="cuda")
    c = coli.GqaCache(k, v, ks, vs, weights=w)
    g = gen(torch, 61)
    n = 150
    table = torch.tensor([[n_pages - 1, 3, n_pages - 7]], dtype=torch.int32)
    new = torch.randn(n, 2 * kv, dim, generator=g)
    t = torch.arange(n)
    slots = table[0].long()[t // page] * page + t % page
    coli.gqa_append(c, new[:, :kv].contiguous().cuda(), new[:, kv:].contiguous().cuda(), slots.cuda())
    rk, rv = (torch.empty(n, kv, dim, device="cuda") for _ in "kv")
    coli.gqa_read(c, table.cuda(), i32(torch, [0, n]), rk, rv)
    step = new.unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True) / 7
    off = (torch.cat([rk, rv], 1).cpu() - new).unflatten(-1, (4, 32)).abs()
    assert (off <= step * (0.5 + 7.5 * 2.0 ** -8)).all()                 # half a step, and the scale's own rounding seven times
    q = torch.randn(1, 1, 16, dim, generator=g).to(torch.bfloat16)
    out = torch.empty(1, 1, 16, dim, device="cuda")
    coli.gqa_attend(c, q.cuda(), table.cuda(), i32(torch, [n]), 0.09, out, weigh=True)
    coli.sync_check()
    kd, vd = rk.cpu().double(), rv.cpu().double()
    p = torch.softmax(torch.einsum("hgd,thd->hgt", q[0, 0].double().view(kv, 2, dim), kd) * 0.09, -1)
    ref = torch.einsum("hgt,thd->hgd", p, vd).view(16, dim)
    size = torch.einsum("hgt,thd->hgd", p, vd.abs()).view(16, dim)
    # two roundings of the probabilities to bf16; f32 sums of up to 136 times the largest scale (1) in 20 additions
    assert ((out[0, 0].cpu().double() - ref).abs() <= (2.0 ** -7 + 1e-3) * size + 20 * 136 * 2.0 ** -23).all()
    got = w[table[0].long().cuda()].transpose(0, 1).flatten(1, 2)[:, :n].cpu()
    assert ((got.double() - p.sum(1)).abs() <= 1e-5).all()
    dst = torch.tensor([[n_pages - 2]], dtype=torch.int32)
    kept, length = torch.zeros(1, kv, 60, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    coli.gqa_evict(c, table.cuda(), i32(torch, [n]), 60, 5, dst.cuda(), kept, length)
    ek, ev = (torch.empty(60, kv, dim, device="cuda") for _ in "kv")
    coli.gqa_read(c, dst.cuda(), i32(torch, [0, 60]), ek, ev)
    coli.sync_check()
    for h in range(kv):
        ref = stays(got[h].tolist(), n, 60, 5)
        assert kept[0, h].tolist() == ref
        assert torch.equal(ek[:, h], rk[ref, h]) and torch.equal(ev[:, h], rv[ref, h])
        assert torch.equal(w[n_pages - 2, h, :60].cpu(), got[h, ref])
    assert int((w != 0).sum()) == kv * (n + 60)                           # nothing else was weighed


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_many_units(dtype):
    """Several units per SM and sequences of all sizes in one call; equal calls, equal bits."""
    torch, coli = setup()
    g = gen(torch, 71)
    lens = [int(x) for x in torch.randint(0, 90, (60,), generator=g)] + [700, 1]
    more = [int(x) for x in torch.randint(0, 200, (62,), generator=g)]
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    total = [a + b for a, b in zip(lens, more)]
    q, kv = packed_qkv(torch, lens, total, 12, 4, 64, g, kind)
    cu_q, cu_k = ([0] + list(torch.tensor(x).cumsum(0).tolist()) for x in (lens, total))
    dev = kv.cuda()
    outs = []
    for _ in range(2):
        out = torch.empty(cu_q[-1], 12, 64, device="cuda")
        coli.gqa_prefill(q.cuda(), dev[:, :4], dev[:, 4:8], i32(torch, cu_q), i32(torch, cu_k), 0.12, out)
        coli.sync_check()
        outs.append(out)
    assert torch.equal(*outs)
    ref, tol, _ = reference_prompt(torch, q, kv[:, :4], kv[:, 4:8], cu_q, cu_k, 0.12, "f32")
    assert ((outs[0].cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("n", [(1 << 30) + 1, (1 << 31) - 32, (1 << 31) - 1])
def test_lengths_past_what_a_sequence_may_have(n):
    """Page tables that repeat a page can hold more than 2^30 tokens; such a length is recorded, as others out of range are, and the
    sequence beside it is served."""
    torch, coli = setup()
    page = 65536
    k, v = (torch.randint(0, 256, (2, 1, page, 32), dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.full((2, 1, page, 1), 0.1, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    w = torch.rand(2, 1, page, device="cuda")
    c = coli.GqaCache(k, v, ks, vs, w)
    table = torch.zeros(2, 32768, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 1, 2, 64, device="cuda")

    def call(lens):
        out, kept, new = torch.zeros(2, 1, 2, 64, device="cuda"), i32(torch, [[[9] * 40]] * 2), i32(torch, [9, 9])
        coli.gqa_attend(c, q, table, i32(torch, lens), 0.1, out)
        coli.gqa_evict(c, table, i32(torch, lens), 40, 8, i32(torch, [[1], [1]]), kept, new)
        return out, kept, new

    good = call([0, 300])
    coli.sync_check()
    out, kept, new = call([n, 300])
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_EINVAL
    assert torch.equal(out[1], good[0][1]) and torch.equal(kept, good[1]) and new.tolist() == [0, 40]


# ------------------------------------------------------------------ waits
@pytest.fixture
def limit():
    torch, coli = setup()
    coli.sync_check()
    yield coli.set_wait_limit
    torch.cuda.synchronize()
    coli.set_wait_limit(0)


def test_step_wait_runs_out(limit):
    """With a limit of a nanosecond an ordinary wait of some microseconds is too long: the keys' scales lie in pinned host memory,
    which bulk copies read over the CPU-GPU link.  The call ends with COLI_ETIMEOUT and the next one is as before."""
    torch, coli = setup()
    n, kv, page, seqs = 4096, 8, 64, 16
    per = n // page
    k, v = (torch.randint(0, 256, (seqs * per, kv, page, 64), dtype=torch.uint8, device="cuda") for _ in "kv")
    vs = torch.full((seqs * per, kv, page, 4), 0.1, dtype=torch.bfloat16, device="cuda")
    ks = vs.cpu().pin_memory()
    c = coli._GqaCache(kv, 128, 32, page, seqs * per, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), None)
    table, lens = torch.arange(seqs * per, dtype=torch.int32, device="cuda").view(seqs, per), i32(torch, [n] * seqs)
    q = torch.randn(seqs, 1, 64, 128, device="cuda")

    def call():                                          # through the C entry: the binding wants CUDA tensors
        out = torch.zeros(seqs, 1, 64, 128, device="cuda")
        rc = coli._lib.coli_gqa_attend(ctypes.byref(c), coli.COLI_F32, q.data_ptr(), seqs, 1, 64, table.data_ptr(), per, lens.data_ptr(), 0.09,
                                       0, coli.COLI_F32, out.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        return out

    good = call()
    coli.sync_check()
    limit(1)
    call()
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_ETIMEOUT
    limit(0)
    assert torch.equal(call(), good)
    coli.sync_check()


def test_cluster_step_wait_runs_out(limit):
    """As above where two CTAs share a sequence's head, with the values' scales there, too."""
    torch, coli = setup()
    n, kv, page, seqs = 2048, 8, 64, 16
    per = n // page
    k, v = (torch.randint(0, 256, (seqs * per, kv, page, 64), dtype=torch.uint8, device="cuda") for _ in "kv")
    ks, vs = (torch.full((seqs * per, kv, page, 4), 0.1, dtype=torch.bfloat16).pin_memory() for _ in "kv")
    c = coli._GqaCache(kv, 128, 32, page, seqs * per, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), None)
    table, lens = torch.arange(seqs * per, dtype=torch.int32, device="cuda").view(seqs, per), i32(torch, [n] * seqs)
    q = torch.randn(seqs, 1, 64, 128, device="cuda")

    def call():
        out = torch.zeros(seqs, 1, 64, 128, device="cuda")
        rc = coli._lib.coli_gqa_attend(ctypes.byref(c), coli.COLI_F32, q.data_ptr(), seqs, 1, 64, table.data_ptr(), per, lens.data_ptr(), 0.09,
                                       0, coli.COLI_F32, out.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        return out

    good = call()
    coli.sync_check()
    limit(1)
    for _ in range(30):                                  # in any of them
        call()
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_ETIMEOUT
    limit(0)
    assert torch.equal(call(), good)
    coli.sync_check()


def test_weighed_step_of_several_sets_wait_runs_out(limit):
    """As above for the pass that adds the weights, which goes over a head's keys once for each 8 of its 16 query rows."""
    torch, coli = setup()
    n, kv, page, seqs = 4096, 8, 64, 16
    per = n // page
    k, v = (torch.randint(0, 256, (seqs * per, kv, page, 64), dtype=torch.uint8, device="cuda") for _ in "kv")
    vs = torch.full((seqs * per, kv, page, 4), 0.1, dtype=torch.bfloat16, device="cuda")
    ks = vs.cpu().pin_memory()
    w = torch.zeros(seqs * per, kv, page, device="cuda")
    c = coli._GqaCache(kv, 128, 32, page, seqs * per, k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), w.data_ptr())
    table, lens = torch.arange(seqs * per, dtype=torch.int32, device="cuda").view(seqs, per), i32(torch, [n] * seqs)
    q = torch.randn(seqs, 2, 64, 128, device="cuda")

    def call():
        out = torch.zeros(seqs, 2, 64, 128, device="cuda")
        w.zero_()
        rc = coli._lib.coli_gqa_attend(ctypes.byref(c), coli.COLI_F32, q.data_ptr(), seqs, 2, 64, table.data_ptr(), per, lens.data_ptr(), 0.09,
                                       1, coli.COLI_F32, out.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        return out

    good = call()
    coli.sync_check()
    assert abs(float(w.double().sum()) - seqs * 2 * 64) < 1e-3 * seqs * 2 * 64
    limit(1)
    for _ in range(30):                                  # in any of them
        call()
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_ETIMEOUT
    limit(0)
    assert torch.equal(call(), good)
    assert abs(float(w.double().sum()) - seqs * 2 * 64) < 1e-3 * seqs * 2 * 64
    coli.sync_check()


def test_prompt_wait_runs_out(limit):
    """Finding the first unit among 20000 sequences takes long enough."""
    torch, coli = setup()
    g = gen(torch, 2)
    n, B = 100, 20000
    cu = torch.cat([torch.zeros(B - n, dtype=torch.int32), torch.arange(n + 1, dtype=torch.int32)]).cuda()
    q, kv = packed_qkv(torch, [n], [n], 2, 1, 128, g, torch.bfloat16)
    q, kv = q.cuda(), kv.cuda()

    def call():
        out = torch.zeros(n, 2, 128, device="cuda")
        coli.gqa_prefill(q, kv[:, :1], kv[:, 1:2], cu, cu, 0.09, out)
        return out

    good = call()
    coli.sync_check()
    limit(1)
    call()
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_ETIMEOUT
    limit(0)
    assert torch.equal(call(), good)
    coli.sync_check()


def test_calls_longer_than_the_limit(limit):
    """The limit is one wait's: a call may take many times as long (512 sequences on the same pages; 24000 tokens of a prompt)."""
    torch, coli = setup()
    g = gen(torch, 3)
    s, table, _ = filled(torch, coli, [12000], 2, 64, 128, 32, g)
    B = 512
    table, n = table.cuda().expand(B, -1).contiguous(), i32(torch, [12000] * B)
    q = torch.randn(B, 1, 16, 128, device="cuda").to(torch.bfloat16)
    p, kv, cu = torch.randn(24000, 16, 128, device="cuda").to(torch.bfloat16), torch.randn(24000, 2, 128, device="cuda").to(torch.bfloat16), i32(torch, [0, 24000])
    outs = []
    for ns in (0, 500000):
        out, out_p = torch.zeros_like(q), torch.zeros_like(p)
        limit(ns)
        coli.gqa_attend(s.c, q, table, n, 0.06, out)
        coli.gqa_prefill(p, kv, kv, cu, cu, 0.09, out_p)
        coli.sync_check()
        outs.append((out, out_p))
    assert same(torch, *outs)
