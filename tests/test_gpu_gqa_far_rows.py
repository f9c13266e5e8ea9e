"""A cache of as many rows as coli.h allows: a sequence on its last pages, where a row and a token add up to more than 2^31, has the bits
of the same sequence in a small one."""
import pytest

from test_gpu_gqa import gen, setup

pytestmark = pytest.mark.gpu

PAGE, DIM, N = 64, 64, 250


def test_last_rows():
    torch, coli = setup()
    n_pages = ((1 << 31) - 1) // PAGE
    rows = n_pages * PAGE
    if torch.cuda.mem_get_info()[0] < rows * (DIM + 4 + 4) + (8 << 30):
        pytest.skip("needs 163 GB")
    g = gen(torch, 71)
    new = torch.randn(N, 2, DIM, generator=g).cuda()
    q = torch.randn(1, 1, 4, DIM, generator=g).cuda()
    t, lens = torch.arange(N, device="cuda"), torch.tensor([N], dtype=torch.int32, device="cuda")

    def run(n_pages, table, dst):
        make = lambda last, kind: torch.empty(n_pages, 1, PAGE, last, device="cuda", dtype=kind)  # noqa: E731
        c = coli.GqaCache(make(DIM // 2, torch.uint8), make(DIM // 2, torch.uint8), make(1, torch.bfloat16), make(1, torch.bfloat16),
                          torch.empty(n_pages, 1, PAGE, device="cuda"))
        table, dst = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (table, dst))
        coli.gqa_append(c, new[:, :1], new[:, 1:], table[0].long()[t // PAGE] * PAGE + t % PAGE)
        out, kept, short = torch.empty_like(q), torch.zeros(1, 1, 70, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        coli.gqa_attend(c, q, table, lens, 0.2, out, weigh=True)
        wide = torch.full((1, 4000), -1, dtype=torch.int32, device="cuda")      # lengths that take the other kernels
        wide[:, :table.shape[1]] = table
        out2 = coli.gqa_attend(c, q, wide, lens, 0.2, torch.empty_like(q))
        coli.gqa_evict(c, table, lens, 70, 5, dst, kept, short)
        read = []
        for pages, n in ((table, N), (dst, 70)):
            k, v = torch.empty(n, 1, DIM, device="cuda"), torch.empty(n, 1, DIM, device="cuda")
            coli.gqa_read(c, pages, torch.tensor([0, n], dtype=torch.int32, device="cuda"), k, v)
            read += [k, v]
        coli.sync_check()
        weights = c.weights[table[0].long()].flatten()[:N].clone()
        return [out, out2, kept, short, weights, *read]

    want = run(6, [5, 0, 4, 2], [1, 3])
    try:
        got = run(n_pages, [n_pages - 1, 1, n_pages - 2, n_pages - 3], [0, n_pages - 4])
    finally:
        torch.cuda.empty_cache()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert abs(float(got[4].double().sum()) - 4) < 1e-4
