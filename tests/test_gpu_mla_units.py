"""The expanded attention's search for units of work by number: a CTA is handed numbers by the hardware, which promises no
order, and has to find each of them from wherever its last search ended.  A small kernel around the library's search
(csrc/mla_units.cuh) is compiled here and asked in several orders; the units come from a list made in Python."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

from gpu_util import cuda_or_skip

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "mla_units.cuh"
using namespace coli;
__global__ void find(const MlaPrefillArgs a, const int *order, int n, Unit *out, int *total) {
    int most;
    const int lane = threadIdx.x, pairs = all_pairs(a, lane, false, most);
    Place at = no_place(most);
    if (lane == 0) *total = pairs * a.H;
    for (int k = 0; k < n; k++) {
        const int i = order[k];
        Unit u;
        u.n = -2;
        if (i < pairs * a.H) u = unit_of(a, i, pairs, at, lane);
        if (lane == 0) out[k] = u;
        __syncwarp();
    }
}
extern "C" int run(const int *cu_q, const int *cu_k, int n_seq, int Tq, int Tk, int H, const int *order, int n, void *out, int *total) {
    MlaPrefillArgs a{};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.n_seq = n_seq;
    a.Tq = Tq;
    a.Tk = Tk;
    a.H = H;
    find<<<1, 32>>>(a, order, n, (Unit *)out, total);
    return (int)cudaDeviceSynchronize();
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cuda_or_skip()
    import __graft_entry__
    build = __graft_entry__._load_build_module()
    at = tmp_path_factory.mktemp("units")
    (at / "units.cu").write_text(SOURCE)
    subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-shared", "-o", str(at / "units.so"), str(at / "units.cu")], check=True)
    return ctypes.CDLL(str(at / "units.so"))


def expected(n_qs, n_ks, H):
    """The units in order: most key tiles first, then by sequence, later pairs first, heads of a pair side by side."""
    cq, ck = np.cumsum([0] + n_qs), np.cumsum([0] + n_ks)
    pairs = []
    for b, (n, m) in enumerate(zip(n_qs, n_ks)):
        for k in range(-(-n // 256)):
            nt = []
            for x in range(2):
                rows = min(128, n - 256 * k - 128 * x)
                limit = 256 * k + 128 * x + rows + m - n if rows > 0 else 0
                nt.append(-(-min(limit, m) // 128) if limit > 0 else 0)
            pairs.append((-max(nt), b, -k, [256 * k, n, m, int(cq[b]), int(ck[b]), nt[0], nt[1], max(nt)]))
    return [[h] + p[3] for p in sorted(pairs, key=lambda p: p[:3]) for h in range(H)]


@pytest.mark.parametrize("seed,n_seq,H", [(1, 1, 3), (2, 7, 1), (3, 70, 2), (4, 200, 1)])
def test_units_in_any_order(lib, seed, n_seq, H):
    import torch
    r = random.Random(seed)
    n_qs = [r.choice((0, 1, 100, 128, 129, 256, 257, 700, 2000)) for _ in range(n_seq)]
    n_ks = [max(0, n + r.choice((-300, -1, 0, 0, 1, 127, 128, 900))) for n in n_qs]
    n_qs[0], n_ks[0] = 1500, 2100
    want = expected(n_qs, n_ks, H)
    n = len(want)
    up = list(range(n))
    any_order = [r.randrange(n) for _ in range(3 * n)]
    steps = [i for j in range(0, n, 5) for i in (j, max(0, j - 3), min(n - 1, j + 7))]       # forward with steps back
    cu = [torch.tensor([0] + list(np.cumsum(v)), dtype=torch.int32).cuda() for v in (n_qs, n_ks)]
    for order in (up, up[::-1], any_order, steps):
        o = torch.tensor(order, dtype=torch.int32).cuda()
        out, total = torch.full((len(order), 9), -7, dtype=torch.int32).cuda(), torch.zeros(1, dtype=torch.int32).cuda()
        torch.cuda.synchronize()
        rc = lib.run(ctypes.c_void_p(cu[0].data_ptr()), ctypes.c_void_p(cu[1].data_ptr()), n_seq, sum(n_qs), sum(n_ks), H,
                     ctypes.c_void_p(o.data_ptr()), len(order), ctypes.c_void_p(out.data_ptr()), ctypes.c_void_p(total.data_ptr()))
        assert rc == 0 and int(total) == n
        got = out.cpu().tolist()
        # head, q0, nq, nk, qrow, krow, nt[0], nt[1], n
        assert got == [want[i] for i in order]
