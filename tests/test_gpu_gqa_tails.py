"""Prompts of f32 tensors whose queries see one key far above very many others: the others' share of the output, some tenths of a
per cent, is there as the definition has it.

Tolerance.  All keys but one score 0, that one `above`: every probability of the tail is the same p, off by u = 2^-11 as an f16 number of
11 bits, or by half a step of the smallest ones, 2^-25, where the largest score's is 2^7 or more: n of them by n 2^-32.  Values of 0 and
1 are exact; exp and sums 1e-4."""
import math

import pytest

from test_gpu_gqa import gen, setup

pytestmark = pytest.mark.gpu


def call(torch, coli, q, k, v, scale):
    out = torch.full(q.shape, -5.0, device="cuda")
    cu = [torch.tensor([0, t.shape[0]], dtype=torch.int32, device="cuda") for t in (q, k)]
    coli.gqa_prefill(q.cuda(), k.cuda(), v.cuda(), *cu, scale, out)
    coli.sync_check()
    return out.cpu().double()


@pytest.mark.parametrize("at", [0, 9000, 19999])
@pytest.mark.parametrize("above", [12.0, 16.0, 17.0, 18.0])
@pytest.mark.parametrize("dim", [64, 128])
def test_one_key_above_many(dim, above, at):
    torch, coli = setup()
    n = 20000
    q, k, v = torch.zeros(1, 1, dim), torch.zeros(n, 1, dim), torch.zeros(n, 1, dim)
    q[0, 0, 0] = k[at, 0, 0] = 1.0
    v[:, 0, 0] = 1.0                                     # what the tail has
    v[at, 0, 0], v[at, 0, 1] = 0.0, 1.0
    v[:, 0, 2] = 1.0                                     # everyone has this
    got = call(torch, coli, q, k, v, above)[0, 0]
    z = math.exp(above) + n - 1
    tail = (n - 1) / z
    slack = lambda x: (2.0 ** -11 + 1e-4) * x + n * 2.0 ** -32  # noqa: E731
    assert abs(float(got[0]) - tail) <= slack(tail)
    assert abs(float(got[1]) - (1 - tail)) <= slack(1.0)
    assert abs(float(got[2]) - 1.0) <= slack(1.0)


@pytest.mark.parametrize("above", [14.0, 17.0])
def test_one_key_above_random_ones(above):
    """The same with random scores and values around it; several queries and heads."""
    torch, coli = setup()
    g = gen(torch, 5)
    n, dim = 12000, 64
    q, k, v = torch.randn(3, 2, dim, generator=g) * 0.01, torch.randn(n, 1, dim, generator=g), torch.randn(n, 1, dim, generator=g)
    q[:, :, 0], k[:, 0, 0] = 1.0, 0.0
    k[7000, 0, 0] = above
    v[:, 0, 3], v[7000] = 1.0, 0.0
    v[7000, 0, 1] = 1.0
    got = call(torch, coli, q, k, v, 1.0)
    s = torch.einsum("ihd,jd->hij", q.double(), k[:, 0].double())
    s = s.masked_fill(torch.arange(n)[None, None] > torch.arange(3)[None, :, None] + n - 3, -math.inf)
    p = torch.softmax(s, -1)
    ref, size = torch.einsum("hij,jd->ihd", p, v[:, 0].double()), torch.einsum("hij,jd->ihd", p, v[:, 0].abs().double())
    # scores: sums of |q| |k| below 1 but for the one key (exact there: powers and small numbers of bits), 2^-10 of them; magnitudes up to 8
    slack = (2.0 ** -10 + 2 * 2.0 ** -10 * 1.0 + 1e-4) * size + n * 2.0 ** -32 * 8
    assert ((got - ref).abs() <= slack).all()
