"""Prompts of f32 tensors through grouped-head attention against the definition in 64 bits on the f32 tensors as they are, and
what a query does not see: whatever it holds, no bit of the query's output changes.

Tolerance.  An element of q, k or v becomes f16 with its row's power of two: off by u = 2^-11 of itself, or, where it is small, by half an
f16 step of 2^-24: 2^-39 of the row's largest magnitude, which goes to 2^14 .. 2^15; 2^-29 for a key's row of ordinary size (its largest
magnitude in 2^-5 .. 2^11; a power of 2^4); 2^-40 size for a value's, size the upper end of the place of its largest magnitude between
2^-4, 2^6, 2^16 and so on, which goes to 2^15.  A score s_ij = scale q_i . k_j is then off by at most
    d_ij = scale ((2 u + u^2 + 128 x 2^-24) sum |q| |k| + sum (|q| of k's small step, |k| of q's)),
the third term for the f32 sum of up to 128 products.  With e^d weights around, out' - out = sum p_j (e^(delta_j) - 1) (v_j - out) /
sum p_j e^(delta_j), at most e^(max d) sum p_j (e^(d_j) - 1) |v_j - out|.  Values and probabilities are off by u each: 2 u + u^2 of
sum p |v|; exp, sums and the division by 1e-4 of it.  Small f16 weights of the product are off by half a step of 2^-24.  They are
p_j size_j times something that takes the largest of a query's to 100 or more, with values of 2^15 |v_j| / size_j: n 2^-25 / 100 of the largest
p size, less than n 2^-31."""
import math

import pytest

from test_gpu_gqa import PROMPTS, gen, packed_qkv, setup

pytestmark = pytest.mark.gpu

U = 2.0 ** -11


def i32(torch, x):
    return torch.tensor([int(i) for i in x], dtype=torch.int32, device="cuda")


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def small(torch, rows, lo, hi, step):
    """What a small element of each row is off by."""
    most = rows.abs().amax(-1)
    return torch.where((most >= lo) & (most < hi) | (most == 0), step, 2.0 ** -39 * most)


def definition(torch, q, k, v, cu_q, cu_k, scale):
    """Outputs, tolerances and lse in 64 bits, and the lse's tolerance."""
    Tq, H, D = q.shape
    group = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, tol = torch.zeros(Tq, H, D, dtype=torch.float64), torch.zeros(Tq, H, D, dtype=torch.float64)
    lse, lse_tol = torch.full((Tq, H), -math.inf, dtype=torch.float64), torch.zeros(Tq, H, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = q1 - q0, k1 - k0
        if n == 0 or m == 0:
            continue
        seen = torch.arange(m)[None, :] <= torch.arange(n)[:, None] + m - n
        some = seen.any(-1)
        for h in range(H):
            x, y, z = q[q0:q1, h], k[k0:k1, h // group], v[k0:k1, h // group]
            a = (x @ y.T * scale).masked_fill(~seen, -math.inf)
            p = torch.zeros_like(a)
            p[some] = torch.softmax(a[some], -1)
            d = abs(scale) * (2 * U + U * U + 128 * 2.0 ** -24) * (x.abs() @ y.abs().T)
            d += abs(scale) * x.abs().sum(-1, keepdim=True) * small(torch, y, 2.0 ** -5, 2.0 ** 11, 2.0 ** -29)[None, :]
            d += abs(scale) * 2.0 ** -39 * x.abs().amax(-1, keepdim=True) * y.abs().sum(-1)[None, :]
            d = d.masked_fill(~seen, 0.0)
            o = p @ z
            w = p * torch.expm1(d)
            most = d.amax(-1, keepdim=True).exp()
            # sum_j w_ij |z_j - o_i|, some rows at a time
            move = torch.empty_like(o)
            for i in range(0, n, 16):
                move[i:i + 16] = (w[i:i + 16, :, None] * (z[None] - o[i:i + 16, None]).abs()).sum(1)
            out[q0:q1, h] = o
            size = z.abs().amax(-1)
            size = torch.where(size == 0, 64.0, 2.0 ** (6 + 10 * ((size.log2().floor() + 4) / 10).floor()))
            tol[q0:q1, h] = most * move + (2 * U + U * U + 1e-4) * (p @ z.abs()) + 2.0 ** -40 * (p @ size)[:, None] + m * 2.0 ** -31 * (p * size).amax(-1, keepdim=True)
            lse[q0:q1, h] = torch.logsumexp(a, -1)
            lse_tol[q0:q1, h] = d.amax(-1) + 1e-5 * (1 + a.masked_fill(~seen, 0).abs().amax(-1))
    return out, tol, lse, lse_tol


def call(torch, coli, q, k, v, cu_q, cu_k, scale, out=None, lse=None):
    out = torch.full(q.shape, -5.0, device="cuda") if out is None else out
    coli.gqa_prefill(q.cuda(), k.cuda(), v.cuda(), i32(torch, cu_q), i32(torch, cu_k), scale, out, lse)
    coli.sync_check()
    return out.cpu()


@pytest.mark.parametrize("lens_q,lens_k,H,K,D", PROMPTS)
@pytest.mark.parametrize("scale", [1.0, -0.4])
def test_definition(lens_q, lens_k, H, K, D, scale):
    torch, coli = setup()
    g = gen(torch, sum(lens_q) + H + K)
    q, kv = packed_qkv(torch, lens_q, lens_k, H, K, D, g, torch.float32, 1.5)
    cu_q, cu_k = offsets(lens_q), offsets(lens_k)
    lse = torch.empty(cu_q[-1], H, device="cuda")
    k, v = kv[:, :K].contiguous(), kv[:, K:2 * K].contiguous()
    got = call(torch, coli, q, k, v, cu_q, cu_k, scale / math.sqrt(D), lse=lse).double()
    ref, tol, ref_lse, lse_tol = definition(torch, q, k, v, cu_q, cu_k, scale / math.sqrt(D))
    assert ((got - ref).abs() <= tol).all()
    none = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse.cpu()), none) and ((lse.cpu().double() - ref_lse).abs() <= lse_tol)[~none].all()


@pytest.mark.parametrize("dim", [64, 128])
def test_rows_of_all_sizes(dim):
    """Each row of q, k and v has a size of its own: keys 2^-30 to 2^3, queries 2^-60 to 2^4, values 2^-90 to 2^90, beside one another."""
    torch, coli = setup()
    g = gen(torch, dim)
    q, kv = packed_qkv(torch, [150, 40], [290, 40], 6, 2, dim, g, torch.float32)
    size = lambda lo, hi, *shape: 2.0 ** torch.randint(lo, hi + 1, shape, generator=g).float()  # noqa: E731
    q = q * size(-60, 4, 190, 6, 1)
    k, v = kv[:, :2] * size(-30, 3, 330, 2, 1), kv[:, 2:4] * size(-90, 90, 330, 2, 1)
    got = call(torch, coli, q, k, v, [0, 150, 190], [0, 290, 330], 0.1).double()
    ref, tol, *_ = definition(torch, q, k, v, [0, 150, 190], [0, 290, 330], 0.1)
    assert torch.isfinite(got).all() and ((got - ref).abs() <= tol).all()


@pytest.mark.parametrize("size_q,size_k,size_v", [(-100, 66, 0), (83, -83, 100), (0, 0, -100), (-16, -16, -16), (100, -70, -60), (3, 110, 112)])
def test_powers_of_two(size_q, size_k, size_v):
    """Tensors a power of two larger or smaller, and a scale that takes the scores back, change no bit but that power of the outputs."""
    torch, coli = setup()
    g = gen(torch, 8)
    q, kv = packed_qkv(torch, [70], [190], 4, 2, 64, g, torch.float32)
    k, v = kv[:, :2].contiguous(), kv[:, 2:4].contiguous()
    want = call(torch, coli, q, k, v, [0, 70], [0, 190], 0.125)
    got = call(torch, coli, q * 2.0 ** size_q, k * 2.0 ** size_k, v * 2.0 ** size_v, [0, 70], [0, 190], 0.125 * 2.0 ** (-size_q - size_k))
    assert torch.equal(got, want * 2.0 ** size_v)


JUNK = [3e38, -3e38, 1e12, 1e30, 1e-38, math.nan, math.inf, -math.inf]


@pytest.mark.parametrize("where", ["k", "v", "both"])
def test_strangers_do_not_matter(where):
    """Other sequences' rows and rows of no sequence."""
    torch, coli = setup()
    g = gen(torch, 11)
    q, kv = packed_qkv(torch, [100, 60, 70], [100, 60, 70], 8, 2, 128, g, torch.float32)
    cu = [0, 100, 160]                                                    # two sequences; the third's rows are no one's
    k, v = kv[:, :2].contiguous(), kv[:, 2:4].contiguous()
    seven = lambda: torch.full((230, 8, 128), 7.0, device="cuda")  # noqa: E731
    want = call(torch, coli, q, k, v, cu, cu, 0.09, out=seven())
    assert (want[160:] == 7).all()
    for junk in JUNK:
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for rows, same in ((slice(160, None), 160), (slice(100, 160), 100)):
            if where != "v":
                q2[rows], k2[rows] = junk, junk
            if where != "k":
                v2[rows] = junk
            got = call(torch, coli, q2, k2, v2, cu, cu, 0.09, out=seven())
            assert torch.equal(got[:same], want[:same]), (junk, same)
            assert (got[160:] == 7).all()


@pytest.mark.parametrize("lens_q,lens_k,H,K,D", [([150], [150], 4, 2, 64), ([70], [300], 14, 2, 128), ([300, 7], [300, 40], 2, 2, 128)])
def test_masked_keys_do_not_matter(lens_q, lens_k, H, K, D):
    """Keys and values of a query's own sequence behind those that it sees; one element of a row, or all of it."""
    torch, coli = setup()
    g = gen(torch, H + D)
    q, kv = packed_qkv(torch, lens_q, lens_k, H, K, D, g, torch.float32)
    cu_q, cu_k = offsets(lens_q), offsets(lens_k)
    k, v = kv[:, :K].contiguous(), kv[:, K:2 * K].contiguous()
    want = call(torch, coli, q, k, v, cu_q, cu_k, 0.09)
    for junk in JUNK:
        for back, columns in ((1, slice(None)), (20, slice(3, 4))):
            k2, v2 = k.clone(), v.clone()
            for b, n in enumerate(lens_k):
                if back < n:
                    k2[cu_k[b] + n - back, :, columns] = junk
                    if math.isfinite(junk):               # rows beside values that are not are computed in another order
                        v2[cu_k[b] + n - back, :, columns] = junk
            got = call(torch, coli, q, k2, v2, cu_q, cu_k, 0.09)
            for b, n in enumerate(lens_q):
                blind = max(0, n - back)                  # queries that do not see that key
                assert torch.equal(got[cu_q[b]:cu_q[b] + blind], want[cu_q[b]:cu_q[b] + blind]), (junk, back)


@pytest.mark.parametrize("dim", [64, 128])
def test_large_values_that_are_seen(dim):
    """A large value beside ordinary ones in other rows reaches the rows that see it by its weight, and in full range: a sum of
    weights times 3e38 is no larger than 3e38."""
    torch, coli = setup()
    g = gen(torch, 14)
    q, kv = packed_qkv(torch, [200], [200], 2, 1, dim, g, torch.float32)
    k, v = kv[:, :1].contiguous(), kv[:, 1:2].contiguous()
    v[40, 0, 5], v[41, 0, 6], v[130, 0, 7] = 1e12, -1e30, 1e20
    v[:, 0, 9] = 3e38
    got = call(torch, coli, q, k, v, [0, 200], [0, 200], 0.1).double()
    ref, tol, *_ = definition(torch, q, k, v, [0, 200], [0, 200], 0.1)
    assert torch.isfinite(got).all() and ((got - ref).abs() <= tol).all()


@pytest.mark.parametrize("size", [-70, -37, -9, 12, 31, 90])
def test_values_of_another_size_beside_junk(size):
    """Values that are all large or all small, ordinary ones in between, junk where nobody looks: the same bits, the definition's values."""
    torch, coli = setup()
    g = gen(torch, 17)
    q, kv = packed_qkv(torch, [300, 20], [500, 20], 4, 1, 64, g, torch.float32)
    k, v = kv[:, :1].contiguous(), kv[:, 1:2] * 2.0 ** size
    v[100:200] *= 2.0 ** -size                            # a few tiles of ordinary ones
    want = call(torch, coli, q, k, v, [0, 300, 320], [0, 500, 520], 0.1)
    ref, tol, *_ = definition(torch, q, k, v, [0, 300, 320], [0, 500, 520], 0.1)
    assert ((want.double() - ref).abs() <= tol).all()
    for junk in JUNK:
        v2, k2 = v.clone(), k.clone()
        k2[450:500], k2[510:] = junk, junk
        if math.isfinite(junk):
            v2[450:500], v2[510:] = junk, junk
        got = call(torch, coli, q, k2, v2, [0, 300, 320], [0, 500, 520], 0.1)
        assert torch.equal(got[:250], want[:250]) and torch.equal(got[300:310], want[300:310]), junk
