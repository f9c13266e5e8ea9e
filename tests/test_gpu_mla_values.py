"""Latent attention on the GPU where values are special: NaN and infinities in operands that count and in places that a
query does not see, rows of scale 0, queries of widely spread magnitudes, more query rows than a launch has columns.

Tolerances.  out = sum_t p_t c_t: rounding p to 16 bits moves it by r * sum_t p_t |c_t| (r = 2^-8 for a bf16 cache; 2^-11
for the E4M3 one's three terms), scores off by d by expm1(2 d) of the same, f32 sums and exp by 1e-4 of it for these
lengths, a bf16 output by 2^-8 of itself.  d = scale * max_t sum_i e_i |k_ti| + 2^-21 of the same sum with |q_i|, where e_i is
what the operand of element q_i is off by.  bf16 cache: 0 for bf16 queries, 2^-8 |q_i| for f32 ones.  E4M3 cache: the row
is scaled so that its largest element M lies in [2^7, 2^8); the first E4M3 term leaves 2^-4 of an element or 2^-10, the
second 2^-4 of that or 2^-10 / 32: 2^-8 |q_i|, and no less than 2^-15, at most 2^-22 M unscaled; for f32 queries the
f16 in between adds 2^-11 |q_i|; a bf16 element has 8 bits, which the two terms hold, so 2^-22 M alone is left."""
import math

import pytest

from test_gpu_mla import U16, UF16, filled, gen, new_cache, rotation, sequence, setup, values

pytestmark = pytest.mark.gpu


def attend(torch, coli, c, table, lens, ql, qr, scale, out_bf16=False, stream=None):
    out = torch.full(ql.shape, 7.0, device="cuda", dtype=torch.bfloat16 if out_bf16 else torch.float32)
    ls = torch.full(ql.shape[:3], 7.0, device="cuda")
    coli.mla_attend(c, ql.cuda(), qr.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale, out, ls)
    coli.sync_check()
    return out.cpu(), ls.cpu()


def check(torch, c, table, lens, ql, qr, scale, out, ls, skip=lambda b, j: None):
    """Every row against the definition in 64 bits, but for the heads that skip(b, j) names."""
    B, n_q, H, L = ql.shape
    e4m3 = c.scales is not None
    r = UF16 if e4m3 else U16
    vals = values(torch, c)
    for b in range(B):
        rows = sequence(torch, vals, table, b, lens[b], c.page_size)
        for j in range(n_q):
            n = lens[b] - (n_q - 1 - j)
            heads = torch.tensor([h for h in range(H) if h not in (skip(b, j) or ())], dtype=torch.long)
            if not len(heads):
                continue
            o, l = out[b, j, heads].double(), ls[b, j, heads].double()
            if n <= 0:
                assert (o == 0).all() and (l == -math.inf).all()
                continue
            q, k = torch.cat([ql[b, j, heads], qr[b, j, heads]], -1).double(), rows[:n]
            s = q @ k.T * scale
            p = torch.softmax(s, -1)
            ref, size = p @ k[:, :L], p @ k[:, :L].abs()
            e = torch.zeros_like(q)
            if ql.dtype == torch.float32:
                e += U16 * q.abs() + (UF16 * q.abs() if e4m3 else 0.0)
            if e4m3:
                e += 2.0 ** -22 * q.abs().amax(-1, keepdim=True)
            d = abs(scale) * ((e + 2.0 ** -21 * q.abs()) @ k.abs().T).amax(-1, keepdim=True)
            tol = (r + torch.expm1(2 * d) + 1e-4) * size + (U16 if out.dtype == torch.bfloat16 else 0.0) * ref.abs() + 1e-30
            assert ((o - ref).abs() <= tol).all(), (b, j, float(((o - ref).abs() / tol).max()))
            want = torch.logsumexp(s, -1)
            assert ((l - want).abs() <= 1e-4 + d[:, 0] + 2e-6 * want.abs()).all(), (b, j, float((l - want).abs().max()))


def queries(torch, g, B, n_q, H, L, R, bf16, scale=1.0):
    t = torch.bfloat16 if bf16 else torch.float32
    return (torch.randn(B, n_q, H, L, generator=g) * scale).to(t), (torch.randn(B, n_q, H, R, generator=g) * scale).to(t)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_nan_query(e4m3, bf16):
    """A NaN in a head's query makes that head's output and lse NaN, and nothing else."""
    torch, coli = setup()
    g = gen(torch, 1)
    lens, L, R = [300, 40, 1], 256, 32
    c, table = filled(torch, coli, e4m3, L, R, 16, lens, g)
    ql, qr = queries(torch, g, 3, 1, 40, L, R, bf16)
    ql[0, 0, 3, 7] = qr[1, 0, 5, 2] = ql[2, 0, 39, 255] = float("nan")
    bad = {0: [3], 1: [5], 2: [39]}
    out, ls = attend(torch, coli, c, table, lens, ql, qr, 0.06)
    for b, (h,) in bad.items():
        assert torch.isnan(out[b, 0, h]).all() and torch.isnan(ls[b, 0, h])
    check(torch, c, table, lens, ql, qr, 0.06, out, ls, lambda b, j: bad[b])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("token", [0, 200, 1000, 2999])
@pytest.mark.parametrize("where", [3, 255, 270])
def test_nan_row(e4m3, token, where):
    """A NaN in a cached row that counts, in its latent or its rotary part, makes its sequence's outputs NaN, and no other's."""
    torch, coli = setup()
    g = gen(torch, 2)
    lens, L, R, page, H = [3000, 90], 256, 32, 16, 1024      # many heads: few CTAs share the tokens, several tiles each
    c, table = filled(torch, coli, e4m3, L, R, page, lens, g)
    c.rows[int(table[0, token // page]), token % page].view(torch.uint8 if e4m3 else torch.int16)[where] = 0x7F if e4m3 else 0x7FC0
    ql, qr = queries(torch, g, 2, 1, H, L, R, True)
    out, ls = attend(torch, coli, c, table, lens, ql, qr, 0.06)
    assert torch.isnan(out[0]).all() and torch.isnan(ls[0]).all()
    check(torch, c, table, lens, ql, qr, 0.06, out, ls, lambda b, j: range(H) if b == 0 else ())


@pytest.mark.parametrize("token", [5, 130, 1000, 2999])
def test_infinite_row(token):
    """An infinity in the rotary part of a bf16 row: the heads that it gives a score of +inf are NaN, those of -inf do not see it."""
    torch, coli = setup()
    g = gen(torch, 3)
    L, R, page, H, lens = 256, 32, 16, 1024, [3000]
    c, table = filled(torch, coli, False, L, R, page, lens, g)
    at = (int(table[0, token // page]), token % page, L + 4)
    c.rows[at] = float("inf")
    ql, qr = queries(torch, g, 1, 1, H, L, R, True)
    up = [h for h in range(H) if qr[0, 0, h, 4] > 0]
    out, ls = attend(torch, coli, c, table, lens, ql, qr, 0.06)
    assert 0 < len(up) < H
    assert torch.isnan(out[0, 0, up]).all() and torch.isnan(ls[0, 0, up]).all()
    c.rows[at] = 1e30                     # as good as +inf for a negative factor
    down = [h for h in range(H) if h not in up]
    again, ls2 = attend(torch, coli, c, table, lens, ql, qr, 0.06)
    assert torch.equal(out[0, 0, down], again[0, 0, down]) and torch.equal(ls[0, 0, down], ls2[0, 0, down])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_query(e4m3, bf16, sign):
    """An infinite query element gives scores of +inf and -inf: that head is NaN, and nothing else."""
    torch, coli = setup()
    g = gen(torch, 4)
    lens, L, R = [300, 140], 256, 32
    c, table = filled(torch, coli, e4m3, L, R, 16, lens, g)
    ql, qr = queries(torch, g, 2, 1, 40, L, R, bf16)
    ql[0, 0, 3, 7] = qr[1, 0, 5, 2] = sign * float("inf")
    bad = {0: [3], 1: [5]}
    out, ls = attend(torch, coli, c, table, lens, ql, qr, 0.06)
    for b, (h,) in bad.items():
        assert torch.isnan(out[b, 0, h]).all() and torch.isnan(ls[b, 0, h])
    check(torch, c, table, lens, ql, qr, 0.06, out, ls, lambda b, j: bad[b])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("fill", [0.0, 1.0, float("nan")])
def test_append_keeps_nan(interleaved, norm, fill):
    """A token with a NaN leaves NaN in its E4M3 row (all of its latent part under a norm), whatever stands beside it, zeros included."""
    torch, coli = setup()
    L, R = 128, 16
    c = new_cache(torch, coli, True, L, R, 16, 1, junk=False)
    kv = torch.full((3, L + R), fill)
    kv[0, 5] = kv[1, L + 3] = float("nan")      # latent, rotary
    kv[2, :] = 2.0
    w = torch.ones(L).cuda() if norm else None
    pos = torch.full((3,), 2, dtype=torch.int32).cuda()
    coli.mla_append(c, kv.cuda(), w, 1e-6, pos, rotation(torch, 4, R).cuda(), torch.arange(3).cuda(), interleaved)
    coli.sync_check()
    got = values(torch, c)
    pair = (2, 3) if interleaved else (3, 3 + R // 2)
    assert torch.isnan(got[0, :L]).all() if norm else torch.isnan(got[0, 5])
    assert torch.isnan(got[1, L + pair[0]]) and torch.isnan(got[1, L + pair[1]])
    assert not torch.isnan(got[2]).any()
    if fill == fill and not norm:
        assert not torch.isnan(got[0, :5]).any() and not torch.isnan(got[1, :L]).any()


@pytest.mark.parametrize("below", [94.5, 96.0, 97.5, 99.0, 140.0])
def test_rows_of_scale_0_outweigh(below):
    """Rows of scale 0 (value 0, score 0) after tiles whose scores lie far below: they take all the weight."""
    torch, coli = setup()
    L, R, page, n, H = 128, 16, 64, 1500, 1024    # many heads: few CTAs share the tokens, three tiles each
    c = new_cache(torch, coli, True, L, R, page, 24, junk=False)
    c.rows.view(-1, L + R)[:128, :2] = 1.0
    c.scales.view(-1)[:128] = 1.0               # the first tile: scores of -below log2 units; the others: scale 0
    ql, qr = torch.zeros(1, 1, H, L), torch.zeros(1, 1, H, R)
    ql[..., 0] = -below * math.log(2.0)
    table = torch.arange(24, dtype=torch.int32)[None]
    out, ls = attend(torch, coli, c, table, [n], ql, qr, 1.0)
    # lse = ln(1372 + 128 2^-below); out = 128 2^-below / 1372 of the first tile's rows
    assert ((ls - math.log(1372.0)).abs() <= 1e-4).all()
    assert (out.abs() <= 2.0 ** (1 - below)).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n_q,n", [(2, 200), (3, 129), (4, 257), (130, 140)])
def test_tokens_that_some_queries_do_not_see(e4m3, value, n_q, n):
    """A newest token's row that is not finite leaves the queries before it alone."""
    torch, coli = setup()
    g = gen(torch, 5)
    L, R, page, H = 256, 32, 16, 5
    c, table = filled(torch, coli, e4m3, L, R, page, [n, 70], g)
    at = (int(table[0, (n - 1) // page]), (n - 1) % page)
    if e4m3:
        c.scales[at] = value
        c.rows[at].view(torch.uint8)[::3] = 0x7F
    else:
        c.rows[at[0], at[1], ::3] = value
    ql, qr = queries(torch, g, 2, n_q, H, L, R, True)
    out, ls = attend(torch, coli, c, table, [n, 70], ql, qr, 0.06)
    vals = c.rows[at].view(torch.uint8 if e4m3 else torch.int16)
    vals.zero_()                                # for the reference alone: no query that is checked sees the row
    if e4m3:
        c.scales[at] = 0.0
    check(torch, c, table, [n, 70], ql, qr, 0.06, out, ls, lambda b, j: range(H) if b == 0 and j == n_q - 1 else ())
    if value != value or e4m3:
        assert torch.isnan(out[0, n_q - 1]).all()


def test_tensors_of_another_device(monkeypatch):
    """The library launches on the current device: tensors of another one are refused before that, with COLI_EDEVICE."""
    torch, coli = setup()
    c = new_cache(torch, coli, True, 512, 64, 64, 3)
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    q, rot, pos, pages, lens = z(2, 4, 192), rotation(torch, 8, 64).cuda(), z(2, dtype=torch.int32), z(2, 1, dtype=torch.int32), z(2, dtype=torch.int32)
    on, orr, cu = z(2, 4, 128), z(2, 4, 64), z(2, dtype=torch.int32)
    ql, qr = z(2, 1, 4, 512), z(2, 1, 4, 64)
    calls = [lambda: coli.mla_query(q, pos, rot, on, orr), lambda: coli.mla_append(c, z(2, 576), None, 1.0, pos, rot, pos.long()),
             lambda: coli.mla_read(c, pages[:1], cu, z(2, 576)), lambda: coli.mla_attend(c, ql, qr, pages, lens, 1.0, ql.clone()),
             lambda: coli.mla_prefill(q, z(2, 4, 256), orr[:, 0], cu, cu, 1.0, on)]
    for f in calls:
        f()
    coli.sync_check()
    monkeypatch.setattr(coli, "_device", lambda: 1, raising=False)
    for f in calls:
        with pytest.raises(coli.ColiError) as e:
            f()
        assert e.value.code == coli.COLI_EDEVICE
    monkeypatch.undo()
    host = lambda t: pytest.raises(coli.ColiError, match="CUDA tensor")  # noqa: E731
    with host(pos):
        coli.mla_query(q, pos.cpu(), rot, on, orr)
    with host(pages):
        coli.mla_read(c, pages[:1].cpu(), cu, z(2, 576))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_more_query_rows_than_the_device_has_columns(e4m3, bf16):
    """12800 query rows a sequence: every CTA takes several blocks of rows, each over all sequences."""
    torch, coli = setup()
    g = gen(torch, 6)
    lens, L, R = [150, 300], 128, 16
    c, table = filled(torch, coli, e4m3, L, R, 16, lens, g)
    ql, qr = queries(torch, g, 2, 100, 128, L, R, bf16)
    out, ls = attend(torch, coli, c, table, lens, ql, qr, 0.08, out_bf16=bf16)
    check(torch, c, table, lens, ql, qr, 0.08, out, ls)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("latent,rope", [(1.0, 1.0), (1.0, 1e-3), (1.0, 1e-5), (1e-3, 1.0), (1e-5, 1.0), (3e4, 1e-30), (1e-30, 1e-30)])
def test_query_magnitudes(e4m3, bf16, latent, rope):
    """Parts of a query that differ by orders of magnitude."""
    torch, coli = setup()
    g = gen(torch, 7)
    lens, L, R, H = [700, 33], 512, 64, 20
    c, table = filled(torch, coli, e4m3, L, R, 64, lens, g)
    ql, qr = queries(torch, g, 2, 1, H, L, R, False)
    t = torch.bfloat16 if bf16 else torch.float32
    ql, qr = (ql * latent).to(t), (qr * rope).to(t)
    scale = 0.07 / max(1.0, latent)
    out, ls = attend(torch, coli, c, table, lens, ql, qr, scale)
    check(torch, c, table, lens, ql, qr, scale, out, ls)


@pytest.mark.parametrize("e4m3", [False, True])
def test_tables_wider_than_the_lengths(e4m3):
    """Tables as wide as the longest context that a server allows, short sequences on them, more of them than SMs."""
    torch, coli = setup()
    g = gen(torch, 8)
    lens = [(37 * i) % 300 for i in range(200)]
    c, table = filled(torch, coli, e4m3, 256, 32, 64, lens, g, columns=4000)
    ql, qr = queries(torch, g, 200, 1, 16, 256, 32, True)
    out, ls = attend(torch, coli, c, table, lens, ql, qr, 0.06)
    check(torch, c, table, lens, ql, qr, 0.06, out, ls)
