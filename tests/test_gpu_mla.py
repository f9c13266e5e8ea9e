"""Latent attention on the GPU against plain 64-bit computations of the
definitions: the queries' rotation, the cache write and read back, attention
over the cache (absorbed form) and of prompts (expanded form).

Tolerances follow from the roundings of the operators.  One rounding to bf16
(8 significant bits) is off by at most 2^-8 of the value, one to f16 (11 bits)
by 2^-11 (normal range), one to E4M3 (4 bits, steps of 2^-9 below its normal
range) by 2^-4 of the value or 2^-10 of the row's scale.  An attention output
is sum_t p_t v_t: rounding every p_t to 16 bits moves it by at most r * sum_t
p_t |v_t| (r = 2^-8 for bf16, 2^-11 for f16), a rounded q moves the scores by
at most d = r * scale * max_t sum_i |q_i| |k_ti| and with them every p_t by at
most a factor exp(2 d), f32 sums, exp and the f32 score add 1e-4 at most for
the lengths used here, and a bf16 output rounds once more."""
import math
import random

import numpy as np
import pytest

from gpu_util import cuda_or_skip

pytestmark = pytest.mark.gpu

U16, UF16 = 2.0 ** -8, 2.0 ** -11    # half a step of bf16 and of f16, relative to the value


def setup():
    torch = cuda_or_skip()
    import bit_weight_gemv_fmt1_gb300 as coli
    return torch, coli


def gen(torch, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rotation(torch, n_pos, R):
    f = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotated(torch, x, rot, interleaved):
    """64-bit rotation of x [..., R] by rot [..., R]."""
    x, rot = x.double(), rot.double()
    h = x.shape[-1] // 2
    c, s = rot[..., :h], rot[..., h:]
    y = torch.empty_like(x)
    ia, ib = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, h), slice(h, None))
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y


# ------------------------------------------------------------------ query
@pytest.mark.parametrize("T,H,N,R", [(1, 128, 128, 64), (37, 5, 128, 64), (3, 1, 0, 16), (130, 7, 64, 48), (2, 3, 192, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("types", ["f32", "bf16", "mixed", "joined"])
def test_query(T, H, N, R, interleaved, types):
    torch, coli = setup()
    g = gen(torch, T + H + N + R)
    pad = 16
    q = torch.randn(T, H * (N + R) + pad, generator=g)
    rot = rotation(torch, 300, R)
    pos = torch.randint(0, 300, (T,), generator=g, dtype=torch.int32)
    qd = q.cuda()[:, :H * (N + R)].unflatten(1, (H, N + R))      # token stride with padding
    if types == "joined":
        out = torch.full((T, H, N + R), float("nan"), device="cuda", dtype=torch.bfloat16)
        on, orr = out[..., :N], out[..., N:]
    else:
        on = torch.full((T, H, N), float("nan"), device="cuda", dtype=torch.bfloat16 if types == "bf16" else torch.float32)
        orr = torch.full((T, H, R), float("nan"), device="cuda", dtype=torch.float32 if types == "f32" else torch.bfloat16)
    coli.mla_query(qd, pos.cuda(), rot.cuda(), on if N else None, orr, interleaved=interleaved)
    coli.sync_check()
    x = q[:, :H * (N + R)].view(T, H, N + R)
    if N:
        assert torch.equal(on.cpu(), x[..., :N].to(on.dtype))
    ref = rotated(torch, x[..., N:], rot[pos.long()][:, None], interleaved)
    size = x[..., N:].double().abs().amax(-1, keepdim=True) * 2
    tol = size * 2.0 ** -22 + (0 if orr.dtype == torch.float32 else U16) * ref.abs()
    assert ((orr.cpu().double() - ref).abs() <= tol).all()


def test_query_position_out_of_range():
    torch, coli = setup()
    q = torch.randn(3, 2, 80, device="cuda")
    pos = torch.tensor([0, 9, 1], dtype=torch.int32, device="cuda")
    on, orr = torch.ones(3, 2, 64, device="cuda"), torch.ones(3, 2, 16, device="cuda")
    coli.mla_query(q, pos, rotation(torch, 9, 16).cuda(), on, orr)
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_EINVAL
    assert (orr[1] == 0).all() and (orr[0] != 0).any()
    coli.sync_check()


# ------------------------------------------------------------------ cache
def new_cache(torch, coli, e4m3, L, R, page, n_pages, junk=True):
    """A cache whose rows hold NaN until they are written."""
    if e4m3:
        rows = torch.full((n_pages, page, L + R), 0x7F if junk else 0, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        scales = torch.full((n_pages, page), float("nan") if junk else 0.0, device="cuda")
    else:
        rows = torch.full((n_pages, page, L + R), float("nan") if junk else 0.0, dtype=torch.bfloat16, device="cuda")
        scales = None
    return coli.MlaCache(rows, L, R, scales)


def values(torch, c):
    """The cache's values in 64 bits, on the host: [slots, L + R]."""
    n = c.latent + c.rope
    if c.scales is None:
        return c.rows.cpu().view(-1, n).double()
    return c.rows.cpu().view(-1, n).float().double() * c.scales.cpu().view(-1, 1).double()


@pytest.mark.parametrize("T,L,R,page", [(1, 512, 64, 64), (8, 512, 64, 16), (133, 512, 64, 48), (50, 128, 16, 32), (21, 384, 48, 16),
                                        (9, 256, 32, 128)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved,norm", [(False, True), (True, False), (True, True)])
def test_append(T, L, R, page, e4m3, interleaved, norm):
    torch, coli = setup()
    g = gen(torch, T + L + R)
    kv = torch.randn(T, L + R + 4, generator=g) * (10.0 ** (torch.rand(T, 1, generator=g) * 8 - 4))
    w = torch.rand(L, generator=g) + 0.5
    rot = rotation(torch, 500, R)
    pos = torch.randint(0, 500, (T,), generator=g, dtype=torch.int32)
    n_pages = -(-T // page) + 2
    c = new_cache(torch, coli, e4m3, L, R, page, n_pages)
    slots = torch.randperm(n_pages * page, generator=g)[:T]
    skipped = T // 3
    given = slots.clone()
    given[skipped] = -1 if T > 1 else slots[0]
    coli.mla_append(c, kv.cuda()[:, :L + R], w.cuda() if norm else None, 1e-6, pos.cuda(), rot.cuda(), given.cuda(), interleaved)
    coli.sync_check()
    x = kv[:, :L].double()
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    ref = torch.cat([x, rotated(torch, kv[:, L:L + R], rot[pos.long()], interleaved)], 1)
    got = values(torch, c)
    live = [t for t in range(T) if T == 1 or t != skipped]
    amax = ref.abs().amax(1, keepdim=True)
    if e4m3:
        scale = c.scales.cpu().view(-1)[slots].double()
        assert ((scale - amax[:, 0] / 448).abs() <= 1e-6 * amax[:, 0])[live].all()
        tol = torch.maximum(2.0 ** -4 * ref.abs(), 2.0 ** -10 * amax / 448) * (1 + 1e-4) + 2e-6 * amax
    else:
        tol = U16 * ref.abs() * (1 + 1e-4) + 2e-6 * amax
    assert ((got[slots] - ref).abs() <= tol)[live].all()
    untouched = torch.ones(n_pages * page, dtype=torch.bool)
    untouched[slots[live]] = False
    assert torch.isnan(got[untouched]).all()


def test_append_special_rows():
    """A row of zeros (scale 0), a tiny one and a huge one; slots and positions out of range are reported and not written."""
    torch, coli = setup()
    c = new_cache(torch, coli, True, 128, 16, 16, 2)
    kv = torch.zeros(5, 144)
    kv[1] = 1e-30
    kv[2] = 1e30
    kv[3:] = 1.0
    slots = torch.tensor([0, 1, 2, 32, 5])
    pos = torch.tensor([0, 0, 0, 0, 8], dtype=torch.int32)
    coli.mla_append(c, kv.cuda(), None, 1.0, pos.cuda(), rotation(torch, 8, 16).cuda(), slots.cuda())
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_EINVAL
    got = values(torch, c)
    assert (got[0] == 0).all() and float(c.scales.view(-1)[0]) == 0.0
    assert torch.allclose(got[1], torch.full((144,), 1e-30, dtype=torch.float64), rtol=1e-5)
    assert torch.allclose(got[2], torch.full((144,), 1e30, dtype=torch.float64), rtol=1e-5)
    assert torch.isnan(got[3:]).all()


def filled(torch, coli, e4m3, L, R, page, lens, g, amplitude=1.0, spread=2.0, columns=0):
    """A cache with sequences of these lengths on shuffled pages (everything else NaN) and its page table
    (-1 past a sequence's pages)."""
    per = [-(-n // page) for n in lens]
    total = sum(per) + 2
    c = new_cache(torch, coli, e4m3, L, R, page, total)
    order = torch.randperm(total, generator=g)
    table = torch.full((len(lens), max(max(per), 1) + columns), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, :per[b]] = order[at:at + per[b]].to(torch.int32)
        at += per[b]
        if not n:
            continue
        t = torch.arange(n)
        slot = table[b, t // page].long() * page + t % page
        x = torch.randn(n, L + R, generator=g) * amplitude
        if e4m3:
            x *= spread ** (torch.rand(n, 1, generator=g) * 2 - 1)
            s = x.abs().amax(1) / 448
            c.scales.view(-1)[slot.cuda()] = s.cuda()
            codes = (x / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            c.rows.view(torch.uint8).view(-1, L + R)[slot.cuda()] = codes.view(torch.uint8).cuda()
        else:
            c.rows.view(-1, L + R)[slot.cuda()] = x.to(torch.bfloat16).cuda()
    return c, table


def sequence(torch, vals, table, b, n, page):
    t = torch.arange(n)
    return vals[table[b, t // page].long() * page + t % page]


@pytest.mark.parametrize("lens,page", [([1], 16), ([300, 0, 17, 64], 64), ([5, 1000, 33], 48), ([0, 0, 3], 16)])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("L,R", [(512, 64), (128, 48)])
def test_read(lens, page, e4m3, bf16, L, R):
    torch, coli = setup()
    c, table = filled(torch, coli, e4m3, L, R, page, lens, gen(torch, sum(lens)), columns=1)
    total = sum(lens)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    out = torch.full((total + 3, L + R + 8), 7.0, device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
    coli.mla_read(c, table.cuda(), cu.cuda(), out[:, :L + R])
    coli.sync_check()
    vals = values(torch, c)
    want = torch.cat([sequence(torch, vals, table, b, n, page) for b, n in enumerate(lens)]).float().to(out.dtype)
    assert torch.equal(out[:total, :L + R].cpu(), want)
    assert (out[total:] == 7).all() and (out[:, L + R:] == 7).all()


def test_read_bad_page():
    torch, coli = setup()
    c, table = filled(torch, coli, True, 128, 16, 16, [40, 20], gen(torch, 3))
    table[0, 1] = 99
    out = torch.ones(60, 144, device="cuda")
    coli.mla_read(c, table.cuda(), torch.tensor([0, 40, 60], dtype=torch.int32).cuda(), out)
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_EINVAL
    assert (out[16:32] == 0).all() and not (out[:16] == 0).all(1).any() and not (out[32:] == 0).all(1).any()


# ------------------------------------------------------------------ attend
def attend_case(torch, coli, e4m3, L, R, page, lens, n_q, H, seed, q_bf16=True, out_bf16=True, amplitude=1.0, q_scale=1.0, edit=None,
                columns=0, lse=True):
    """Runs coli.mla_attend and checks it against the definition in 64 bits."""
    g = gen(torch, seed)
    c, table = filled(torch, coli, e4m3, L, R, page, lens, g, amplitude, columns=columns)
    if edit is not None:
        edit(c, table)
    B = len(lens)
    qt = torch.bfloat16 if q_bf16 else torch.float32
    ql = (torch.randn(B, n_q, H, L, generator=g) * q_scale).to(qt)
    qr = (torch.randn(B, n_q, H, R, generator=g) * q_scale).to(qt)
    out = torch.full((B, n_q, H, L), float("nan"), device="cuda", dtype=torch.bfloat16 if out_bf16 else torch.float32)
    ls = torch.full((B, n_q, H), float("nan"), device="cuda") if lse else None
    scale = 1.0 / math.sqrt(128 + R)
    coli.mla_attend(c, ql.cuda(), qr.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale, out, ls)
    coli.sync_check()
    check_attend(torch, c, table, lens, page, ql, qr, scale, out, ls, q_bf16, out_bf16)
    return out


def check_attend(torch, c, table, lens, page, ql, qr, scale, out, ls, q_bf16=True, out_bf16=True):
    B, n_q, H, L = ql.shape
    r = UF16 if c.scales is not None else U16
    vals = values(torch, c)
    got = out.cpu().double()
    q = torch.cat([ql, qr], -1).double()
    for b in range(B):
        rows = sequence(torch, vals, table, b, lens[b], page)
        for j in range(n_q):
            n = lens[b] - (n_q - 1 - j)
            if n <= 0:
                assert (got[b, j] == 0).all(), (b, j)
                assert ls is None or (ls[b, j].cpu() == -math.inf).all()
                continue
            k = rows[:n]
            s = q[b, j] @ k.T * scale
            p = torch.softmax(s, -1)
            ref, size = p @ k[:, :L], p @ k[:, :L].abs()
            d = 0.0 if q_bf16 else r * scale * float((q[b, j].abs() @ k.abs().T).max())
            # the f32 score: 2^-21 of the sum of its terms' magnitudes at most
            d += 2.0 ** -21 * abs(scale) * float((q[b, j].abs() @ k.abs().T).max())
            rel = r + (math.exp(2 * d) - 1) + 1e-4
            tol = rel * size + (U16 if out_bf16 else 0) * ref.abs() + 1e-30
            err = (got[b, j] - ref).abs()
            assert (err <= tol).all(), (b, j, float((err / tol).max()))
            if ls is not None:
                want = torch.logsumexp(s, -1)
                assert ((ls[b, j].cpu().double() - want).abs() <= 1e-4 + d + 2e-6 * want.abs()).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H", [1, 3, 16, 20, 64, 128])
def test_attend_lengths(e4m3, H):
    """Lengths around pages, tiles and zero, in one ragged batch; NaN in everything that must not be read."""
    torch, coli = setup()
    attend_case(torch, coli, e4m3, 512, 64, 64, [0, 1, 15, 64, 127, 128, 129, 400, 2, 641], 1, H, 100 + H)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n_q,H", [(2, 16), (3, 20), (5, 7), (4, 128), (130, 3)])
def test_attend_several_queries(e4m3, n_q, H):
    """The newest tokens see one another causally; sequences shorter than n_q leave rows empty."""
    torch, coli = setup()
    attend_case(torch, coli, e4m3, 512, 64, 16, [n_q, 0, 1, 200, n_q + 127], n_q, H, 200 + n_q)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("L,R", [(128, 16), (256, 32), (384, 48), (512, 16), (128, 64)])
@pytest.mark.parametrize("page", [16, 48, 128, 1024])
def test_attend_dims_and_pages(e4m3, L, R, page):
    torch, coli = setup()
    attend_case(torch, coli, e4m3, L, R, page, [300, 7, 0, 131], 2, 17, L + R + page, columns=3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_bf16,out_bf16", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("H", [2, 40, 128])
def test_attend_types(e4m3, q_bf16, out_bf16, H):
    torch, coli = setup()
    attend_case(torch, coli, e4m3, 512, 64, 32, [500, 33, 1], 1, H, 300 + H, q_bf16, out_bf16, lse=H != 40)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,lens", [(128, [30000]), (16, [9000, 20000, 5]), (64, [129] * 200), (8, [40, 17000])])
def test_attend_long(e4m3, H, lens):
    """Work split over the tokens of long sequences, and more sequences than SMs."""
    torch, coli = setup()
    attend_case(torch, coli, e4m3, 512, 64, 64, lens, 1, H, 400 + H)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("q_scale", [30.0, 1e-3, 0.0])
def test_attend_score_ranges(e4m3, q_scale):
    """Scores of hundreds (the maximum keeps moving, one token takes all) and scores that are all alike."""
    torch, coli = setup()
    attend_case(torch, coli, e4m3, 512, 64, 64, [1500, 260], 1, 64, 500, amplitude=1.0, q_scale=q_scale)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("order", [1, -1])
def test_attend_moving_maximum(e4m3, order):
    """Rows that grow (or shrink) along the sequence: every tile raises the maximum by far, or none after the first."""
    torch, coli = setup()
    n, page, L, R, H = 2000, 64, 512, 64, 32
    g = gen(torch, 7)
    c, table = filled(torch, coli, e4m3, L, R, page, [n], g)
    t = torch.arange(n)
    slot = (table[0, t // page].long() * page + t % page).cuda()
    base = torch.randn(1, L + R, generator=g)
    x = base * torch.linspace(*((0.05, 1.0) if order > 0 else (1.0, 0.05)), n)[:, None] + 0.05 * torch.randn(n, L + R, generator=g)
    if e4m3:
        s = x.abs().amax(1) / 448
        c.scales.view(-1)[slot] = s.cuda()
        c.rows.view(torch.uint8).view(-1, L + R)[slot] = (x / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    else:
        c.rows.view(-1, L + R)[slot] = x.to(torch.bfloat16).cuda()
    q = (base.expand(H, -1) * torch.linspace(-3, 3, H)[:, None]).view(1, 1, H, L + R).to(torch.bfloat16)
    ql, qr = q[..., :L].contiguous(), q[..., L:].contiguous()
    out = torch.empty(1, 1, H, L, device="cuda")
    ls = torch.empty(1, 1, H, device="cuda")
    coli.mla_attend(c, ql.cuda(), qr.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda(), 0.07, out, ls)
    coli.sync_check()
    check_attend(torch, c, table, [n], page, ql, qr, 0.07, out, ls, True, False)


def test_attend_row_scales():
    """E4M3 rows with scales from 1e-9 to 1e3, and rows of scale 0 (value 0, score 0) among them."""
    torch, coli = setup()

    def edit(c, table):
        n = c.page_size * c.n_pages
        f = 10.0 ** torch.linspace(-7, 2, n)[torch.randperm(n, generator=gen(torch, 1))]
        f[::13] = 0.0
        c.scales.mul_(f.view(c.n_pages, c.page_size).cuda())
    attend_case(torch, coli, True, 512, 64, 16, [700, 90], 1, 24, 600, q_scale=0.02, edit=edit)
    attend_case(torch, coli, True, 512, 64, 16, [700, 90], 1, 24, 600, q_scale=0.02, edit=lambda c, t: c.scales.mul_(0.0))


def test_attend_repeats_bit_for_bit():
    torch, coli = setup()
    a = [attend_case(torch, coli, True, 512, 64, 64, [5000, 77, 3000], 1, 64, 700) for _ in range(2)]
    assert torch.equal(a[0].view(torch.int16), a[1].view(torch.int16))


def test_attend_bad_pages_and_lengths():
    torch, coli = setup()
    c, table = filled(torch, coli, False, 512, 64, 16, [100, 40], gen(torch, 3))
    q = torch.randn(2, 1, 16, 576, device="cuda").to(torch.bfloat16)
    ql, qr = q[..., :512].contiguous(), q[..., 512:].contiguous()
    out = torch.empty_like(ql)
    for lens, page in (([100, 41 + 16 * 7], None), ([-1, 40], None), ([100, 40], 1 << 20), ([100, 40], -1)):
        tb = table.clone()
        if page is not None:
            tb[0, 2] = page
        coli.mla_attend(c, ql, qr, tb.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.1, out)
        with pytest.raises(coli.ColiError) as e:
            coli.sync_check()
        assert e.value.code == coli.COLI_EINVAL
        coli.sync_check()


def test_attend_streams_and_graph():
    """On a side stream, and replayed from a CUDA graph with new contents and lengths."""
    torch, coli = setup()
    g = gen(torch, 11)
    lens = [900, 40]
    c, table = filled(torch, coli, True, 512, 64, 64, lens, g)
    ql, qr = torch.randn(2, 1, 64, 512, generator=g).to(torch.bfloat16), torch.randn(2, 1, 64, 64, generator=g).to(torch.bfloat16)
    qld, qrd, tb = ql.cuda(), qr.cuda(), table.cuda()
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    out, ls = torch.empty(2, 1, 64, 512, device="cuda"), torch.empty(2, 1, 64, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        coli.mla_attend(c, qld, qrd, tb, ln, 0.08, out, ls)
    st.synchronize()
    check_attend(torch, c, table, lens, 64, ql, qr, 0.08, out, ls, True, False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        coli.mla_attend(c, qld, qrd, tb, ln, 0.08, out, ls)
    for new in ([900, 40], [3, 33], [0, 1]):
        ln.copy_(torch.tensor(new, dtype=torch.int32))
        ql = torch.randn(2, 1, 64, 512, generator=g).to(torch.bfloat16)
        qld.copy_(ql)
        graph.replay()
        torch.cuda.synchronize()
        check_attend(torch, c, table, new, 64, ql, qr, 0.08, out, ls, True, False)


# ------------------------------------------------------------------ prefill
def prefill_case(torch, coli, n_qs, n_ks, H, N, R, V, seed, f32_in=False, out_bf16=True, q_scale=1.0, junk=True, lse=True):
    g = gen(torch, seed)
    Tq, Tk = sum(n_qs), sum(n_ks)
    dt = torch.float32 if f32_in else torch.bfloat16
    q = (torch.randn(Tq, H, N + R, generator=g) * q_scale).to(dt)
    kv = torch.randn(Tk, H, N + V, generator=g).to(dt)
    wide = torch.randn(Tk, R + 24, generator=g).to(dt)       # k_rope as part of wider rows
    cq = [0] + [int(v) for v in np.cumsum(n_qs)]
    ck = [0] + [int(v) for v in np.cumsum(n_ks)]
    out = torch.full((Tq, H, V), float("nan"), device="cuda", dtype=torch.bfloat16 if out_bf16 else torch.float32)
    ls = torch.full((Tq, H), float("nan"), device="cuda") if lse else None
    scale = 1.0 / math.sqrt(N + R)
    coli.mla_prefill(q.cuda(), kv.cuda(), wide.cuda()[:, 8:8 + R], torch.tensor(cq, dtype=torch.int32).cuda(),
                     torch.tensor(ck, dtype=torch.int32).cuda(), scale, out, ls)
    coli.sync_check()
    k_rope = wide[:, 8:8 + R]
    got = out.cpu().double()
    for b in range(len(n_qs)):
        n, m = n_qs[b], n_ks[b]
        seen = torch.arange(m)[None, :] <= torch.arange(n)[:, None] + m - n
        for h in range(H):
            qq = q[cq[b]:cq[b + 1], h].double()
            kk = torch.cat([kv[ck[b]:ck[b + 1], h, :N], k_rope[ck[b]:ck[b + 1]]], 1).double()
            vv = kv[ck[b]:ck[b + 1], h, N:].double()
            s = (qq @ kk.T * scale).masked_fill(~seen, -math.inf)
            lz = torch.logsumexp(s, -1) if m else torch.full((n,), -math.inf, dtype=torch.float64)
            empty = lz == -math.inf
            p = torch.exp(s - lz.masked_fill(empty, 0.0)[:, None])
            ref, size = p @ vv, p @ vv.abs()
            mags = float((qq.abs() @ kk.abs().T).max()) if n and m else 0.0
            # f32 inputs: q, k and v are rounded to bf16 first
            d = (2 * U16 if f32_in else 0.0) * scale * mags + 2.0 ** -21 * scale * mags
            rel = U16 + (U16 if f32_in else 0.0) + (math.exp(2 * d) - 1) + 1e-4
            tol = rel * size + (U16 if out_bf16 else 0.0) * ref.abs() + 1e-30
            o = got[cq[b]:cq[b + 1], h]
            assert (o[empty] == 0).all()
            err = (o - ref).abs()
            assert (err <= tol).all(), (b, h, float((err / tol).max()))
            if lse:
                got_l = ls[cq[b]:cq[b + 1], h].cpu().double()
                assert (got_l[empty] == -math.inf).all()
                assert ((got_l - lz)[~empty].abs() <= 1e-4 + d + 2e-6 * lz[~empty].abs()).all()
    return out


@pytest.mark.parametrize("n_qs,n_ks", [([1], [1]), ([128], [128]), ([300], [300]), ([5, 0, 257, 1, 129], [5, 0, 257, 1, 129]),
                                       ([7, 130, 1], [100, 400, 256]), ([200, 10], [50, 0]), ([513], [700])])
@pytest.mark.parametrize("H", [1, 3])
def test_prefill_lengths(n_qs, n_ks, H):
    """Ragged sequences, cached prefixes, queries that see no key (more queries than keys)."""
    torch, coli = setup()
    prefill_case(torch, coli, n_qs, n_ks, H, 128, 64, 128, sum(n_qs) + sum(n_ks) + H)


@pytest.mark.parametrize("N,R,V", [(128, 64, 64), (64, 64, 128), (64, 16, 64), (128, 48, 128), (64, 32, 128)])
def test_prefill_dims(N, R, V):
    torch, coli = setup()
    prefill_case(torch, coli, [140, 33], [140, 290], 4, N, R, V, N + R + V)


@pytest.mark.parametrize("f32_in,out_bf16", [(True, False), (True, True), (False, False)])
def test_prefill_types(f32_in, out_bf16):
    torch, coli = setup()
    prefill_case(torch, coli, [200, 9], [230, 9], 5, 128, 64, 128, 31, f32_in, out_bf16, lse=out_bf16)


@pytest.mark.parametrize("q_scale", [30.0, 0.0])
def test_prefill_score_ranges(q_scale):
    torch, coli = setup()
    prefill_case(torch, coli, [600], [900], 2, 128, 64, 128, 32, q_scale=q_scale)


def test_prefill_long():
    torch, coli = setup()
    prefill_case(torch, coli, [2500, 1100], [2500, 1500], 2, 128, 64, 128, 33)


@pytest.mark.parametrize("N,R,V", [(128, 64, 128), (64, 32, 64), (128, 64, 64)])
def test_prefill_many_units(N, R, V):
    """Several units of work per SM, of every mix of sizes, from more sequences than a warp has lanes; equal calls give equal bits."""
    torch, coli = setup()
    r = random.Random(7)
    n_qs = [r.choice((0, 1, 100, 128, 129, 256, 257, 300, 513)) for _ in range(70)]
    n_ks = [max(0, n + r.choice((-200, -1, 0, 0, 1, 127, 128, 300))) for n in n_qs]
    one = prefill_case(torch, coli, n_qs, n_ks, 8, N, R, V, 34)
    two = prefill_case(torch, coli, n_qs, n_ks, 8, N, R, V, 34)
    assert torch.equal(one, two)


def test_prefill_isolates_sequences():
    """Infinities and NaN in one sequence stay there, whichever rows share a tile with its neighbours'."""
    torch, coli = setup()
    g = gen(torch, 40)
    n, H = [60, 45, 70], 2
    cu = torch.tensor([0, 60, 105, 175], dtype=torch.int32).cuda()
    q = torch.randn(175, H, 192, generator=g).to(torch.bfloat16)
    kv = torch.randn(175, H, 256, generator=g).to(torch.bfloat16)
    kr = torch.randn(175, 64, generator=g).to(torch.bfloat16)
    outs = []
    for poison in (False, True):
        k2, r2, q2 = kv.clone(), kr.clone(), q.clone()
        if poison:
            k2[60:105] = float("nan")
            k2[80:90] = float("inf")
            r2[60:105] = float("inf")
            q2[60:105] = float("nan")
        out = torch.empty(175, H, 128, device="cuda", dtype=torch.bfloat16)
        coli.mla_prefill(q2.cuda(), k2.cuda(), r2.cuda(), cu, cu, 0.07, out)
        coli.sync_check()
        outs.append(out.cpu())
    for s in (slice(0, 60), slice(105, 175)):
        assert torch.equal(outs[0][s], outs[1][s])


def test_prefill_bad_offsets():
    torch, coli = setup()
    q = torch.randn(20, 2, 192, device="cuda").to(torch.bfloat16)
    kv = torch.randn(20, 2, 256, device="cuda").to(torch.bfloat16)
    kr = torch.randn(20, 64, device="cuda").to(torch.bfloat16)
    out = torch.empty(20, 2, 128, device="cuda", dtype=torch.bfloat16)
    good = [0, 10, 20]
    for cq, ck in ((good, [0, 10, 21]), (good, [0, -5, 20]), (good, [0, 25, 20])):
        coli.mla_prefill(q, kv, kr, torch.tensor(cq, dtype=torch.int32).cuda(), torch.tensor(ck, dtype=torch.int32).cuda(), 0.1, out)
        with pytest.raises(coli.ColiError) as e:
            coli.sync_check()
        assert e.value.code == coli.COLI_EINVAL
        coli.sync_check()


# ------------------------------------------------------------------ the binding
def test_binding_refusals():
    """Tensors of other shapes, types or layouts are refused before the library sees them."""
    torch, coli = setup()
    c = new_cache(torch, coli, True, 512, 64, 64, 3)
    q = torch.zeros(2, 4, 192, device="cuda")
    rot = rotation(torch, 8, 64).cuda()
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    on, orr = torch.zeros(2, 4, 128, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    ql, qr = torch.zeros(2, 1, 4, 512, device="cuda", dtype=torch.bfloat16), torch.zeros(2, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    pages, lens = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    for f in (lambda: coli.MlaCache(c.rows, 448, 64, c.scales), lambda: coli.MlaCache(c.rows, 512, 64),
              lambda: coli.MlaCache(c.rows[:, ::2], 512, 64, c.scales[:, ::2]), lambda: coli.MlaCache(c.rows.float(), 512, 64, c.scales),
              lambda: coli.mla_query(q, pos.long(), rot, on, orr), lambda: coli.mla_query(q, pos, rot[:, :32], on, orr),
              lambda: coli.mla_query(q, pos, rot, on.transpose(0, 1).contiguous(), orr), lambda: coli.mla_query(q.half(), pos, rot, on, orr),
              lambda: coli.mla_append(c, torch.zeros(2, 575, device="cuda"), None, 1.0, pos, rot, pos.long()),
              lambda: coli.mla_append(c, torch.zeros(2, 576, device="cuda"), None, 1.0, pos, rot, pos),
              lambda: coli.mla_read(c, pages, lens, torch.zeros(2, 512, device="cuda")),
              lambda: coli.mla_attend(c, ql.transpose(2, 3), qr, pages, lens, 1.0, ql), lambda: coli.mla_attend(c, ql, qr.float(), pages, lens, 1.0, ql),
              lambda: coli.mla_attend(c, ql, qr, pages.t(), lens, 1.0, ql), lambda: coli.mla_attend(c, ql, qr, pages, lens[:1], 1.0, ql),
              lambda: coli.mla_prefill(q, torch.zeros(2, 4, 256, device="cuda"), orr[:, 0], pos, lens[:1], 1.0, on)):
        with pytest.raises(coli.ColiError):
            f()
