"""Grouped-head attention on the GPU against plain 64-bit computations of the definitions: the 4-bit cache's write and read
back, attention of prompts and over the cache, the rows' weights, the eviction.

Tolerances.  Codes, scales, kept tokens and moved rows are exact.  An attention output is sum_t p_t v_t.  Prompts: rounding
every p_t to bf16 moves it by at most 2^-8 sum_t p_t |v_t|, to f16 (f32 inputs) by 2^-11 of that.  Over the cache p_t is rounded to bf16 and its product with the
row's scale once more, (1 + 2^-8)^2 - 1 = 2^-7 + 2^-16 in all, and sum_t p_t s_t (128 + n_t) - 136 sum_t p_t s_t is added up in f32: each of at most len / 16 + 8 additions
may be off by 2^-23 of 136 max_t s_t.  f32 scores, exp and sums move the p_t by less than 1e-4 of themselves for these
lengths, and a bf16 output rounds once more (2^-8).  An f32 query becomes f16 (2^-11 of each element), which moves a score by at
most d = 2^-11 scale sum_i |q_i| |k_ti| and p_t by a factor exp(2 d)."""
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


# ------------------------------------------------------------------ cache
class Store:
    """A cache of random codes whose scales are NaN, and weights -7, until they are written; host mirror by `rows`."""

    def __init__(self, torch, coli, n_pages, kv, page, dim, gs, g, weights=True):
        self.torch = torch
        self.k, self.v = (torch.randint(0, 256, (n_pages, kv, page, dim // 2), generator=g, dtype=torch.uint8).cuda() for _ in "kv")
        self.ks, self.vs = (torch.full((n_pages, kv, page, dim // gs), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        self.w = torch.full((n_pages, kv, page), -7.0, device="cuda") if weights else None
        self.c = coli.GqaCache(self.k, self.v, self.ks, self.vs, weights=self.w)
        self.page, self.kv, self.dim, self.gs, self.n_pages = page, kv, dim, gs, n_pages

    def rows(self, which, ids, n):
        """The first n rows of pages ids as values in 64 bits, [kv, n, dim]."""
        torch = self.torch
        ids = [int(i) for i in ids]
        b = getattr(self, which).cpu()[ids].int()
        x = torch.stack([b & 15, b >> 4], -1).flatten(-2).double() - 8
        s = getattr(self, which + "s").cpu()[ids].double()
        x = (x.unflatten(-1, (s.shape[-1], self.gs)) * s[..., None]).flatten(-2)
        return x.transpose(0, 1).flatten(1, 2)[:, :n]


def tables(torch, lens, page, g, spare=0, columns=0):
    """Page tables on shuffled pages (-1 past a sequence's pages), and spare page ids."""
    per = [-(-n // page) for n in lens]
    total = sum(per) + 2 + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(per + [1]) + columns), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:at + spare], total


def filled(torch, coli, lens, kv, page, dim, gs, g, spare=0, columns=0, weights=True, spread=3.0):
    """A store that holds sequences of these lengths, scales of random size, everything else as Store leaves it."""
    table, more, total = tables(torch, lens, page, g, spare, columns)
    s = Store(torch, coli, total, kv, page, dim, gs, g, weights)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            m = min(page, n - i * page)
            for t in (s.ks, s.vs):
                t[int(table[b, i]), :, :m] = (0.3 * spread ** (torch.rand(kv, m, dim // gs, generator=g) * 2 - 1)).to(torch.bfloat16).cuda()
            if s.w is not None:
                s.w[int(table[b, i]), :, :m] = torch.rand(kv, m, generator=g).cuda()
    return s, table, more


def quantised(x, gs):
    """Codes and scales (as f32) of f32 rows x [..., dim], by the definition in f32."""
    x = x.reshape(*x.shape[:-1], -1, gs)
    amax = np.abs(x).max(-1)
    fine = np.isfinite(x).all(-1)
    import torch
    with np.errstate(all="ignore"):
        scale = torch.from_numpy((np.where(fine, amax, np.nan) / np.float32(7)).astype(np.float32)).to(torch.bfloat16).float().numpy()
        by = np.where(scale > 0, scale, np.float32(1)).astype(np.float32)
        code = np.clip(np.rint(x / by[..., None]), -8, 7) + 8
    code = np.where(fine[..., None], code, 8).astype(np.uint8)
    code = code.reshape(*code.shape[:-2], -1)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


@pytest.mark.parametrize("T,kv,dim,gs,page", [(1, 8, 128, 32, 64), (8, 8, 128, 128, 16), (133, 3, 128, 64, 48), (50, 1, 64, 32, 32), (21, 5, 64, 64, 16)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_append(T, kv, dim, gs, page, kind):
    torch, coli = setup()
    g = gen(torch, T + kv + dim + gs)
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    rows = (torch.randn(T, 2 * kv + 1, dim, generator=g) * (10.0 ** (torch.rand(T, 2 * kv + 1, 1, generator=g) * 8 - 4))).to(dtype)
    rows[0, 0, :gs] = 0.0                                                 # a group of zeros
    if T > 1:
        rows[1, 0, 3] = float("nan")
        rows[1, kv, dim - 1] = float("-inf")
    n_pages = -(-T // page) + 2
    s = Store(torch, coli, n_pages, kv, page, dim, gs, g)
    before = s.k.cpu().clone(), s.v.cpu().clone()
    slots = torch.randperm(n_pages * page, generator=g)[:T]
    given = slots.clone()
    skipped = T // 2 if T > 1 else -1
    if T > 1:
        given[skipped] = -1
    dev = rows.cuda()
    coli.gqa_append(s.c, dev[:, :kv], dev[:, kv:2 * kv], given.cuda())    # parts of one row, tokens with padding
    coli.sync_check()
    k, v, ks, vs, w = s.k.cpu(), s.v.cpu(), s.ks.float().cpu().numpy(), s.vs.float().cpu().numpy(), s.w.cpu()
    written = torch.zeros(n_pages, page, dtype=torch.bool)
    for t in range(T):
        if t == skipped:
            continue
        p, o = divmod(int(slots[t]), page)
        written[p, o] = True
        for got, scales, x in ((k, ks, rows[t, :kv]), (v, vs, rows[t, kv:2 * kv])):
            code, scale = quantised(x.float().numpy(), gs)
            assert (got[p, :, o].numpy() == code).all()
            np.testing.assert_array_equal(scales[p, :, o], scale)
        assert (w[p, :, o] == 0).all()
    keep = ~written
    assert torch.equal(k.transpose(1, 2)[keep], before[0].transpose(1, 2)[keep])
    assert torch.equal(v.transpose(1, 2)[keep], before[1].transpose(1, 2)[keep])
    assert np.isnan(ks.swapaxes(1, 2)[keep.numpy()]).all() and (w.transpose(1, 2)[keep] == -7).all()


def test_append_special_rows():
    """Magnitudes whose scale vanishes or is the largest; slots out of range are reported and not written."""
    torch, coli = setup()
    s = Store(torch, coli, 2, 1, 16, 64, 32, gen(torch, 0))
    x = torch.zeros(5, 1, 64)
    x[0] = 1e-44
    x[1] = 3e38
    x[2, 0, ::2] = -1e-30
    x[3:] = 1.0
    slots = torch.tensor([0, 1, 2, 32, -2])
    k0 = s.k.cpu().clone()
    coli.gqa_append(s.c, x.cuda(), x.cuda(), slots.cuda())
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_EINVAL
    for t in range(3):
        code, scale = quantised(x[t].numpy(), 32)
        assert (s.k.cpu()[0, :, t].numpy() == code).all()
        np.testing.assert_array_equal(s.ks.float().cpu()[0, :, t].numpy(), scale)
    assert torch.equal(s.k.cpu()[0, :, 3:], k0[0, :, 3:]) and torch.equal(s.k.cpu()[1], k0[1])
    coli.sync_check()


@pytest.mark.parametrize("lens,kv,dim,gs,page", [([1], 8, 128, 32, 64), ([0, 33, 7, 0, 100], 3, 128, 64, 16), ([47, 1], 1, 64, 64, 48), ([200], 2, 64, 32, 32)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_read(lens, kv, dim, gs, page, kind):
    torch, coli = setup()
    g = gen(torch, sum(lens) + kv)
    s, table, _ = filled(torch, coli, lens, kv, page, dim, gs, g, columns=1)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, dtype = int(cu[-1]), torch.float32 if kind == "f32" else torch.bfloat16
    out = torch.full((T + 3, 2 * kv + 1, dim), -3.0, device="cuda", dtype=dtype)
    coli.gqa_read(s.c, table.cuda(), torch.from_numpy(cu).cuda(), out[:, :kv], out[:, kv:2 * kv])
    coli.sync_check()
    got = out.cpu()
    for b, n in enumerate(lens):
        for which, part in (("k", got[:, :kv]), ("v", got[:, kv:2 * kv])):
            ref = s.rows(which, table[b, : -(-n // page)], n).transpose(0, 1)
            assert torch.equal(part[cu[b]:cu[b + 1]], ref.to(dtype))
    assert (got[T:] == -3).all() and (got[:, 2 * kv] == -3).all()


def test_read_bad_pages():
    """A page id out of range and a sequence longer than its list: rows of zeros, reported."""
    torch, coli = setup()
    g = gen(torch, 5)
    s, table, _ = filled(torch, coli, [40], 2, 16, 64, 32, g)
    for bad in (-1, s.n_pages):
        t = table.clone()
        t[0, 1] = bad
        k, v = (torch.ones(50, 2, 64, device="cuda") for _ in "kv")
        coli.gqa_read(s.c, t.cuda(), torch.tensor([0, 50], dtype=torch.int32, device="cuda"), k, v)
        with pytest.raises(coli.ColiError) as e:
            coli.sync_check()
        assert e.value.code == coli.COLI_EINVAL
        assert (k[16:32] == 0).all() and (v[48:] == 0).all()
        assert torch.equal(k[:16].cpu().double(), s.rows("k", table[0, :1], 16).transpose(0, 1))


# ------------------------------------------------------------------ prompts
def reference_prompt(torch, q, k, v, cu_q, cu_k, scale, kind):
    """Outputs, tolerances and lse in 64 bits; q, k, v as they are (bf16) or rounded to f16 (f32 inputs; a power of two that goes
    with them changes no bit of values above 2^-14, and below they are off by 2^-25)."""
    Tq, H, D = q.shape
    group = H // k.shape[1]
    u = UF16 if q.dtype is torch.float32 else U16
    q, k, v = ((x.to(torch.float16) if x.dtype is torch.float32 else x).double() for x in (q, k, v))
    out, tol = torch.zeros(Tq, H, D, dtype=torch.float64), torch.zeros(Tq, H, D, dtype=torch.float64)
    lse = torch.full((Tq, H), -math.inf, dtype=torch.float64)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = q1 - q0, k1 - k0
        if n == 0 or m == 0:
            continue
        seen = torch.arange(m)[None, :] <= torch.arange(n)[:, None] + m - n
        for h in range(H):
            a = (q[q0:q1, h] @ k[k0:k1, h // group].T * scale).masked_fill(~seen, -math.inf)
            some = seen.any(-1)
            p = torch.zeros_like(a)
            p[some] = torch.softmax(a[some], -1)
            out[q0:q1, h] = p @ v[k0:k1, h // group]
            tol[q0:q1, h] = (u + 1e-4) * (p @ v[k0:k1, h // group].abs())
            lse[q0:q1, h] = torch.logsumexp(a, -1)
    if kind == "bf16":
        tol += U16 * out.abs()
    return out, tol * (1 + 1e-3) + 1e-6, lse


def packed_qkv(torch, lens_q, lens_k, H, K, D, g, dtype, amplitude=1.0):
    """q, and k and v as parts of one row with padding, on the host."""
    q = (torch.randn(sum(lens_q), H, D, generator=g) * amplitude).to(dtype)
    kv = torch.randn(sum(lens_k), 2 * K + 1, D, generator=g).to(dtype)
    return q, kv


PROMPTS = [
    ([1], [1], 8, 8, 128), ([1], [300], 32, 8, 128), ([5, 0, 1, 33], [5, 7, 1, 40], 28, 4, 128), ([300], [300], 5, 1, 64),
    ([130, 257], [259, 257], 16, 2, 128), ([64, 31], [20, 0], 6, 3, 128), ([40], [40], 33, 1, 64), ([17, 300, 2], [17, 300, 200], 48, 3, 128),
    ([3], [700], 128, 1, 128), ([600], [600], 4, 4, 64)]


@pytest.mark.parametrize("lens_q,lens_k,H,K,D", PROMPTS)
@pytest.mark.parametrize("kind_in,kind_out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
def test_prompt(lens_q, lens_k, H, K, D, kind_in, kind_out):
    torch, coli = setup()
    g = gen(torch, sum(lens_q) + H + K)
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    q, kv = packed_qkv(torch, lens_q, lens_k, H, K, D, g, types[kind_in], 1.5)
    cu_q, cu_k = ([0] + list(np.cumsum(x)) for x in (lens_q, lens_k))
    Tq = cu_q[-1]
    out = torch.full((Tq + 2, H, D), -5.0, device="cuda", dtype=types[kind_out])
    lse = torch.full((Tq, H), -5.0, device="cuda")
    scale = 1.0 / math.sqrt(D)
    dev = kv.cuda()
    coli.gqa_prefill(q.cuda(), dev[:, :K], dev[:, K:2 * K], torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                     torch.tensor(cu_k, dtype=torch.int32, device="cuda"), scale, out[:Tq], lse)
    coli.sync_check()
    ref, tol, ref_lse = reference_prompt(torch, q, kv[:, :K], kv[:, K:2 * K], cu_q, cu_k, scale, kind_out)
    assert ((out[:Tq].cpu().double() - ref).abs() <= tol).all()
    assert (out[Tq:] == -5).all()
    got = lse.cpu().double()
    none = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(got), none)
    assert ((got - ref_lse)[~none].abs() <= 1e-4 * (1 + ref_lse[~none].abs())).all()


@pytest.mark.parametrize("size_q,size_k,size_v", [(1e-30, 1e20, 1.0), (1e25, 1e-25, 1e30), (1.0, 1.0, 1e-30), (1e-5, 1e-5, 1e-5)])
def test_prompt_f32_magnitudes(size_q, size_k, size_v):
    """f32 inputs of any size: the powers of two that come with f16 leave every score and output in its place."""
    torch, coli = setup()
    g = gen(torch, 8)
    q, kv = packed_qkv(torch, [70], [90], 4, 2, 64, g, torch.float32)
    q[::3] *= 2.0 ** -20                                  # each row of q has a power of its own
    scale = 0.125 / size_q / size_k
    out = torch.empty(70, 4, 64, device="cuda")
    cu = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (70, 90)]
    coli.gqa_prefill((q * size_q).cuda(), (kv[:, :2] * size_k).contiguous().cuda(), (kv[:, 2:4] * size_v).contiguous().cuda(), *cu, scale, out)
    coli.sync_check()
    q[::3] *= 2.0 ** 20                                   # the reference rounds to f16 where all rows are in range: a row's
    ref, tol, _ = reference_prompt(torch, q, kv[:, :2], kv[:, 2:4], [0, 70], [0, 90], 0.125, "f32")
    small, small_tol, _ = reference_prompt(torch, q, kv[:, :2], kv[:, 2:4], [0, 70], [0, 90], 0.125 * 2.0 ** -20, "f32")
    ref[::3], tol[::3] = small[::3], small_tol[::3]
    # q * size_q, k * size_k and v * size_v are f32 products: off by 2^-24 before the kernel sees them, and may round the other way
    # to f16: one more 2^-11 of each q and k in the scores (|s| <= 12, 2 x 2^-11 x 12), of each v in the output
    some = ref.abs() * 0 + kv[:, 2:4].abs().max().double()
    assert ((out.cpu().double() / size_v - ref).abs() <= tol + (UF16 + 4 * UF16 * 12) * some).all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_prompt_scales(scale):
    torch, coli = setup()
    g = gen(torch, 9)
    q, kv = packed_qkv(torch, [200], [260], 6, 2, 128, g, torch.bfloat16)
    out = torch.empty(200, 6, 128, device="cuda")
    dev = kv.cuda()
    cu = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (200, 260)]
    coli.gqa_prefill(q.cuda(), dev[:, :2], dev[:, 2:4], *cu, scale, out)
    ref, tol, _ = reference_prompt(torch, q, kv[:, :2], kv[:, 2:4], [0, 200], [0, 260], scale, "f32")
    # scores of up to 30 x scale units, off by 2^-20 of themselves
    assert ((out.cpu().double() - ref).abs() <= tol * (1 + 3 * abs(scale))).all()


def test_prompt_strangers_do_not_matter():
    """NaN and infinities in other sequences' rows, between and behind them, change no bit; outputs of no sequence stay."""
    torch, coli = setup()
    g = gen(torch, 11)
    q, kv = packed_qkv(torch, [100, 60, 70], [100, 60, 70], 8, 2, 128, g, torch.bfloat16)
    cu = torch.tensor([0, 100, 160], dtype=torch.int32, device="cuda")   # two sequences; the third's rows are no one's

    def run(q, kv):
        out = torch.full((230, 8, 128), 7.0, device="cuda", dtype=torch.bfloat16)
        d = kv.cuda()
        coli.gqa_prefill(q.cuda(), d[:, :2], d[:, 2:4], cu, cu, 0.09, out)
        coli.sync_check()
        return out.cpu()

    want = run(q, kv)
    assert (want[160:] == 7).all()
    for junk in (float("nan"), float("inf"), -float("inf")):
        q2, kv2 = q.clone(), kv.clone()
        q2[160:], kv2[160:] = junk, junk
        assert torch.equal(run(q2, kv2), want)
        q2[100:160], kv2[100:160] = junk, junk
        assert torch.equal(run(q2, kv2)[:100], want[:100])


def test_prompt_nan_rows():
    """A NaN in a query or in a key that a query sees makes that row NaN and leaves the rows that do not see it alone."""
    torch, coli = setup()
    g = gen(torch, 12)
    q, kv = packed_qkv(torch, [150], [150], 4, 2, 64, g, torch.bfloat16)
    cu = torch.tensor([0, 150], dtype=torch.int32, device="cuda")

    def run(q, kv):
        out = torch.empty(150, 4, 64, device="cuda")
        d = kv.cuda()
        coli.gqa_prefill(q.cuda(), d[:, :2], d[:, 2:4], cu, cu, 0.12, out)
        return out.cpu()

    want = run(q, kv)
    q2 = q.clone()
    q2[77, 3, 5] = float("nan")
    got = run(q2, kv)
    assert torch.isnan(got[77, 3]).all()
    got[77, 3] = want[77, 3]
    assert torch.equal(got, want)
    kv2 = kv.clone()
    kv2[90, 1, 3] = float("nan")             # key of head 1: query heads 2 and 3 from row 90 on
    got = run(q, kv2)
    assert torch.equal(got[:90], want[:90]) and torch.equal(got[:, :2], want[:, :2]) and torch.isnan(got[90:, 2:]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("lens_q,lens_k,H,K,D", [([150, 40], [150, 90], 4, 2, 64), ([70], [300], 14, 2, 128), ([300], [300], 2, 2, 128)])
def test_prompt_masked_values(lens_q, lens_k, H, K, D, kind):
    """Values that are not finite reach the rows that see them and no others: infinities keep their sign, and where a row sees
    infinities of both signs or a NaN it is NaN."""
    torch, coli = setup()
    g = gen(torch, H + D)
    dtype = torch.bfloat16 if kind == "bf16" else torch.float32
    q, kv = packed_qkv(torch, lens_q, lens_k, H, K, D, g, dtype)
    cu_q, cu_k = ([0] + [int(x) for x in np.cumsum(v)] for v in (lens_q, lens_k))
    bad = {}                                              # (key, head, column): value
    for b in range(len(lens_k)):
        n = lens_k[b]
        for back, col, x in ((1, 0, "nan"), (3, 1, "inf"), (3, 5, "-inf"), (9, 5, "inf"), (9, 40, "nan"), (20, 41, "inf"), (33, D - 1, "-inf")):
            if back <= n:
                bad[(cu_k[b] + n - back, b % K, col)] = float(x)
    dirty = kv.clone()
    for (t, h, col), x in bad.items():
        dirty[t, K + h, col] = x

    def run(kv):
        out = torch.empty(cu_q[-1], H, D, device="cuda", dtype=torch.float32)
        d = kv.cuda()
        coli.gqa_prefill(q.cuda(), d[:, :K], d[:, K:2 * K], torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                         torch.tensor(cu_k, dtype=torch.int32, device="cuda"), 0.09, out)
        coli.sync_check()
        return out.cpu().double()

    got = run(dirty)
    # what a row sees: finite values as they are, then the others added
    clean = kv.clone()
    for (t, h, col), x in bad.items():
        clean[t, K + h, col] = 0.0
    ref, tol, _ = reference_prompt(torch, q, clean[:, :K], clean[:, K:2 * K], cu_q, cu_k, 0.09, "f32")
    for b in range(len(lens_q)):
        for i in range(lens_q[b]):
            seen = cu_k[b] + i + lens_k[b] - lens_q[b]
            for (t, h, col), x in bad.items():
                if cu_k[b] <= t <= seen:
                    ref[cu_q[b] + i, h * H // K:(h + 1) * H // K, col] += x
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fine)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)])
    assert ((got - ref).abs()[fine] <= tol[fine]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_prompt_rows_without_keys_beside_infinite_values(kind):
    """More queries than keys, and values that are not finite: the first queries, which share a tile with some that see
    those, give zeros."""
    torch, coli = setup()
    g = gen(torch, 21)
    q, kv = packed_qkv(torch, [100, 9], [70, 3], 4, 2, 64, g, torch.bfloat16 if kind == "bf16" else torch.float32)
    kv[0, 2, 3] = kv[70, 3, 5] = float("nan")
    kv[1, 3, 7], kv[69, 2, 9], kv[72, 2, 0] = float("inf"), float("-inf"), float("inf")
    out, lse = torch.full((109, 4, 64), -5.0, device="cuda"), torch.full((109, 4), -5.0, device="cuda")
    dev = kv.cuda()
    coli.gqa_prefill(q.cuda(), dev[:, :2], dev[:, 2:4], torch.tensor([0, 100, 109], dtype=torch.int32, device="cuda"),
                     torch.tensor([0, 70, 73], dtype=torch.int32, device="cuda"), 0.12, out, lse)
    coli.sync_check()
    for first, last in ((0, 30), (100, 106)):
        assert (out[first:last] == 0).all() and (lse[first:last] == -math.inf).all()
    assert torch.isnan(out[30:100, :2, 3]).all() and torch.isnan(out[106:, 2:, 5]).all()
    assert torch.isfinite(out[30:100, :2, 10:]).all() and torch.isfinite(lse[30:100]).all()


def test_prompt_bad_offsets():
    torch, coli = setup()
    q, k = torch.zeros(10, 2, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(10, 1, 64, device="cuda", dtype=torch.bfloat16)
    for cu in ([0, 11], [0, -1], [3, 1], [-2, 5]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        coli.gqa_prefill(q, k, k, cu, cu, 1.0, torch.empty_like(q))
        with pytest.raises(coli.ColiError) as e:
            coli.sync_check()
        assert e.value.code == coli.COLI_EINVAL
    coli.sync_check()


# ------------------------------------------------------------------ steps
def reference_step(torch, s, table, lens, q, scale, kind_q, kind_out):
    """Outputs, their tolerances, lse, weights of rows [b][kv, len] and their tolerances, in 64 bits."""
    B, nq, H, D = q.shape
    group = H // s.kv
    x = q.double()
    out, tol = torch.zeros(B, nq, H, D, dtype=torch.float64), torch.zeros(B, nq, H, D, dtype=torch.float64)
    lse = torch.full((B, nq, H), -math.inf, dtype=torch.float64)
    weights, w_tol = [], []
    for b, n in enumerate(lens):
        ids = table[b, : -(-n // s.page)]
        k, v = s.rows("k", ids, n), s.rows("v", ids, n)
        vs = s.vs.cpu()[[int(i) for i in ids]].double() if n else torch.zeros(1)
        vs = vs.transpose(0, 1).flatten(1, 2)[:, :n] if n else vs
        got, off = torch.zeros(s.kv, n, dtype=torch.float64), torch.zeros(s.kv, n, dtype=torch.float64)
        for j in range(nq):
            m = n - (nq - 1 - j)
            if m <= 0:
                continue
            for h in range(H):
                kh = h // group
                a = k[kh, :m] @ x[b, j, h] * scale
                p = torch.softmax(a, -1)
                d = (k[kh, :m].abs() @ x[b, j, h].abs()).max() * abs(scale)    # no score is larger, nor its terms together
                r = math.expm1(2 * UF16 * d) if kind_q == "f32" else 0.0
                out[b, j, h] = p @ v[kh, :m]
                tol[b, j, h] = (2 * U16 + U16 * U16 + 1e-4 + r) * (p @ v[kh, :m].abs()) + r * out[b, j, h].abs() + (n / 16 + 8) * 2.0 ** -23 * 136 * vs[kh, :m].max()
                lse[b, j, h] = torch.logsumexp(a, -1)
                got[kh, :m] += p
                # scores: f32 sums of codes 0..15 (2 d at most) in some 20 additions; x and m in units of log2; exp; 1 / l
                off[kh, :m] += p * (r + 2.0 ** -19 + 64 * 2.0 ** -23 * d)
        weights.append(got)
        w_tol.append(off)
    if kind_out == "bf16":
        tol += U16 * out.abs()
    return out, tol * (1 + 1e-3) + 1e-6, lse, weights, w_tol


def run_step(torch, coli, s, table, lens, q, scale, kind_out, weigh=False, with_lse=True):
    out = torch.full(q.shape, -5.0, device="cuda", dtype=torch.bfloat16 if kind_out == "bf16" else torch.float32)
    lse = torch.full(q.shape[:3], -5.0, device="cuda") if with_lse else None
    coli.gqa_attend(s.c, q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), scale, out, lse, weigh=weigh)
    coli.sync_check()
    return out, lse


STEPS = [
    ([1], 1, 8, 8, 128, 32, 64), ([1000], 1, 32, 8, 128, 32, 64), ([0, 1, 2, 31, 32, 33, 65], 1, 28, 4, 128, 64, 16), ([300, 5, 40], 3, 28, 4, 128, 64, 48),
    ([2, 0, 100, 1], 4, 6, 3, 64, 32, 32), ([257], 1, 16, 1, 64, 64, 16), ([90, 700], 2, 33, 1, 128, 128, 128), ([2500, 3, 1200], 1, 12, 2, 128, 128, 16),
    ([130], 5, 16, 1, 128, 32, 64), ([50] * 40, 1, 8, 2, 64, 32, 16)]


@pytest.mark.parametrize("lens,n_q,H,K,D,gs,page", STEPS)
@pytest.mark.parametrize("kind_q,kind_out,weigh", [("bf16", "bf16", False), ("f32", "f32", False), ("bf16", "f32", True)])
def test_step(lens, n_q, H, K, D, gs, page, kind_q, kind_out, weigh):
    torch, coli = setup()
    g = gen(torch, sum(lens) + H + K + gs)
    s, table, _ = filled(torch, coli, lens, K, page, D, gs, g, columns=2)
    before = s.w.cpu().clone()
    q = torch.randn(len(lens), n_q, H, D, generator=g).to(torch.float32 if kind_q == "f32" else torch.bfloat16)
    scale = 0.5 / math.sqrt(D)
    out, lse = run_step(torch, coli, s, table, lens, q, scale, kind_out, weigh)
    ref, tol, ref_lse, weights, w_tol = reference_step(torch, s, table, lens, q, scale, kind_q, kind_out)
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    got = lse.cpu().double()
    none = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(got), none)
    bound = 1e-4 if kind_q == "bf16" else 2e-2
    assert ((got - ref_lse)[~none].abs() <= bound * (1 + ref_lse[~none].abs())).all()
    w = s.w.cpu()
    want = before.double()
    slack = torch.zeros_like(want)
    if weigh:
        for b, n in enumerate(lens):
            for i in range(-(-n // page)):
                m = min(page, n - i * page)
                want[int(table[b, i]), :, :m] += weights[b][:, i * page:i * page + m]
                slack[int(table[b, i]), :, :m] = w_tol[b][:, i * page:i * page + m] + 2.0 ** -24 * 2
    assert ((w.double() - want).abs() <= slack).all()
    again, _ = run_step(torch, coli, s, table, lens, q, scale, kind_out)
    assert torch.equal(out, again)                       # equal calls, equal bits


@pytest.mark.parametrize("magnitude", [1e-30, 1e-4, 1e4, 1e30])
def test_step_magnitudes(magnitude):
    """Queries of any size: the power of two that their rows are scaled by leaves the scores as they are."""
    torch, coli = setup()
    g = gen(torch, 3)
    s, table, _ = filled(torch, coli, [70], 2, 16, 128, 32, g)
    q = torch.randn(1, 1, 8, 128, generator=g)
    q[..., ::3] *= 2.0 ** -18
    q = (q * magnitude).to(torch.bfloat16)
    scale = 0.05 / magnitude
    out, _ = run_step(torch, coli, s, table, [70], q, scale, "f32")
    ref, tol, *_ = reference_step(torch, s, table, [70], q, scale, "bf16", "f32")
    assert ((out.cpu().double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("size", [2.0 ** -55, 2.0 ** 36])
def test_step_value_sizes(size):
    """Values' scales at both ends of their range: the powers of two of the products take nothing away."""
    torch, coli = setup()
    g = gen(torch, 4)
    s, table, _ = filled(torch, coli, [300, 40], 2, 16, 128, 32, g, spread=1.0)
    q = torch.randn(2, 1, 8, 128, generator=g).to(torch.bfloat16)
    want, lse = run_step(torch, coli, s, table, [300, 40], q, 0.1, "f32")
    s.vs.mul_(size)
    got, lse2 = run_step(torch, coli, s, table, [300, 40], q, 0.1, "f32")
    assert torch.equal(got, want * size) and torch.equal(lse, lse2)      # every step of the sum is that power of two larger


def test_step_strangers_do_not_matter():
    """Rows past a length (any scale, infinities too), pages past the last one and other heads' rows change no bit."""
    torch, coli = setup()
    g = gen(torch, 21)
    lens = [45, 3, 0, 129]
    s, table, _ = filled(torch, coli, lens, 2, 48, 128, 32, g, columns=3)
    q = torch.randn(4, 2, 8, 128, generator=g).to(torch.bfloat16)
    want, _ = run_step(torch, coli, s, table, lens, q, 0.1, "f32")
    assert torch.isfinite(want).all()
    for junk in (float("inf"), -float("inf"), 3e38):
        for t in (s.ks, s.vs):
            t[torch.isnan(t) | torch.isinf(t) | (t > 1e38)] = junk
        got, _ = run_step(torch, coli, s, table, lens, q, 0.1, "f32")
        assert torch.equal(got, want)
    other = torch.full_like(table, 1 << 30)
    for b, n in enumerate(lens):
        other[b, : -(-n // 48)] = table[b, : -(-n // 48)]
    got, _ = run_step(torch, coli, s, other, lens, q, 0.1, "f32")
    assert torch.equal(got, want)


def test_step_nan():
    """A NaN scale that a query sees, or a NaN or infinity in the query, gives NaN; queries and heads that do not see it stay."""
    torch, coli = setup()
    g = gen(torch, 22)
    lens = [60]
    s, table, _ = filled(torch, coli, lens, 2, 64, 128, 32, g)
    q = torch.randn(1, 3, 8, 128, generator=g).to(torch.bfloat16)
    want, _ = run_step(torch, coli, s, table, lens, q, 0.1, "f32")
    page = int(table[0, 0])
    keep = s.ks[page, 1, 58, 2].clone()
    s.ks[page, 1, 58, 2] = float("nan")                  # head 1: query heads 4..7; token 58: queries 1 and 2
    got, lse = run_step(torch, coli, s, table, lens, q, 0.1, "f32")
    assert torch.isnan(got[0, 1:, 4:]).all() and torch.isnan(lse[0, 1:, 4:]).all()
    assert torch.equal(got[0, 0], want[0, 0]) and torch.equal(got[:, :, :4], want[:, :, :4])
    s.ks[page, 1, 58, 2] = keep
    keep = s.vs[page, 0, 59, 1].clone()
    s.vs[page, 0, 59, 1] = float("nan")                  # dims 32..63 of query heads 0..3, query 2 alone
    got, _ = run_step(torch, coli, s, table, lens, q, 0.1, "f32")
    assert torch.isnan(got[0, 2, :4, 32:64]).all()
    got[0, 2, :4, 32:64] = want[0, 2, :4, 32:64]
    assert torch.equal(got, want)
    s.vs[page, 0, 59, 1] = keep
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[0, 1, 5, 17] = bad
        got, _ = run_step(torch, coli, s, table, lens, q2, 0.1, "f32")
        assert torch.isnan(got[0, 1, 5]).all()
        got[0, 1, 5] = want[0, 1, 5]
        assert torch.equal(got, want)


def test_step_bad_pages_and_lengths():
    torch, coli = setup()
    g = gen(torch, 23)
    s, table, _ = filled(torch, coli, [40, 30], 2, 16, 64, 32, g)
    q = torch.randn(2, 1, 4, 64, generator=g).to(torch.bfloat16)
    want, _ = run_step(torch, coli, s, table, [40, 30], q, 0.1, "f32")
    for change in ("page", "negative", "long"):
        t, lens = table.clone(), [40, 30]
        if change == "page":
            t[0, 1] = s.n_pages
        lens[0] = {"page": 40, "negative": -1, "long": 3 * 16 + 1}[change]
        out = torch.empty(2, 1, 4, 64, device="cuda")
        coli.gqa_attend(s.c, q.cuda(), t.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.1, out)
        with pytest.raises(coli.ColiError) as e:
            coli.sync_check()
        assert e.value.code == coli.COLI_EINVAL
        assert torch.equal(out[1], want[1])
    coli.sync_check()


# ------------------------------------------------------------------ eviction
def stays(w, n, keep, recent):
    """Tokens that stay, from the definition."""
    if n <= keep:
        return list(range(n))
    old = n - recent
    order = sorted(range(old), key=lambda t: (0 if math.isnan(w[t]) else 1, -w[t] if not math.isnan(w[t]) else 0.0, t))
    return sorted(order[:keep - recent]) + list(range(old, n))


@pytest.mark.parametrize("lens,keep,recent,K,D,gs,page", [
    ([10], 4, 1, 1, 64, 32, 16), ([100, 0, 7, 65], 20, 5, 3, 128, 32, 16), ([3000], 1100, 100, 2, 128, 128, 64), ([50, 33], 33, 33, 2, 64, 64, 48),
    ([2100, 1500], 1, 0, 1, 128, 64, 32), ([64], 63, 0, 8, 128, 32, 64), ([5000, 4096], 4095, 3, 1, 64, 32, 128)])
@pytest.mark.parametrize("values", ["random", "ties", "special"])
def test_evict(lens, keep, recent, K, D, gs, page, values):
    torch, coli = setup()
    g = gen(torch, sum(lens) + keep)
    per = -(-keep // page)
    s, table, spare = filled(torch, coli, lens, K, page, D, gs, g, spare=per * len(lens))
    if values == "ties":
        s.w.copy_((torch.randint(0, 3, s.w.shape, generator=g).float() * 0.25).cuda())
    elif values == "special":
        some = torch.tensor([0.0, -0.0, -1.0, float("inf"), float("-inf"), float("nan"), 1e-45, 2.0, 2.0000002])
        s.w.copy_(some[torch.randint(0, len(some), s.w.shape, generator=g)].cuda())
    dst = spare.view(len(lens), per).contiguous()
    before = {n: getattr(s, n).cpu().clone() for n in ("k", "v", "ks", "vs", "w")}
    kept = torch.full((len(lens), K, keep), 9, dtype=torch.int32, device="cuda")
    new = torch.full((len(lens),), 9, dtype=torch.int32, device="cuda")
    coli.gqa_evict(s.c, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), keep, recent, dst.cuda(), kept, new)
    coli.sync_check()
    assert new.cpu().tolist() == [min(keep, n) for n in lens]
    want = {n: x.clone() for n, x in before.items()}
    for b, n in enumerate(lens):
        pages = [int(i) for i in table[b, : -(-n // page)]]
        for h in range(K):
            w = before["w"][pages, h].flatten()[:n].tolist() if n else []
            ref = stays(w, n, keep, recent)
            assert kept[b, h].cpu().tolist() == ref + [-1] * (keep - len(ref))
            for i, t in enumerate(ref):
                for name in want:
                    want[name][int(dst[b, i // page]), h, i % page] = before[name][pages[t // page], h, t % page]
    for name, x in want.items():
        got = getattr(s, name).cpu()
        same = got == x if x.dtype == torch.uint8 else (got == x) | (torch.isnan(got) & torch.isnan(x))
        assert same.all(), name


def test_evict_bad_pages_and_lengths():
    torch, coli = setup()
    g = gen(torch, 31)
    s, table, spare = filled(torch, coli, [40, 30], 1, 16, 64, 32, g, spare=2)
    dst = spare.view(2, 1).contiguous()
    lens = torch.tensor([40, 30], dtype=torch.int32, device="cuda")

    def run(table, lens, dst):
        kept, new = torch.full((2, 1, 10), 9, dtype=torch.int32, device="cuda"), torch.full((2,), 9, dtype=torch.int32, device="cuda")
        coli.gqa_evict(s.c, table.cuda(), lens, 10, 2, dst.cuda(), kept, new)
        return kept.cpu(), new.cpu()

    want, _ = run(table, lens, dst)
    coli.sync_check()
    for change in ("page", "dst", "length"):
        t, d, n = table.clone(), dst.clone(), lens.clone()
        if change == "page":
            t[0, 0] = -3
        elif change == "dst":
            d[0, 0] = s.n_pages
        else:
            n[0] = 49
        kept, new = run(t, n, d)
        with pytest.raises(coli.ColiError) as e:
            coli.sync_check()
        assert e.value.code == coli.COLI_EINVAL
        assert torch.equal(kept[1], want[1]) and int(new[1]) == 10
        if change == "length":
            assert int(new[0]) == 0 and (kept[0] == -1).all()
    coli.sync_check()


# ------------------------------------------------------------------ the binding's refusals
def test_binding_refuses():
    torch, coli = setup()
    g = gen(torch, 41)
    s, table, _ = filled(torch, coli, [20], 2, 16, 64, 32, g)
    q = torch.zeros(1, 1, 4, 64, device="cuda", dtype=torch.bfloat16)
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    t = table.cuda()
    x = torch.zeros(3, 2, 64, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    bad = [
        lambda: coli.GqaCache(s.k, s.v[:, :1], s.ks, s.vs), lambda: coli.GqaCache(s.k.cpu(), s.v, s.ks, s.vs),
        lambda: coli.GqaCache(s.k, s.v, s.ks.float(), s.vs), lambda: coli.GqaCache(s.k, s.v, s.ks, s.vs, weights=s.w[:1]),
        lambda: coli.gqa_attend(s.c, q[..., :32], t, lens, 1.0, q), lambda: coli.gqa_attend(s.c, q, t.long(), lens, 1.0, q.clone()),
        lambda: coli.gqa_attend(s.c, q, t, lens.long(), 1.0, q.clone()), lambda: coli.gqa_attend(s.c, q.expand(1, 2, 4, 64), t, lens, 1.0, q.expand(1, 2, 4, 64)),
        lambda: coli.gqa_append(s.c, x, x.bfloat16(), slots), lambda: coli.gqa_append(s.c, x, x, slots[:2]),
        lambda: coli.gqa_append(s.c, x.transpose(0, 1).contiguous().transpose(0, 1), x, slots), lambda: coli.gqa_append(s.c, x.cpu(), x, slots),
        lambda: coli.gqa_read(s.c, t, torch.tensor([0, 3], dtype=torch.int32, device="cuda"), x, x[:2]),
        lambda: coli.gqa_evict(s.c, t, lens, 5, 1, t, torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda"), lens.clone()),
        lambda: coli.gqa_evict(s.c, t, lens, 4, 1, t, torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda"), lens),
        lambda: coli.gqa_prefill(x, x, x.bfloat16(), slots.int(), slots.int(), 1.0, x.clone()),
        lambda: coli.gqa_prefill(x, x[:, :, :32], x, slots.int(), slots.int(), 1.0, x.clone())]
    for i, f in enumerate(bad):
        with pytest.raises(coli.ColiError):
            f()
            pytest.fail(f"call {i} was not refused")
    none = coli.GqaCache(s.k, s.v, s.ks, s.vs)
    with pytest.raises(coli.ColiError):
        coli.gqa_attend(none, q, t, lens, 1.0, q.clone(), weigh=True)
