"""The latent-attention entry points refuse bad arguments before touching CUDA."""
import ctypes

import pytest

F32, BF16, E4M3 = 0, 1, 2
EINVAL, EFMT = -1, -2


class Cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("latent", ctypes.c_int), ("rope", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_pages", ctypes.c_int64), ("rows", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    lib = ctypes.CDLL(__graft_entry__._load_build_module().build())
    lib.coli_last_error.restype = ctypes.c_char_p
    return lib


A = 1 << 20          # an aligned address nothing dereferences: every call below is refused first
P, I, I64, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float


def cache(**kw):
    d = dict(dtype=E4M3, latent=512, rope=64, page_size=64, n_pages=10, rows=A, scales=A)
    d.update(kw)
    return ctypes.byref(Cache(*[d[n] for n, _ in Cache._fields_]))


def query(lib, **kw):
    d = dict(q=A, q_stride=2 * 192, T=2, H=2, nope=128, rope=64, pos=A, rot=A, n_pos=4, inter=0, dn=F32, on=A, ln=128, dr=F32, orr=A, lr=64)
    d.update(kw)
    return lib.coli_mla_query(P(d["q"]), I64(d["q_stride"]), d["T"], d["H"], d["nope"], d["rope"], P(d["pos"]), P(d["rot"]), d["n_pos"],
                              d["inter"], d["dn"], P(d["on"]), I64(d["ln"]), d["dr"], P(d["orr"]), I64(d["lr"]), None)


def append(lib, c=None, **kw):
    d = dict(kv=A, stride=576, T=2, norm=A, eps=1e-6, pos=A, rot=A, n_pos=4, slots=A)
    d.update(kw)
    return lib.coli_mla_append(c if c is not None else cache(), P(d["kv"]), I64(d["stride"]), d["T"], P(d["norm"]), F(d["eps"]),
                               P(d["pos"]), P(d["rot"]), d["n_pos"], 0, P(d["slots"]), None)


def read(lib, c=None, **kw):
    d = dict(pages=A, ps=4, n=2, cu=A, T=5, dtype=F32, out=A, stride=576)
    d.update(kw)
    return lib.coli_mla_read(c if c is not None else cache(), P(d["pages"]), I64(d["ps"]), d["n"], P(d["cu"]), d["T"], d["dtype"],
                             P(d["out"]), I64(d["stride"]), None)


def attend(lib, c=None, **kw):
    d = dict(dq=BF16, ql=A, qr=A, n=2, n_q=1, H=16, pages=A, ps=4, lens=A, scale=0.1, do=BF16, out=A, lse=None)
    d.update(kw)
    return lib.coli_mla_attend(c if c is not None else cache(), d["dq"], P(d["ql"]), P(d["qr"]), d["n"], d["n_q"], d["H"],
                               P(d["pages"]), I64(d["ps"]), P(d["lens"]), F(d["scale"]), d["do"], P(d["out"]), P(d["lse"]), None)


def prefill(lib, **kw):
    d = dict(dt=BF16, q=A, qs=16 * 192, kv=A, ks=16 * 256, kr=A, krs=64, Tq=4, Tk=5, n=1, cuq=A, cuk=A, H=16, nope=128, rope=64, v=128,
             scale=0.1, do=BF16, out=A, lse=None)
    d.update(kw)
    return lib.coli_mla_prefill(d["dt"], P(d["q"]), I64(d["qs"]), P(d["kv"]), I64(d["ks"]), P(d["kr"]), I64(d["krs"]), d["Tq"], d["Tk"],
                                d["n"], P(d["cuq"]), P(d["cuk"]), d["H"], d["nope"], d["rope"], d["v"], F(d["scale"]), d["do"],
                                P(d["out"]), P(d["lse"]), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=F32), EFMT), (dict(dtype=7), EFMT), (dict(latent=64), EINVAL), (dict(latent=576), EINVAL), (dict(latent=500), EINVAL),
    (dict(rope=0), EINVAL), (dict(rope=24), EINVAL), (dict(rope=80), EINVAL), (dict(page_size=8), EINVAL), (dict(page_size=40), EINVAL),
    (dict(n_pages=0), EINVAL), (dict(n_pages=1 << 26), EINVAL), (dict(rows=None), EINVAL), (dict(rows=A + 8), EINVAL),
    (dict(scales=None), EINVAL)])
def test_caches(lib, kw, code):
    for f in (append, read, attend):
        assert f(lib, cache(**kw)) == code
        assert lib.coli_last_error()


def test_null_cache(lib):
    assert lib.coli_mla_attend(None, BF16, P(A), P(A), 1, 1, 16, P(A), I64(4), P(A), F(1.0), BF16, P(A), None, None) == EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(H=0), EINVAL), (dict(nope=4), EINVAL), (dict(nope=-8), EINVAL), (dict(rope=8), EINVAL),
    (dict(rope=272), EINVAL), (dict(dn=E4M3), EFMT), (dict(dr=5), EFMT), (dict(q_stride=380), EINVAL), (dict(q_stride=390), EINVAL),
    (dict(ln=120), EINVAL), (dict(ln=132), EINVAL), (dict(lr=60), EINVAL), (dict(q=None), EINVAL), (dict(q=A + 4), EINVAL),
    (dict(pos=None), EINVAL), (dict(rot=None), EINVAL), (dict(n_pos=0), EINVAL), (dict(on=None), EINVAL), (dict(orr=A + 2), EINVAL)])
def test_query(lib, kw, code):
    assert query(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(stride=572), EINVAL), (dict(stride=578), EINVAL), (dict(eps=0.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(kv=None), EINVAL), (dict(norm=A + 4), EINVAL), (dict(pos=None), EINVAL), (dict(slots=None), EINVAL), (dict(slots=A + 4), EINVAL)])
def test_append(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), EINVAL), (dict(n=-1), EINVAL), (dict(ps=0), EINVAL), (dict(dtype=E4M3), EFMT), (dict(stride=568), EINVAL),
    (dict(stride=580), EINVAL), (dict(pages=None), EINVAL), (dict(cu=None), EINVAL), (dict(out=A + 8), EINVAL)])
def test_read(lib, kw, code):
    assert read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dq=E4M3), EFMT), (dict(do=9), EFMT), (dict(n=-1), EINVAL), (dict(n_q=0), EINVAL), (dict(H=0), EINVAL), (dict(H=1025), EINVAL),
    (dict(n_q=5000), EINVAL), (dict(ps=0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(ql=None), EINVAL), (dict(qr=A + 8), EINVAL),
    (dict(pages=None), EINVAL), (dict(lens=A + 2), EINVAL), (dict(out=None), EINVAL), (dict(lse=A + 1), EINVAL)])
def test_attend(lib, kw, code):
    assert attend(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=E4M3), EFMT), (dict(do=-1), EFMT), (dict(nope=96), EINVAL), (dict(v=192), EINVAL), (dict(rope=0), EINVAL), (dict(rope=40), EINVAL),
    (dict(Tq=-1), EINVAL), (dict(Tk=-1), EINVAL), (dict(n=-1), EINVAL), (dict(H=0), EINVAL), (dict(qs=16 * 192 - 8), EINVAL),
    (dict(ks=16 * 256 + 4), EINVAL), (dict(krs=56), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(q=None), EINVAL),
    (dict(kv=A + 8), EINVAL), (dict(kr=None), EINVAL), (dict(cuq=None), EINVAL), (dict(cuk=A + 1), EINVAL), (dict(out=None), EINVAL)])
def test_prefill(lib, kw, code):
    assert prefill(lib, **kw) == code


def test_injected_failures_reach_them(lib):
    """The injection gate stands behind the argument checks and before any launch."""
    lib.coli_set_fail_after(I64(0))
    try:
        for f in (query, append, read, attend, prefill):
            assert f(lib) == -6
    finally:
        lib.coli_set_fail_after(I64(-1))


def test_nothing_to_do(lib):
    assert query(lib, T=0, q=None) == 0
    assert append(lib, T=0, kv=None) == 0
    assert read(lib, T=0) == 0 and read(lib, n=0, cu=None) == 0
    assert attend(lib, n=0, ql=None) == 0
    assert prefill(lib, Tq=0, q=None) == 0 and prefill(lib, n=0) == 0
