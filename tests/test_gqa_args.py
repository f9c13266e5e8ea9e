"""The grouped-head attention entry points refuse bad arguments before touching CUDA."""
import ctypes

import pytest

from test_mla_args import A, BF16, E4M3, EFMT, EINVAL, F, F32, I64, P, lib  # noqa: F401


class Cache(ctypes.Structure):
    _fields_ = [("n_kv", ctypes.c_int), ("dim", ctypes.c_int), ("gs", ctypes.c_int), ("page_size", ctypes.c_int), ("n_pages", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("weights", ctypes.c_void_p)]


def cache(**kw):
    d = dict(n_kv=4, dim=128, gs=32, page_size=64, n_pages=10, k=A, v=A, k_scales=A, v_scales=A, weights=A)
    d.update(kw)
    return ctypes.byref(Cache(*[d[n] for n, _ in Cache._fields_]))


def append(lib, c=None, **kw):  # noqa: F811
    d = dict(dt=F32, k=A, ks=512, v=A, vs=512, T=2, slots=A)
    d.update(kw)
    return lib.coli_gqa_append(c if c is not None else cache(), d["dt"], P(d["k"]), I64(d["ks"]), P(d["v"]), I64(d["vs"]), d["T"],
                               P(d["slots"]), None)


def read(lib, c=None, **kw):  # noqa: F811
    d = dict(pages=A, ps=4, n=2, cu=A, T=5, dt=F32, k=A, ks=512, v=A, vs=512)
    d.update(kw)
    return lib.coli_gqa_read(c if c is not None else cache(), P(d["pages"]), I64(d["ps"]), d["n"], P(d["cu"]), d["T"], d["dt"], P(d["k"]),
                             I64(d["ks"]), P(d["v"]), I64(d["vs"]), None)


def attend(lib, c=None, **kw):  # noqa: F811
    d = dict(dq=BF16, q=A, n=2, n_q=1, H=16, pages=A, ps=4, lens=A, scale=0.1, weigh=0, do=BF16, out=A, lse=None)
    d.update(kw)
    return lib.coli_gqa_attend(c if c is not None else cache(), d["dq"], P(d["q"]), d["n"], d["n_q"], d["H"], P(d["pages"]), I64(d["ps"]),
                               P(d["lens"]), F(d["scale"]), d["weigh"], d["do"], P(d["out"]), P(d["lse"]), None)


def evict(lib, c=None, **kw):  # noqa: F811
    d = dict(pages=A, ps=4, n=2, lens=A, keep=60, recent=10, dst=A, ds=1, kept=A, new=A + 64)
    d.update(kw)
    return lib.coli_gqa_evict(c if c is not None else cache(), P(d["pages"]), I64(d["ps"]), d["n"], P(d["lens"]), d["keep"], d["recent"],
                              P(d["dst"]), I64(d["ds"]), P(d["kept"]), P(d["new"]), None)


def prefill(lib, **kw):  # noqa: F811
    d = dict(dt=BF16, q=A, qs=16 * 128, k=A, ks=512, v=A, vs=512, Tq=4, Tk=5, n=1, cuq=A, cuk=A, H=16, K=4, D=128, scale=0.1, do=BF16, out=A,
             lse=None)
    d.update(kw)
    return lib.coli_gqa_prefill(d["dt"], P(d["q"]), I64(d["qs"]), P(d["k"]), I64(d["ks"]), P(d["v"]), I64(d["vs"]), d["Tq"], d["Tk"], d["n"],
                                P(d["cuq"]), P(d["cuk"]), d["H"], d["K"], d["D"], F(d["scale"]), d["do"], P(d["out"]), P(d["lse"]), None)


@pytest.mark.parametrize("kw", [
    dict(n_kv=0), dict(n_kv=1025), dict(dim=96), dict(dim=256), dict(gs=16), dict(gs=48), dict(dim=64, gs=128), dict(page_size=8),
    dict(page_size=40), dict(page_size=65552), dict(n_pages=0), dict(n_pages=1 << 23), dict(k=None), dict(v=A + 8), dict(k_scales=None),
    dict(v_scales=A + 2), dict(weights=A + 4)])
def test_caches(lib, kw):  # noqa: F811
    for f in (append, read, attend, evict):
        assert f(lib, cache(**kw)) == EINVAL
        assert lib.coli_last_error()


def test_null_cache(lib):  # noqa: F811
    assert lib.coli_gqa_append(None, F32, P(A), I64(512), P(A), I64(512), 1, P(A), None) == EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(dt=E4M3), EFMT), (dict(T=-1), EINVAL), (dict(ks=504), EINVAL), (dict(vs=516), EINVAL), (dict(k=None), EINVAL), (dict(v=A + 8), EINVAL),
    (dict(slots=None), EINVAL), (dict(slots=A + 4), EINVAL), (dict(T=1 << 29), EINVAL)])
def test_append(lib, kw, code):  # noqa: F811
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=E4M3), EFMT), (dict(T=-1), EINVAL), (dict(n=-1), EINVAL), (dict(ps=0), EINVAL), (dict(ps=1 << 31), EINVAL), (dict(ks=504), EINVAL),
    (dict(vs=516), EINVAL), (dict(T=1 << 29), EINVAL), (dict(pages=None), EINVAL), (dict(cu=A + 2), EINVAL), (dict(k=A + 8), EINVAL), (dict(v=None), EINVAL)])
def test_read(lib, kw, code):  # noqa: F811
    assert read(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dq=E4M3), EFMT), (dict(do=9), EFMT), (dict(n=-1), EINVAL), (dict(n_q=0), EINVAL), (dict(H=0), EINVAL), (dict(H=1028), EINVAL),
    (dict(H=18), EINVAL), (dict(n_q=5000), EINVAL), (dict(ps=0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(q=None), EINVAL),
    (dict(pages=None), EINVAL), (dict(lens=A + 2), EINVAL), (dict(out=A + 8), EINVAL), (dict(lse=A + 1), EINVAL)])
def test_attend(lib, kw, code):  # noqa: F811
    assert attend(lib, **kw) == code


@pytest.mark.parametrize("ps,page,n", [((1 << 31) - 1, 65536, 1 << 24), (1 << 30, 65536, 1 << 25), ((1 << 31) - 1, 16, 16)])
def test_attend_tiles(lib, ps, page, n):  # noqa: F811
    assert attend(lib, cache(page_size=page, n_pages=1), ps=ps, n=n, H=4) == EINVAL
    assert b"pages_stride" in lib.coli_last_error()


def test_weights_are_needed(lib):  # noqa: F811
    assert attend(lib, cache(weights=None), weigh=1) == EINVAL
    assert evict(lib, cache(weights=None)) == EINVAL


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(keep=0), dict(recent=-1), dict(recent=61), dict(ps=0), dict(ds=0), dict(keep=65), dict(pages=None), dict(lens=None),
    dict(dst=A + 2), dict(kept=None), dict(new=None), dict(new=A), dict(n=1 << 30)])
def test_evict(lib, kw):  # noqa: F811
    assert evict(lib, **kw) == EINVAL


@pytest.mark.parametrize("keep,code", [((1 << 30) + 1, EINVAL), ((1 << 31) - 1, EINVAL)])
def test_evict_keeps_no_more_than_a_sequence_may_have(lib, keep, code):  # noqa: F811
    assert evict(lib, cache(page_size=65536, n_pages=1), keep=keep, ds=1 << 15, n=1) == code
    assert b"2^30" in lib.coli_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dt=E4M3), EFMT), (dict(do=-1), EFMT), (dict(D=96), EINVAL), (dict(K=3), EINVAL), (dict(K=0), EINVAL), (dict(H=0), EINVAL),
    (dict(H=1028), EINVAL), (dict(H=258, K=2, qs=258 * 128), EINVAL), (dict(Tq=-1), EINVAL), (dict(Tk=-1), EINVAL), (dict(n=-1), EINVAL),
    (dict(qs=2040), EINVAL), (dict(ks=516), EINVAL), (dict(vs=504), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(q=None), EINVAL),
    (dict(k=A + 8), EINVAL), (dict(v=None), EINVAL), (dict(cuq=None), EINVAL), (dict(cuk=A + 1), EINVAL), (dict(out=None), EINVAL),
    (dict(lse=A + 2), EINVAL), (dict(Tq=1 << 28), EINVAL), (dict(Tk=1 << 29), EINVAL)])
def test_prefill(lib, kw, code):  # noqa: F811
    assert prefill(lib, **kw) == code


def test_injected_failures_reach_them(lib):  # noqa: F811
    """The injection gate stands behind the argument checks and before any launch."""
    lib.coli_set_fail_after(I64(0))
    try:
        for f in (append, read, attend, evict, prefill):
            assert f(lib) == -6
    finally:
        lib.coli_set_fail_after(I64(-1))


def test_nothing_to_do(lib):  # noqa: F811
    assert append(lib, T=0, k=None) == 0
    assert read(lib, T=0) == 0 and read(lib, n=0, cu=None) == 0
    assert attend(lib, n=0, q=None) == 0
    assert evict(lib, n=0, kept=None) == 0
    assert prefill(lib, Tq=0, q=None) == 0 and prefill(lib, n=0) == 0
