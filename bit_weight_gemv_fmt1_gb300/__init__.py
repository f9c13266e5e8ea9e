"""Python binding of libcoli.so (include/coli.h): argument marshalling only.

Every computation runs in the CUDA library.  There is no other
implementation: if libcoli.so is missing this module raises ImportError
(build it with ``python bit_weight_gemv_fmt1_gb300/build.py`` or
``__graft_entry__.build()``), and every library error is raised as
ColiError with the library's message.

Tensors are passed as torch CUDA tensors (their data pointers) and numpy
arrays (host uploads); ``stream`` defaults to torch's current stream.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libcoli.so")

COLI_OK, COLI_EINVAL, COLI_EFMT, COLI_ENOMEM, COLI_ECUDA, COLI_ETIMEOUT, COLI_EINJECTED, COLI_EDEVICE = \
    0, -1, -2, -3, -4, -5, -6, -7
_NAMES = {-1: "COLI_EINVAL", -2: "COLI_EFMT", -3: "COLI_ENOMEM", -4: "COLI_ECUDA", -5: "COLI_ETIMEOUT",
          -6: "COLI_EINJECTED", -7: "COLI_EDEVICE"}

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: the CUDA library has not been built "
                      "(run __graft_entry__.build() or bit_weight_gemv_fmt1_gb300/build.py)")

_lib = ctypes.CDLL(LIB_PATH)
_vp, _i64, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class _Stats(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_uint64), ("launches", ctypes.c_uint64), ("weight_bytes", ctypes.c_uint64)]


class _MlaCache(ctypes.Structure):
    _fields_ = [("dtype", _int), ("latent", _int), ("rope", _int), ("page_size", _int), ("n_pages", ctypes.c_int64),
                ("rows", _vp), ("scales", _vp)]


class _GqaCache(ctypes.Structure):
    _fields_ = [("n_kv", _int), ("dim", _int), ("gs", _int), ("page_size", _int), ("n_pages", ctypes.c_int64),
                ("k", _vp), ("v", _vp), ("k_scales", _vp), ("v_scales", _vp), ("weights", _vp)]


class _Expert(ctypes.Structure):
    _fields_ = [("gate", _vp), ("up", _vp), ("down", _vp)]


_lib.coli_version.restype = ctypes.c_char_p
_lib.coli_last_error.restype = ctypes.c_char_p
_lib.coli_tensor_upload.argtypes = [_int, _int, _i64, _i64, _vp, _vp, _vp, ctypes.POINTER(_vp)]
_lib.coli_tensor_upload_host.argtypes = [_int, _int, _i64, _i64, _vp, _vp, ctypes.POINTER(_vp)]
_lib.coli_tensor_free.argtypes = [_vp]
_lib.coli_tensor_free.restype = None
_lib.coli_tensor_info.argtypes = [_vp] + [ctypes.POINTER(_int)] * 2 + [ctypes.POINTER(_i64)] * 4
_lib.coli_matmul.argtypes = [_vp, _vp, _vp, _int, _vp]
_lib.coli_matmul_multi.argtypes = [_int, ctypes.POINTER(_vp), _vp, ctypes.POINTER(_vp), _int, _vp]
_lib.coli_matmul_rows.argtypes = [_vp, _i64, _i64, _i64, _int, _vp, _vp, _int, _vp]
_lib.coli_matmul_rows_t.argtypes = [_vp, _i64, _i64, _i64, _int, _vp, _vp, _int, _vp]
_lib.coli_moe_route.argtypes = [_vp, _int, _int, _int, _vp, _vp, _vp]
_lib.coli_moe_block.argtypes = [_vp, _int, ctypes.POINTER(_Expert), _int, _vp, _vp, _int, _vp, _vp]
_lib.coli_moe_block_noalloc.argtypes = [_vp, _int, ctypes.POINTER(_Expert), _int, _vp, _vp, _int, _vp, _vp, _vp]
_lib.coli_expert_table_create.argtypes = [ctypes.POINTER(_Expert), _int, ctypes.POINTER(_vp)]
_lib.coli_expert_table_free.argtypes = [_vp]
_lib.coli_expert_table_free.restype = None
_lib.coli_moe_block_t.argtypes = [_vp, _int, _vp, _vp, _vp, _int, _vp, _vp]
_lib.coli_moe_topk.argtypes = [_vp, _vp, _int, _int, _int, ctypes.c_float, _int, ctypes.c_float, _vp, _vp, _vp]
_lib.coli_moe_router.argtypes = [_vp, _int, _vp, _vp, _int, ctypes.c_float, _int, ctypes.c_float, _vp, _vp, _vp]
_f = ctypes.c_float
_lib.coli_mla_query.argtypes = [_vp, _i64, _int, _int, _int, _int, _vp, _vp, _int, _int, _int, _vp, _i64, _int, _vp, _i64, _vp]
_lib.coli_mla_append.argtypes = [_vp, _vp, _i64, _int, _vp, _f, _vp, _vp, _int, _int, _vp, _vp]
_lib.coli_mla_read.argtypes = [_vp, _vp, _i64, _int, _vp, _int, _int, _vp, _i64, _vp]
_lib.coli_mla_attend.argtypes = [_vp, _int, _vp, _vp, _int, _int, _int, _vp, _i64, _vp, _f, _int, _vp, _vp, _vp]
_lib.coli_mla_prefill.argtypes = [_int, _vp, _i64, _vp, _i64, _vp, _i64, _int, _int, _int, _vp, _vp, _int, _int, _int, _int, _f,
                                  _int, _vp, _vp, _vp]
_lib.coli_gqa_prefill.argtypes = [_int, _vp, _i64, _vp, _i64, _vp, _i64, _int, _int, _int, _vp, _vp, _int, _int, _int, _f, _int, _vp,
                                  _vp, _vp]
_lib.coli_gqa_append.argtypes = [_vp, _int, _vp, _i64, _vp, _i64, _int, _vp, _vp]
_lib.coli_gqa_read.argtypes = [_vp, _vp, _i64, _int, _vp, _int, _int, _vp, _i64, _vp, _i64, _vp]
_lib.coli_gqa_attend.argtypes = [_vp, _int, _vp, _int, _int, _int, _vp, _i64, _vp, _f, _int, _int, _vp, _vp, _vp]
_lib.coli_gqa_evict.argtypes = [_vp, _vp, _i64, _int, _vp, _int, _int, _vp, _i64, _vp, _vp, _vp]
_lib.coli_sync_check.argtypes = [_vp]
_lib.coli_get_stats.argtypes = [ctypes.POINTER(_Stats)]
_lib.coli_get_stats.restype = None
_lib.coli_reset_stats.restype = None
_lib.coli_set_fail_after.argtypes = [_i64]
_lib.coli_set_fail_after.restype = None
_lib.coli_set_wait_limit.argtypes = [_i64]
_lib.coli_set_wait_limit.restype = None

EXPORTS = ("coli_tensor_upload", "coli_tensor_upload_host", "coli_tensor_free", "coli_tensor_info", "coli_matmul", "coli_matmul_multi",
           "coli_matmul_rows", "coli_matmul_rows_t",
           "coli_moe_route", "coli_moe_topk", "coli_moe_router", "coli_moe_block", "coli_moe_block_noalloc",
           "coli_expert_table_create", "coli_expert_table_free", "coli_moe_block_t",
           "coli_mla_query", "coli_mla_append", "coli_mla_read", "coli_mla_attend", "coli_mla_prefill",
           "coli_gqa_prefill", "coli_gqa_append", "coli_gqa_read", "coli_gqa_attend", "coli_gqa_evict",
           "coli_sync_check", "coli_last_error", "coli_get_stats", "coli_reset_stats", "coli_set_fail_after",
           "coli_set_wait_limit", "coli_version")


class ColiError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_NAMES.get(code, code)}: {msg}")
        self.code = code


def _check(rc: int):
    if rc != COLI_OK:
        raise ColiError(rc, _lib.coli_last_error().decode())


_torch = None
_raw_stream = None


def _device() -> int:
    """The current device, on which the library launches and all of a call's tensors have to be."""
    _load_torch()
    return _device()


def _load_torch():
    """torch, imported at first use (uploads and the host calls do without it)."""
    global _torch, _raw_stream, _device
    import torch
    _torch = torch
    # without torch.cuda's look at whether CUDA is initialised, which a call's CUDA tensors have seen to
    _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    # the handle of the current stream without building a Stream object (3 us a call), where torch has it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _DTYPES.update({torch.float32: COLI_F32, torch.bfloat16: COLI_BF16, torch.float8_e4m3fn: COLI_E4M3})
    return torch


def _stream(stream):
    if stream is None:
        torch = _torch or _load_torch()
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream




def _ptr(t):
    return None if t is None else t.data_ptr()


def version() -> str:
    return _lib.coli_version().decode()


class Tensor:
    """An uploaded weight matrix (owns its device memory)."""

    def __init__(self, handle: int, fmt: int, gs: int, O: int, I: int):
        self._h = handle
        self.fmt, self.gs, self.O, self.I = fmt, gs, O, I

    @property
    def handle(self) -> int:
        return self._h

    def info(self) -> dict:
        f, g = _int(), _int()
        O, I, db, ab = _i64(), _i64(), _i64(), _i64()
        _check(_lib.coli_tensor_info(self._h, f, g, O, I, db, ab))
        return dict(fmt=f.value, gs=g.value, O=O.value, I=I.value, device_bytes=db.value, alg_bytes=ab.value)

    def free(self):
        if self._h:
            _lib.coli_tensor_free(self._h)
            self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def tensor_upload(fmt: int, gs: int, O: int, I: int, data: np.ndarray, scales: np.ndarray | None,
                  stream=None) -> Tensor:
    data = np.ascontiguousarray(data)
    sc = None if scales is None else np.ascontiguousarray(scales, dtype=np.float32)
    out = _vp()
    _check(_lib.coli_tensor_upload(int(fmt), int(gs), int(O), int(I), data.ctypes.data,
                                   None if sc is None else sc.ctypes.data, _stream(stream), ctypes.byref(out)))
    return Tensor(out.value, int(fmt), int(gs), int(O), int(I))


def tensor_upload_host(fmt: int, gs: int, O: int, I: int, data: np.ndarray, scales: np.ndarray | None) -> Tensor:
    """As tensor_upload, but the weights stay in pinned host memory and the
    kernels read them zero-copy over the CPU-GPU link."""
    data = np.ascontiguousarray(data)
    sc = None if scales is None else np.ascontiguousarray(scales, dtype=np.float32)
    out = _vp()
    _check(_lib.coli_tensor_upload_host(int(fmt), int(gs), int(O), int(I), data.ctypes.data,
                                        None if sc is None else sc.ctypes.data, ctypes.byref(out)))
    return Tensor(out.value, int(fmt), int(gs), int(O), int(I))


def matmul(W: Tensor, x, y, S: int | None = None, stream=None):
    """y[S, O] = x[S, I] @ W^T (x, y: contiguous float32 CUDA tensors)."""
    S = x.shape[0] if S is None else S
    _check(_lib.coli_matmul(W.handle, _ptr(x), _ptr(y), int(S), _stream(stream)))
    return y


def matmul_rows(W: Tensor, o0: int, stride: int, n_rows: int, n_heads: int, x, y, S: int | None = None,
                stream=None):
    """Per-head row-range matvec of the kv_b absorption path:
    y[s, h, j] = sum_i W[o0 + h*stride + j, i] * x[s, h, i]  (x [S, n_heads, I], y [S, n_heads, n_rows])."""
    S = x.shape[0] if S is None else S
    _check(_lib.coli_matmul_rows(W.handle, int(o0), int(stride), int(n_rows), int(n_heads), _ptr(x), _ptr(y), int(S),
                                 _stream(stream)))
    return y


def matmul_rows_t(W: Tensor, o0: int, stride: int, n_rows: int, n_heads: int, x, y, S: int | None = None,
                  stream=None):
    """Transposed per-head product: y[s, h, i] = sum_j x[s, h, j] * W[o0 + h*stride + j, i]
    (x [S, n_heads, n_rows], y [S, n_heads, I])."""
    S = x.shape[0] if S is None else S
    _check(_lib.coli_matmul_rows_t(W.handle, int(o0), int(stride), int(n_rows), int(n_heads), _ptr(x), _ptr(y),
                                   int(S), _stream(stream)))
    return y


def matmul_multi(Ws, x, ys, S: int | None = None, stream=None):
    n = len(Ws)
    S = x.shape[0] if S is None else S
    Wa = (_vp * n)(*[w.handle for w in Ws])
    Ya = (_vp * n)(*[_ptr(y) for y in ys])
    _check(_lib.coli_matmul_multi(n, Wa, _ptr(x), Ya, int(S), _stream(stream)))
    return ys


def moe_route(ids, n_experts: int, offsets, order, stream=None):
    S, K = ids.shape
    _check(_lib.coli_moe_route(_ptr(ids), int(S), int(K), int(n_experts), _ptr(offsets), _ptr(order),
                               _stream(stream)))
    return offsets, order


def moe_topk(logits, K: int, ids, w, bias=None, top_p: float = 0.0, norm_topk: bool = False,
             routed_scale: float = 1.0, stream=None):
    """Router top-K of device f32 logits [S, E] into ids [S, K] int32 and w [S, K] f32 (see coli.h)."""
    S, E = logits.shape
    _check(_lib.coli_moe_topk(_ptr(logits), _ptr(bias), int(S), int(E), int(K), float(top_p), int(bool(norm_topk)),
                              float(routed_scale), _ptr(ids), _ptr(w), _stream(stream)))
    return ids, w


def moe_router(x, router: Tensor, K: int, ids, w, bias=None, top_p: float = 0.0, norm_topk: bool = False,
               routed_scale: float = 1.0, stream=None):
    """logits = x @ router^T, then moe_topk (one call, see coli.h)."""
    S = x.shape[0]
    _check(_lib.coli_moe_router(_ptr(x), int(S), router.handle, _ptr(bias), int(K), float(top_p),
                                int(bool(norm_topk)), float(routed_scale), _ptr(ids), _ptr(w), _stream(stream)))
    return ids, w


class ExpertTable:
    """An expert table: the host array of coli_expert descriptors (keeps the
    tensors alive) and, from the first block call on, the library's checked
    device copy (coli_expert_table_create), freed with the object."""

    def __init__(self, experts):
        self.experts = list(experts)
        self.arr = (_Expert * len(self.experts))(*[_Expert(g.handle, u.handle, d.handle)
                                                   for (g, u, d) in self.experts])
        self._t = None

    def __len__(self):
        return len(self.experts)

    def handle(self) -> int:
        if self._t is None:
            h = _vp()
            _check(_lib.coli_expert_table_create(self.arr, len(self.experts), ctypes.byref(h)))
            self._t = h.value
        return self._t

    def __del__(self):
        if getattr(self, "_t", None):
            _lib.coli_expert_table_free(self._t)
            self._t = None


def moe_block(x, table: ExpertTable, ids, w, y, stream=None):
    """coli_moe_block_t on the table's device copy."""
    S, K = ids.shape
    _check(_lib.coli_moe_block_t(_ptr(x), int(S), table.handle(), _ptr(ids), _ptr(w), int(K), _ptr(y),
                                 _stream(stream)))
    return y


def moe_block_array(x, table: ExpertTable, ids, w, y, stream=None):
    """coli_moe_block on the host array (the table is checked on every call)."""
    S, K = ids.shape
    _check(_lib.coli_moe_block(_ptr(x), int(S), table.arr, len(table), _ptr(ids), _ptr(w), int(K), _ptr(y),
                               _stream(stream)))
    return y


def moe_block_noalloc(x, table: ExpertTable, ids, w, y, dev_error, stream=None):
    """The decode expert block without any device allocation (see coli.h);
    dev_error is a 1-element int32 CUDA tensor that receives the kernel's
    error code (0 = none)."""
    S, K = ids.shape
    _check(_lib.coli_moe_block_noalloc(_ptr(x), int(S), table.arr, len(table), _ptr(ids), _ptr(w), int(K), _ptr(y),
                                       _ptr(dev_error), _stream(stream)))
    return y


COLI_F32, COLI_BF16, COLI_E4M3 = 0, 1, 2
_DTYPES: dict = {}


def _refuse(msg: str):
    raise ColiError(COLI_EINVAL, msg)


def _dtype(t) -> int:
    """The library's element type of a tensor (COLI_EFMT for one it has not)."""
    if _torch is None:
        _load_torch()
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ColiError(COLI_EFMT, f"no element type for {t.dtype}")
    return d


def _elsewhere(t, dev: int, name: str):
    if not t.is_cuda:
        _refuse(f"{name} must be a CUDA tensor")
    raise ColiError(COLI_EDEVICE, f"{name} lives on device {t.get_device()} but device {dev} is current")


def _packed(t, kind, dev: int, name: str) -> int:
    """Address of t, a contiguous tensor of torch type `kind` on device dev."""
    if t.get_device() != dev:
        _elsewhere(t, dev, name)
    if t.dtype is not kind or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous {kind} CUDA tensor")
    return t.data_ptr()


def _rows3(t, dev: int, name: str) -> int:
    """Stride of the rows of t [T, heads, n]: rows of one stride over tokens and heads, elements packed."""
    if t.get_device() != dev:
        _elsewhere(t, dev, name)
    T, H, n = t.shape
    s0, s1, s2 = t.stride()
    ld = s1 if H > 1 else s0 if T > 1 else n
    if (n > 1 and s2 != 1) or (T > 1 and s0 != H * ld):
        _refuse(f"{name} must be a CUDA tensor whose [tokens, heads] rows have one stride")
    return ld


def _tokens(t, dev: int, name: str) -> int:
    """Token stride of t [T, ...] whose tokens are packed."""
    if t.get_device() != dev:
        _elsewhere(t, dev, name)
    shape, stride, n = t.shape, t.stride(), 1
    for i in range(len(shape) - 1, 0, -1):
        if stride[i] != n and shape[i] != 1:
            _refuse(f"a token of {name} must be packed")
        n *= shape[i]
    return stride[0] if shape[0] > 1 else n


def _heads(t, shape, kind, dev: int, name: str) -> int:
    """Token stride of t, of this shape [T, heads, dim] and type, whose tokens are packed."""
    if t.shape != shape or t.dtype is not kind:
        _refuse(f"{name} must be a {kind} tensor of shape {tuple(shape)}")
    if t.get_device() != dev:
        _elsewhere(t, dev, name)
    T, H, D = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or s1 != D:
        return _tokens(t, dev, name)         # single heads or tokens, whose strides mean nothing, or a refusal
    return s0 if T > 1 else H * D


def _pages(pages, n_seq: int, dev: int, name: str = "pages") -> int:
    n, width = pages.shape
    if pages.get_device() != dev:
        _elsewhere(pages, dev, name)
    if pages.dtype is not _torch.int32 or n != n_seq or (width > 1 and pages.stride(1) != 1):
        _refuse(f"{name} must be an int32 CUDA tensor [n_seq, n] with packed rows")
    return pages.stride(0) if n > 1 else width


class MlaCache:
    """The paged latent cache of coli.h's coli_mla_cache over the caller's
    tensors: rows [n_pages, page_size, latent + rope] bfloat16, or float8_e4m3fn
    with scales float32 [n_pages, page_size].  Keeps the tensors alive."""

    def __init__(self, rows, latent: int, rope: int, scales=None):
        d = _dtype(rows)
        if rows.dim() != 3 or not rows.is_contiguous() or not rows.is_cuda or rows.shape[2] != latent + rope:
            _refuse("rows must be a contiguous CUDA tensor [n_pages, page_size, latent + rope]")
        if d == COLI_E4M3:
            if scales is None or scales.shape != rows.shape[:2]:
                _refuse("an e4m3 cache needs scales [n_pages, page_size]")
            _packed(scales, _torch.float32, rows.get_device(), "scales")
        elif scales is not None:
            _refuse("only an e4m3 cache has scales")
        self.rows, self.scales, self.device = rows, scales, rows.get_device()
        self.latent, self.rope, self.page_size, self.n_pages = int(latent), int(rope), rows.shape[1], rows.shape[0]
        self._c = _MlaCache(d, self.latent, self.rope, self.page_size, self.n_pages, rows.data_ptr(), _ptr(scales))
        self._p = ctypes.addressof(self._c)



def mla_query(q, pos, rot, out_nope, out_rope, interleaved: bool = False, stream=None):
    """Split q [T, heads, nope + rope] into out_nope [T, heads, nope] and the rotated out_rope [T, heads, rope]
    (f32 or bf16 each, possibly two parts of one tensor; out_nope None: nope = 0).  rot [n_pos, rope] = cos | sin."""
    torch = _torch or _load_torch()
    dev = _device()
    T, H, n = q.shape
    T2, H2, R = out_rope.shape
    n_pos, R2 = rot.shape
    N = n - R
    if q.dtype is not torch.float32 or T2 != T or H2 != H or pos.shape[0] != T or R2 != R or \
            (N != 0 if out_nope is None else out_nope.shape != (T, H, N)):
        _refuse("mla_query: q must be float32 [T, heads, nope + rope] and the others must match it")
    if out_nope is None:
        dn = pn = ln = 0
    else:
        dn, pn, ln = _dtype(out_nope), out_nope.data_ptr(), _rows3(out_nope, dev, "out_nope")
    rc = _lib.coli_mla_query(q.data_ptr(), _tokens(q, dev, "q"), T, H, N, R, _packed(pos, torch.int32, dev, "pos"),
                             _packed(rot, torch.float32, dev, "rot"), n_pos, interleaved, dn, pn, ln, _dtype(out_rope),
                             out_rope.data_ptr(), _rows3(out_rope, dev, "out_rope"), _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return out_nope, out_rope


def mla_append(cache: MlaCache, kv, norm, eps: float, pos, rot, slots, interleaved: bool = False, stream=None):
    """Norm (norm None: none), rotate, quantise and store kv [T, latent + rope] at slots [T] of the cache."""
    torch = _torch or _load_torch()
    dev = _device()
    if cache.device != dev:
        _elsewhere(cache.rows, dev, "the cache")
    T, n = kv.shape
    n_pos, R = rot.shape
    if kv.dtype is not torch.float32 or n != cache.latent + R or R != cache.rope or pos.shape[0] != T or \
            slots.shape[0] != T or (norm is not None and norm.shape[0] != cache.latent):
        _refuse("mla_append: kv must be float32 [T, latent + rope] and the others must match it and the cache")
    rc = _lib.coli_mla_append(cache._p, kv.data_ptr(), _tokens(kv, dev, "kv"), T,
                              None if norm is None else _packed(norm, torch.float32, dev, "norm"), eps,
                              _packed(pos, torch.int32, dev, "pos"), _packed(rot, torch.float32, dev, "rot"), n_pos, interleaved,
                              _packed(slots, torch.int64, dev, "slots"), _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)


def mla_read(cache: MlaCache, pages, cu, out, stream=None):
    """Read the first cu[b+1] - cu[b] tokens of each sequence b back into out [T, latent + rope] (f32 or bf16)."""
    torch = _torch or _load_torch()
    dev = _device()
    if cache.device != dev:
        _elsewhere(cache.rows, dev, "the cache")
    n_seq = cu.shape[0] - 1
    T, n = out.shape
    if n != cache.latent + cache.rope:
        _refuse("mla_read: out must have latent + rope columns")
    rc = _lib.coli_mla_read(cache._p, pages.data_ptr(), _pages(pages, n_seq, dev), n_seq, _packed(cu, torch.int32, dev, "cu"), T,
                            _dtype(out), out.data_ptr(), _tokens(out, dev, "out"), _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return out


def mla_attend(cache: MlaCache, q_latent, q_rope, pages, lens, scale: float, out, lse=None, stream=None):
    """Absorbed attention of q_latent [n_seq, n_q, heads, latent] and q_rope [n_seq, n_q, heads, rope] over the cached
    tokens (lens [n_seq] int32, the new ones included) into out [n_seq, n_q, heads, latent]; lse f32 [n_seq, n_q, heads]."""
    torch = _torch or _load_torch()
    dev = _device()
    if cache.device != dev:
        _elsewhere(cache.rows, dev, "the cache")
    B, n_q, H, n = q_latent.shape
    kind = q_latent.dtype
    if n != cache.latent or q_rope.shape != (B, n_q, H, cache.rope) or out.shape != q_latent.shape or \
            lens.shape[0] != B or (lse is not None and lse.shape != (B, n_q, H)):
        _refuse("mla_attend: q_latent, q_rope, lens, out and lse must match one another and the cache")
    rc = _lib.coli_mla_attend(cache._p, _dtype(q_latent), _packed(q_latent, kind, dev, "q_latent"), _packed(q_rope, kind, dev, "q_rope"),
                              B, n_q, H, pages.data_ptr(), _pages(pages, B, dev), _packed(lens, torch.int32, dev, "lens"), scale,
                              _dtype(out), _packed(out, out.dtype, dev, "out"),
                              None if lse is None else _packed(lse, torch.float32, dev, "lse"), _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return out


def mla_prefill(q, kv, k_rope, cu_q, cu_k, scale: float, out, lse=None, stream=None):
    """Causal attention of packed sequences: q [Tq, heads, nope + rope], kv [Tk, heads, nope + v], k_rope [Tk, rope]
    (all bf16 or all f32) into out [Tq, heads, v]; cu_q, cu_k int32 [n_seq + 1]; lse f32 [Tq, heads]."""
    torch = _torch or _load_torch()
    dev = _device()
    Tq, H, dk = q.shape
    Tk, R = k_rope.shape
    V = out.shape[2]
    N = dk - R
    if kv.shape != (Tk, H, N + V) or out.shape != (Tq, H, V) or cu_q.shape != cu_k.shape or kv.dtype is not q.dtype or \
            k_rope.dtype is not q.dtype or (lse is not None and lse.shape != (Tq, H)):
        _refuse("mla_prefill: q, kv, k_rope, cu_q, cu_k, out and lse must match one another")
    rc = _lib.coli_mla_prefill(_dtype(q), q.data_ptr(), _tokens(q, dev, "q"), kv.data_ptr(), _tokens(kv, dev, "kv"), k_rope.data_ptr(),
                               _tokens(k_rope, dev, "k_rope"), Tq, Tk, cu_q.shape[0] - 1, _packed(cu_q, torch.int32, dev, "cu_q"),
                               _packed(cu_k, torch.int32, dev, "cu_k"), H, N, R, V, scale, _dtype(out),
                               _packed(out, out.dtype, dev, "out"), None if lse is None else _packed(lse, torch.float32, dev, "lse"),
                               _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return out


class GqaCache:
    """The paged 4-bit cache of coli.h's coli_gqa_cache over the caller's tensors: k and v uint8 [n_pages, n_kv,
    page_size, dim / 2], k_scales and v_scales bfloat16 [n_pages, n_kv, page_size, dim / gs], weights float32 [n_pages,
    n_kv, page_size] or None.  Keeps the tensors alive."""

    def __init__(self, k, v, k_scales, v_scales, weights=None):
        torch = _torch or _load_torch()
        if k.dim() != 4 or v.shape != k.shape or k_scales.dim() != 4 or k_scales.shape[:3] != k.shape[:3] or \
                v_scales.shape != k_scales.shape or (weights is not None and weights.shape != k.shape[:3]):
            _refuse("k, v must be [n_pages, n_kv, page_size, dim / 2], the scales [n_pages, n_kv, page_size, dim / gs], "
                    "weights [n_pages, n_kv, page_size]")
        dim, groups = 2 * k.shape[3], k_scales.shape[3]
        if not k.is_cuda or groups < 1 or dim % groups:
            _refuse("k must be a CUDA tensor and a row must have whole scale groups")
        dev = k.get_device()
        at = [_packed(k, torch.uint8, dev, "k"), _packed(v, torch.uint8, dev, "v"), _packed(k_scales, torch.bfloat16, dev, "k_scales"),
              _packed(v_scales, torch.bfloat16, dev, "v_scales"), None if weights is None else _packed(weights, torch.float32, dev, "weights")]
        self.k, self.v, self.k_scales, self.v_scales, self.weights, self.device = k, v, k_scales, v_scales, weights, dev
        self.n_pages, self.n_kv, self.page_size, self.dim, self.gs = k.shape[0], k.shape[1], k.shape[2], dim, dim // groups
        self._c = _GqaCache(self.n_kv, self.dim, self.gs, self.page_size, self.n_pages, *at)
        self._p = ctypes.addressof(self._c)


def gqa_prefill(q, k, v, cu_q, cu_k, scale: float, out, lse=None, stream=None):
    """Causal attention of packed sequences: q [Tq, heads, dim], k and v [Tk, kv heads, dim] (all bf16 or all f32) into
    out [Tq, heads, dim]; cu_q, cu_k int32 [n_seq + 1]; lse f32 [Tq, heads]."""
    torch = _torch or _load_torch()
    dev = _device()
    kind, shape, kv_shape = q.dtype, q.shape, k.shape
    Tq, H, D = shape
    Tk, K, D2 = kv_shape
    n = cu_q.shape
    if D2 != D or out.shape != shape or cu_k.shape != n or (lse is not None and lse.shape != (Tq, H)):
        _refuse("gqa_prefill: q, k, v, cu_q, cu_k, out and lse must match one another")
    rc = _lib.coli_gqa_prefill(_dtype(q), q.data_ptr(), _heads(q, shape, kind, dev, "q"), k.data_ptr(), _heads(k, kv_shape, kind, dev, "k"),
                               v.data_ptr(), _heads(v, kv_shape, kind, dev, "v"), Tq, Tk, n[0] - 1, _packed(cu_q, torch.int32, dev, "cu_q"),
                               _packed(cu_k, torch.int32, dev, "cu_k"), H, K, D, scale, _dtype(out), _packed(out, out.dtype, dev, "out"),
                               None if lse is None else _packed(lse, torch.float32, dev, "lse"),
                               _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return out


def gqa_append(cache: GqaCache, k, v, slots, stream=None):
    """Quantise and store k and v [T, kv heads, dim] (both f32 or both bf16) at slots [T] of the cache."""
    torch = _torch or _load_torch()
    dev = _device()
    if cache.device != dev:
        _elsewhere(cache.k, dev, "the cache")
    kind, (T,) = k.dtype, slots.shape
    shape = (T, cache.n_kv, cache.dim)
    rc = _lib.coli_gqa_append(cache._p, _dtype(k), k.data_ptr(), _heads(k, shape, kind, dev, "k"), v.data_ptr(),
                              _heads(v, shape, kind, dev, "v"), T, _packed(slots, torch.int64, dev, "slots"),
                              _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)


def gqa_read(cache: GqaCache, pages, cu, k, v, stream=None):
    """Read the first cu[b+1] - cu[b] tokens of each sequence b back into k and v [T, kv heads, dim] (both f32 or both bf16)."""
    torch = _torch or _load_torch()
    dev = _device()
    if cache.device != dev:
        _elsewhere(cache.k, dev, "the cache")
    n_seq, kind, T = cu.shape[0] - 1, k.dtype, k.shape[0]
    shape = (T, cache.n_kv, cache.dim)
    rc = _lib.coli_gqa_read(cache._p, pages.data_ptr(), _pages(pages, n_seq, dev), n_seq, _packed(cu, torch.int32, dev, "cu"), T,
                            _dtype(k), k.data_ptr(), _heads(k, shape, kind, dev, "k"), v.data_ptr(), _heads(v, shape, kind, dev, "v"),
                            _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return k, v


def gqa_attend(cache: GqaCache, q, pages, lens, scale: float, out, lse=None, weigh: bool = False, stream=None):
    """Attention of q [n_seq, n_q, heads, dim] over the cached tokens (lens [n_seq] int32, the new ones included) into out
    of the same shape; lse f32 [n_seq, n_q, heads].  weigh: each cached row's share is added to the cache's weights."""
    torch = _torch or _load_torch()
    dev = _device()
    if cache.device != dev:
        _elsewhere(cache.k, dev, "the cache")
    shape = q.shape
    B, n_q, H, D = shape
    if D != cache.dim or out.shape != shape or lens.shape != (B,) or (lse is not None and lse.shape != (B, n_q, H)):
        _refuse("gqa_attend: q, lens, out and lse must match one another and the cache")
    rc = _lib.coli_gqa_attend(cache._p, _dtype(q), _packed(q, q.dtype, dev, "q"), B, n_q, H, pages.data_ptr(), _pages(pages, B, dev),
                              _packed(lens, torch.int32, dev, "lens"), scale, weigh, _dtype(out), _packed(out, out.dtype, dev, "out"),
                              None if lse is None else _packed(lse, torch.float32, dev, "lse"),
                              _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return out


def gqa_evict(cache: GqaCache, pages, lens, keep: int, recent: int, dst, kept, new_lens, stream=None):
    """Choose the min(keep, lens[b]) tokens of each sequence and head that stay (the newest `recent` and the most weighted
    others) and write them to the sequence's new pages dst; kept int32 [n_seq, kv heads, keep], new_lens int32 [n_seq]."""
    torch = _torch or _load_torch()
    dev = _device()
    if cache.device != dev:
        _elsewhere(cache.k, dev, "the cache")
    B = lens.shape[0]
    if kept.shape != (B, cache.n_kv, keep) or new_lens.shape != (B,):
        _refuse("gqa_evict: kept must be [n_seq, kv heads, keep], new_lens [n_seq]")
    rc = _lib.coli_gqa_evict(cache._p, pages.data_ptr(), _pages(pages, B, dev), B, _packed(lens, torch.int32, dev, "lens"), keep, recent,
                             dst.data_ptr(), _pages(dst, B, dev, "dst"), _packed(kept, torch.int32, dev, "kept"),
                             _packed(new_lens, torch.int32, dev, "new_lens"), _raw_stream(dev) if stream is None else _stream(stream))
    if rc:
        _check(rc)
    return kept, new_lens


def sync_check(stream=None):
    _check(_lib.coli_sync_check(_stream(stream)))


def stats() -> dict:
    s = _Stats()
    _lib.coli_get_stats(ctypes.byref(s))
    return dict(calls=s.calls, launches=s.launches, weight_bytes=s.weight_bytes)


def reset_stats():
    _lib.coli_reset_stats()


def set_fail_after(n: int):
    _lib.coli_set_fail_after(int(n))


def set_wait_limit(ns: int):
    """Bound of each device-side wait of the attention kernels (ns <= 0: the default, 2 s)."""
    _lib.coli_set_wait_limit(int(ns))


def last_error() -> str:
    return _lib.coli_last_error().decode()
