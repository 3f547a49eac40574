"""NVFP4 weight x bf16 activation matrix-vector products on MI355X (gfx950).

A thin ctypes binding over ``libnvfp4.so``, whose C ABI is declared in
``include/nvfp4.h``.  Every function below has the name of the C entry point
it calls and only marshals arguments: torch tensors in device memory become
raw pointers, and the current torch stream of the tensors' device becomes
the HIP stream.  All arithmetic runs in the library's HIP kernels; if the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

__all__ = [
    "NVFP4Error", "library_path", "load",
    "nvfp4_strerror", "nvfp4_repacked_code_bytes", "nvfp4_repacked_scale_bytes",
    "nvfp4_quantize", "nvfp4_repack", "nvfp4_dequant", "nvfp4_gemv",
    "nvfp4_gemv_argmax_workspace_bytes", "nvfp4_gemv_argmax", "nvfp4_gemv_argmax_noalloc", "nvfp4_swiglu",
    "nvfp4_gemv_swiglu", "nvfp4_gemv_batch", "nvfp4_gemv_batch_workspace_bytes", "NVFP4_MAX_BATCH",
    "mxfp4_repacked_code_bytes", "mxfp4_repacked_scale_bytes", "mxfp4_quantize", "mxfp4_repack",
    "mxfp4_dequant", "mxfp4_gemv",
    "alloc_repacked", "alloc_mx_repacked",
    "NVFP4_KV_MXFP4", "NVFP4_KV_MXFP8", "KvCache", "KvBatch", "alloc_kv_cache", "nvfp4_kv_code_bytes",
    "nvfp4_kv_scale_bytes", "nvfp4_kv_append", "nvfp4_kv_read", "nvfp4_kv_attention_workspace_bytes",
    "nvfp4_kv_attention",
    "nvfp4_rope", "NVFP4_MAX_ROPE",
    "nvfp4_kv_weights", "nvfp4_kv_evict",
    "nvfp4_logprobs_workspace_bytes", "nvfp4_logprobs", "NVFP4_MAX_TOP",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libnvfp4.so")
_lock = threading.Lock()
_lib = None

NVFP4_MAX_N = 65536
NVFP4_MAX_BATCH = 4
NVFP4_MAX_ROPE = 4
NVFP4_MAX_TOP = 64
NVFP4_KV_MXFP4 = 4
NVFP4_KV_MXFP8 = 8
_KV_DTYPE = {torch.bfloat16: 0, torch.float32: 1}      # NVFP4_KV_BF16, NVFP4_KV_F32


class _Product(ctypes.Structure):
    """struct nvfp4_product of nvfp4.h."""
    _fields_ = [("wq", ctypes.c_void_p), ("ws", ctypes.c_void_p), ("tscale", ctypes.c_float),
                ("rows", ctypes.c_int64), ("y", ctypes.c_void_p), ("argmax", ctypes.c_void_p)]


class _KvCache(ctypes.Structure):
    """struct nvfp4_kv_cache of nvfp4.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] +
                [(n, ctypes.c_int32) for n in ("k_format", "v_format", "pages", "page_tokens", "heads", "head_dim")])


class _KvBatch(ctypes.Structure):
    """struct nvfp4_kv_batch of nvfp4.h."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("page_table", "offsets", "past")] + [("tokens", ctypes.c_int64)] +
                [(n, ctypes.c_int32) for n in ("seqs", "table_width", "max_new", "max_context")])


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (where, nvfp4_strerror(status), status))


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libnvfp4.so (built by ``python -m block_scaled_bit_nvfp4_amd.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError("libnvfp4.so is not built (%s); run "
                               "`python -m block_scaled_bit_nvfp4_amd.build`" % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        P, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                                ctypes.c_size_t)
        sigs = {
            "nvfp4_strerror": (ctypes.c_char_p, [i32]),
            "nvfp4_repacked_code_bytes": (sz, [i64, i64]),
            "nvfp4_repacked_scale_bytes": (sz, [i64, i64]),
            "nvfp4_quantize": (i32, [P, i64, i64, f32, P, P, P]),
            "nvfp4_repack": (i32, [P, P, i64, i64, P, P, P]),
            "nvfp4_dequant": (i32, [P, P, f32, i64, i64, P, P, P]),
            "nvfp4_gemv": (i32, [P, P, f32, i64, i64, P, i32, P, P]),
            "nvfp4_gemv_argmax_workspace_bytes": (sz, [i64, i64, i32]),
            "nvfp4_gemv_argmax": (i32, [P, P, f32, i64, i64, P, i32, P, P, P, sz, P]),
            "nvfp4_gemv_argmax_noalloc": (i32, [P, P, f32, i64, i64, P, i32, P, P, P]),
            "nvfp4_swiglu": (i32, [P, i64, i32, P, P]),
            "nvfp4_gemv_swiglu": (i32, [P, P, f32, i64, i64, P, i32, P, P, P]),
            "nvfp4_gemv_batch_workspace_bytes": (sz, [P, i32, i64, i32]),
            "nvfp4_gemv_batch": (i32, [P, i32, i64, P, i32, P, sz, P]),
            "mxfp4_repacked_code_bytes": (sz, [i64, i64]),
            "mxfp4_repacked_scale_bytes": (sz, [i64, i64]),
            "mxfp4_quantize": (i32, [P, i64, i64, f32, P, P, P]),
            "mxfp4_repack": (i32, [P, P, i64, i64, P, P, P]),
            "mxfp4_dequant": (i32, [P, P, f32, i64, i64, P, P, P]),
            "mxfp4_gemv": (i32, [P, P, f32, i64, i64, P, i32, P, P]),
            "nvfp4_kv_code_bytes": (sz, [i32, i32, i32, i32, i32]),
            "nvfp4_kv_scale_bytes": (sz, [i32, i32, i32, i32, i32]),
            "nvfp4_kv_append": (i32, [P, P, i32, P, i64, P, i64, P]),
            "nvfp4_kv_read": (i32, [P, P, i32, P, i64, P, i64, P]),
            "nvfp4_kv_attention_workspace_bytes": (sz, [P, P, i32]),
            "nvfp4_kv_attention": (i32, [P, P, P, i64, i32, f32, i32, P, P, i64, P, P, sz, P]),
            "nvfp4_rope": (i32, [P, i32, i32, i64, i32, i32, i32, P, i32, P, P, f32, P]),
            "nvfp4_kv_weights": (i32, [P, P, P, i64, i32, f32, i32, P, P, f32, P, i64, P]),
            "nvfp4_kv_evict": (i32, [P, P, i32, i32, i32, P, P, i64, P, P, P]),
            "nvfp4_logprobs_workspace_bytes": (sz, [i64, i64, i32]),
            "nvfp4_logprobs": (i32, [i32, P, i64, i64, i64, f32, P, i32, P, P, P, i32, P, P, P, sz, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_BF16 = (torch.bfloat16, torch.int16)      # bf16 values or their bit patterns
_I32 = (torch.int32,)
_ANY = None


def _checked(*specs):
    """Validate the tensors of one call before any pointer reaches the
    library: each spec is (name, tensor, allowed dtypes or None, least byte
    count, may be None).  A tensor must be a contiguous torch.Tensor of an
    allowed dtype holding at least the bytes the call's shape implies, and all
    tensors must sit on one GPU (checked after the rest).  Raises TypeError or
    ValueError; does no arithmetic on the data."""
    device = None
    for name, t, dtypes, nbytes, optional in specs:
        if t is None:
            if optional:
                continue
            raise ValueError("%s is required" % name)
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s: expected a torch.Tensor, got %r" % (name, type(t)))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
        if dtypes is not None and t.dtype not in dtypes:
            raise ValueError("%s: dtype %s, expected %s" % (name, t.dtype, " or ".join(map(str, dtypes))))
        have = t.numel() * t.element_size()
        if nbytes > 0 and have < nbytes:
            raise ValueError("%s holds %d bytes, the call needs %d" % (name, have, nbytes))
    for name, t, _, _, _ in specs:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("%s must be in GPU memory (is on %s)" % (name, t.device))
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError("%s is on %s, other arguments on %s" % (name, t.device, device))


def _prod(*v):
    out = 1
    for x in v:
        out *= int(x)
    return out


def _stream(stream, *tensors):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise NVFP4Error(status, where)


def nvfp4_strerror(status: int) -> str:
    return load().nvfp4_strerror(int(status)).decode()


def nvfp4_repacked_code_bytes(rows: int, cols: int) -> int:
    return int(load().nvfp4_repacked_code_bytes(rows, cols))


def nvfp4_repacked_scale_bytes(rows: int, cols: int) -> int:
    return int(load().nvfp4_repacked_scale_bytes(rows, cols))


def nvfp4_gemv_argmax_workspace_bytes(rows: int, cols: int, n: int) -> int:
    return int(load().nvfp4_gemv_argmax_workspace_bytes(rows, cols, n))


def _planes(wq, ws, rows, cols, mx=False):
    nq = (mxfp4_repacked_code_bytes if mx else nvfp4_repacked_code_bytes)(rows, cols)
    ns = (mxfp4_repacked_scale_bytes if mx else nvfp4_repacked_scale_bytes)(rows, cols)
    return ("wq", wq, _U8, nq, False), ("ws", ws, _U8, ns, False)


def nvfp4_quantize(W, rows, cols, tscale, codes, scales, stream=None):
    _checked(("W", W, _F32, 4 * _prod(rows, cols), False),
             ("codes", codes, _U8, _prod(rows, cols) // 2, False),
             ("scales", scales, _U8, _prod(rows, cols) // 16, False))
    _check(load().nvfp4_quantize(_ptr(W), rows, cols, float(tscale), _ptr(codes), _ptr(scales),
                                 _stream(stream, W)), "nvfp4_quantize")


def nvfp4_repack(codes, scales, rows, cols, wq, ws, stream=None):
    _checked(("codes", codes, _U8, _prod(rows, cols) // 2, False),
             ("scales", scales, _U8, _prod(rows, cols) // 16, False), *_planes(wq, ws, rows, cols))
    _check(load().nvfp4_repack(_ptr(codes), _ptr(scales), rows, cols, _ptr(wq), _ptr(ws),
                               _stream(stream, codes)), "nvfp4_repack")


def nvfp4_dequant(wq, ws, tscale, rows, cols, out_f32=None, out_bf16=None, stream=None):
    _checked(*_planes(wq, ws, rows, cols), ("out_f32", out_f32, _F32, 4 * _prod(rows, cols), True),
             ("out_bf16", out_bf16, _BF16, 2 * _prod(rows, cols), True))
    _check(load().nvfp4_dequant(_ptr(wq), _ptr(ws), float(tscale), rows, cols, _ptr(out_f32),
                                _ptr(out_bf16), _stream(stream, wq)), "nvfp4_dequant")


def nvfp4_gemv(wq, ws, tscale, rows, cols, X, n, Y, stream=None):
    _checked(*_planes(wq, ws, rows, cols), ("X", X, _BF16, 2 * _prod(n, cols), False),
             ("Y", Y, _F32, 4 * _prod(n, rows), False))
    _check(load().nvfp4_gemv(_ptr(wq), _ptr(ws), float(tscale), rows, cols, _ptr(X), int(n), _ptr(Y),
                             _stream(stream, wq)), "nvfp4_gemv")


def nvfp4_gemv_argmax(wq, ws, tscale, rows, cols, X, n, logits, argmax, workspace, stream=None):
    _checked(*_planes(wq, ws, rows, cols), ("X", X, _BF16, 2 * _prod(n, cols), False),
             ("logits", logits, _F32, 4 * _prod(n, rows), True), ("argmax", argmax, _I32, 4 * int(n), False),
             ("workspace", workspace, _ANY, 0, False))
    nbytes = workspace.numel() * workspace.element_size()
    _check(load().nvfp4_gemv_argmax(_ptr(wq), _ptr(ws), float(tscale), rows, cols, _ptr(X), int(n),
                                    _ptr(logits), _ptr(argmax), _ptr(workspace), nbytes,
                                    _stream(stream, wq)), "nvfp4_gemv_argmax")


def nvfp4_gemv_argmax_noalloc(wq, ws, tscale, rows, cols, X, n, logits, argmax, stream=None):
    _checked(*_planes(wq, ws, rows, cols), ("X", X, _BF16, 2 * _prod(n, cols), False),
             ("logits", logits, _F32, 4 * _prod(n, rows), True), ("argmax", argmax, _I32, 4 * int(n), False))
    _check(load().nvfp4_gemv_argmax_noalloc(_ptr(wq), _ptr(ws), float(tscale), rows, cols, _ptr(X), int(n),
                                            _ptr(logits), _ptr(argmax), _stream(stream, wq)),
           "nvfp4_gemv_argmax_noalloc")


def nvfp4_swiglu(gu, F, n, h, stream=None):
    _checked(("gu", gu, _F32, 8 * _prod(n, F), False), ("h", h, _BF16, 2 * _prod(n, F), False))
    _check(load().nvfp4_swiglu(_ptr(gu), int(F), int(n), _ptr(h), _stream(stream, gu)), "nvfp4_swiglu")


def nvfp4_gemv_swiglu(wq_gu, ws_gu, tscale, hidden, F, X, n, gu, h, stream=None):
    _checked(*_planes(wq_gu, ws_gu, 2 * int(F), hidden), ("X", X, _BF16, 2 * _prod(n, hidden), False),
             ("gu", gu, _F32, 8 * _prod(n, F), True), ("h", h, _BF16, 2 * _prod(n, F), False))
    _check(load().nvfp4_gemv_swiglu(_ptr(wq_gu), _ptr(ws_gu), float(tscale), int(hidden), int(F), _ptr(X),
                                    int(n), _ptr(gu), _ptr(h), _stream(stream, wq_gu)), "nvfp4_gemv_swiglu")


def _batch(products, cols, n, X=None, workspace=None):
    """Product descriptions (dicts with wq, ws, tscale, rows and optional y,
    argmax) -> (ctypes array of nvfp4_product, count), after the same tensor
    checks as the single-product calls."""
    products = list(products)
    specs = []
    for i, q in enumerate(products):
        rows = int(q["rows"])
        wq, ws = _planes(q["wq"], q["ws"], rows, cols)
        specs += [("products[%d].wq" % i,) + wq[1:], ("products[%d].ws" % i,) + ws[1:],
                  ("products[%d].y" % i, q.get("y"), _F32, 4 * _prod(n, rows), True),
                  ("products[%d].argmax" % i, q.get("argmax"), _I32, 4 * int(n), True)]
    if X is not None:
        specs.append(("X", X, _BF16, 2 * _prod(n, cols), False))
    specs.append(("workspace", workspace, _ANY, 0, True))
    _checked(*specs)
    arr = (_Product * max(1, len(products)))()
    for i, q in enumerate(products):
        arr[i] = _Product(_ptr(q["wq"]), _ptr(q["ws"]), float(q["tscale"]), int(q["rows"]), _ptr(q.get("y")),
                          _ptr(q.get("argmax")))
    return arr, len(products)


def nvfp4_gemv_batch_workspace_bytes(products, cols, n) -> int:
    arr, count = _batch(products, cols, n)
    return int(load().nvfp4_gemv_batch_workspace_bytes(arr, count, int(cols), int(n)))


def nvfp4_gemv_batch(products, cols, X, n, workspace=None, stream=None):
    """Several products of one X in one launch (nvfp4_gemv_batch); products:
    dicts with wq, ws, tscale, rows, and y and/or argmax tensors."""
    arr, count = _batch(products, cols, n, X, workspace)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(load().nvfp4_gemv_batch(arr, count, int(cols), _ptr(X), int(n), _ptr(workspace), nbytes,
                                   _stream(stream, X)), "nvfp4_gemv_batch")


def alloc_repacked(rows: int, cols: int, device="cuda"):
    """Allocate (uninitialised) code and scale planes for nvfp4_repack."""
    nq, ns = nvfp4_repacked_code_bytes(rows, cols), nvfp4_repacked_scale_bytes(rows, cols)
    if nq == 0:
        raise NVFP4Error(-2, "alloc_repacked")
    return (torch.empty(nq, dtype=torch.uint8, device=device),
            torch.empty(ns, dtype=torch.uint8, device=device))


# ------------------------------------------------------------------- MXFP4 --

def mxfp4_repacked_code_bytes(rows: int, cols: int) -> int:
    return int(load().mxfp4_repacked_code_bytes(rows, cols))


def mxfp4_repacked_scale_bytes(rows: int, cols: int) -> int:
    return int(load().mxfp4_repacked_scale_bytes(rows, cols))


def mxfp4_quantize(W, rows, cols, tscale, codes, scales, stream=None):
    _checked(("W", W, _F32, 4 * _prod(rows, cols), False),
             ("codes", codes, _U8, _prod(rows, cols) // 2, False),
             ("scales", scales, _U8, _prod(rows, cols) // 32, False))
    _check(load().mxfp4_quantize(_ptr(W), rows, cols, float(tscale), _ptr(codes), _ptr(scales),
                                 _stream(stream, W)), "mxfp4_quantize")


def mxfp4_repack(codes, scales, rows, cols, wq, ws, stream=None):
    _checked(("codes", codes, _U8, _prod(rows, cols) // 2, False),
             ("scales", scales, _U8, _prod(rows, cols) // 32, False), *_planes(wq, ws, rows, cols, mx=True))
    _check(load().mxfp4_repack(_ptr(codes), _ptr(scales), rows, cols, _ptr(wq), _ptr(ws),
                               _stream(stream, codes)), "mxfp4_repack")


def mxfp4_dequant(wq, ws, tscale, rows, cols, out_f32=None, out_bf16=None, stream=None):
    _checked(*_planes(wq, ws, rows, cols, mx=True), ("out_f32", out_f32, _F32, 4 * _prod(rows, cols), True),
             ("out_bf16", out_bf16, _BF16, 2 * _prod(rows, cols), True))
    _check(load().mxfp4_dequant(_ptr(wq), _ptr(ws), float(tscale), rows, cols, _ptr(out_f32),
                                _ptr(out_bf16), _stream(stream, wq)), "mxfp4_dequant")


def mxfp4_gemv(wq, ws, tscale, rows, cols, X, n, Y, stream=None):
    _checked(*_planes(wq, ws, rows, cols, mx=True), ("X", X, _BF16, 2 * _prod(n, cols), False),
             ("Y", Y, _F32, 4 * _prod(n, rows), False))
    _check(load().mxfp4_gemv(_ptr(wq), _ptr(ws), float(tscale), rows, cols, _ptr(X), int(n), _ptr(Y),
                             _stream(stream, wq)), "mxfp4_gemv")


def alloc_mx_repacked(rows: int, cols: int, device="cuda"):
    """Allocate (uninitialised) MXFP4 code and scale planes for mxfp4_repack."""
    nq, ns = mxfp4_repacked_code_bytes(rows, cols), mxfp4_repacked_scale_bytes(rows, cols)
    if nq == 0:
        raise NVFP4Error(-2, "alloc_mx_repacked")
    return (torch.empty(nq, dtype=torch.uint8, device=device),
            torch.empty(ns, dtype=torch.uint8, device=device))


# ------------------------------------------- paged, quantised key/value cache

def _int32(name, value):
    """value as an int, refused where ctypes would cut it down to another one."""
    value = int(value)
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError("%s is %d, past 32 bits" % (name, value))
    return value


def _kv_shape(format, pages, page_tokens, heads, head_dim):
    return (_int32("format", format), _int32("pages", pages), _int32("page_tokens", page_tokens),
            _int32("heads", heads), _int32("head_dim", head_dim))


def nvfp4_kv_code_bytes(format: int, pages: int, page_tokens: int, heads: int, head_dim: int) -> int:
    return int(load().nvfp4_kv_code_bytes(*_kv_shape(format, pages, page_tokens, heads, head_dim)))


def nvfp4_kv_scale_bytes(format: int, pages: int, page_tokens: int, heads: int, head_dim: int) -> int:
    return int(load().nvfp4_kv_scale_bytes(*_kv_shape(format, pages, page_tokens, heads, head_dim)))


class KvCache:
    """struct nvfp4_kv_cache over four plane tensors (uint8), checked once and
    kept by the caller: each side's planes hold the same number of pages, which
    the key codes' size gives."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, k_format, v_format, page_tokens, heads, head_dim):
        page = nvfp4_kv_code_bytes(k_format, 1, page_tokens, heads, head_dim)
        if page == 0 or nvfp4_kv_code_bytes(v_format, 1, page_tokens, heads, head_dim) == 0:
            raise NVFP4Error(-2, "KvCache")
        _checked(("k_codes", k_codes, _U8, page, False))
        pages = k_codes.numel() // page
        shape = (pages, page_tokens, heads, head_dim)
        _checked(("k_codes", k_codes, _U8, page, False),
                 ("k_scales", k_scales, _U8, nvfp4_kv_scale_bytes(k_format, *shape), False),
                 ("v_codes", v_codes, _U8, nvfp4_kv_code_bytes(v_format, *shape), False),
                 ("v_scales", v_scales, _U8, nvfp4_kv_scale_bytes(v_format, *shape), False))
        self.planes = (k_codes, k_scales, v_codes, v_scales)
        self.device, self._index = k_codes.device, k_codes.get_device()
        self.pages, self.page_tokens, self.heads, self.head_dim = shape
        self.k_format, self.v_format = int(k_format), int(v_format)
        self._c = _KvCache(*[t.data_ptr() for t in self.planes], self.k_format, self.v_format, *shape)
        self._ref = ctypes.addressof(self._c)


class KvBatch:
    """struct nvfp4_kv_batch: the new tokens of a step.  page_table [seqs, width],
    offsets [seqs + 1] and past [seqs] are int32 tensors that the kernels read
    when they run, so a program may keep one KvBatch and change their contents;
    tokens, max_new and max_context are host numbers (bounds, see nvfp4.h)."""

    def __init__(self, page_table, offsets, past, tokens, max_new, max_context):
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be an int32 tensor [seqs, width]")
        seqs, width = page_table.shape
        _checked(("page_table", page_table, _I32, 4, False), ("offsets", offsets, _I32, 4 * (seqs + 1), False),
                 ("past", past, _I32, 4 * seqs, False))
        self.arrays = (page_table, offsets, past)
        self.device, self._index = page_table.device, page_table.get_device()
        self.tokens, self._seqs = int(tokens), seqs
        self.max_new, self.max_context = _int32("max_new", max_new), _int32("max_context", max_context)
        self._c = _KvBatch(*[t.data_ptr() for t in self.arrays], self.tokens, seqs, width, self.max_new,
                           self.max_context)
        self._ref = ctypes.addressof(self._c)


def alloc_kv_cache(pages, page_tokens, heads, head_dim, k_format=NVFP4_KV_MXFP8, v_format=NVFP4_KV_MXFP8,
                   device="cuda"):
    """A KvCache over newly allocated (uninitialised) planes."""
    shape = (pages, page_tokens, heads, head_dim)
    sizes = [nvfp4_kv_code_bytes(k_format, *shape), nvfp4_kv_scale_bytes(k_format, *shape),
             nvfp4_kv_code_bytes(v_format, *shape), nvfp4_kv_scale_bytes(v_format, *shape)]
    if 0 in sizes:
        raise NVFP4Error(-2, "alloc_kv_cache")
    return KvCache(*[torch.empty(n, dtype=torch.uint8, device=device) for n in sizes], k_format, v_format,
                   page_tokens, heads, head_dim)


def _rows(name, t, cache, batch, heads, dtypes):
    """Check a [tokens, heads, head_dim] tensor whose tokens may be strided (the
    heads of a token are not); its token stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: expected a torch.Tensor, got %r" % (name, type(t)))
    if t.dtype not in dtypes:
        raise ValueError("%s: dtype %s, expected %s" % (name, t.dtype, " or ".join(map(str, dtypes))))
    dim, tokens = cache.head_dim, batch.tokens
    if t.shape != (tokens, heads, dim):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (tokens, heads, dim)))
    token, head, element = t.stride()
    if tokens and (element != 1 or (heads > 1 and head != dim)):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    if t.get_device() != cache._index:
        raise ValueError("%s is on %s, the cache on %s" % (name, t.device, cache.device))
    return token if tokens > 1 else heads * dim


def _flat(name, t, cache, dtype, n):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.is_contiguous() and t.numel() >= n and
            t.get_device() == cache._index):
        raise ValueError("%s must be a contiguous %s tensor of %d elements on %s" % (name, dtype, n, cache.device))


# torch's getter of the current stream's handle; its public one builds an object
# around it, 2 us of a call that takes 10.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _kv_stream(stream, cache):
    if stream is None and _raw_stream is not None:
        return _raw_stream(cache._index)
    return _stream(stream, *cache.planes)


def _kv_pair(cache, batch):
    if not isinstance(cache, KvCache) or not isinstance(batch, KvBatch):
        raise TypeError("expected a KvCache and a KvBatch")
    if cache._index != batch._index:
        raise ValueError("the batch is on %s, the cache on %s" % (batch.device, cache.device))


def nvfp4_kv_append(cache, batch, K, V, stream=None):
    _kv_pair(cache, batch)
    ks = _rows("K", K, cache, batch, cache.heads, _KV_DTYPE)
    vs = _rows("V", V, cache, batch, cache.heads, (K.dtype,))
    _check(load().nvfp4_kv_append(cache._ref, batch._ref, _KV_DTYPE[K.dtype], K.data_ptr(), ks, V.data_ptr(), vs,
                                  _kv_stream(stream, cache)), "nvfp4_kv_append")


def nvfp4_kv_read(cache, batch, K=None, V=None, stream=None):
    _kv_pair(cache, batch)
    if K is None and V is None:
        raise ValueError("K or V is required")
    ks = 0 if K is None else _rows("K", K, cache, batch, cache.heads, _KV_DTYPE)
    vs = 0 if V is None else _rows("V", V, cache, batch, cache.heads, _KV_DTYPE)
    dtype = V.dtype if K is None else K.dtype
    if V is not None and V.dtype != dtype:
        raise ValueError("K is %s, V %s" % (dtype, V.dtype))
    _check(load().nvfp4_kv_read(cache._ref, batch._ref, _KV_DTYPE[dtype],
                                None if K is None else K.data_ptr(), ks, None if V is None else V.data_ptr(), vs,
                                _kv_stream(stream, cache)), "nvfp4_kv_read")


def nvfp4_kv_attention_workspace_bytes(cache, batch, q_heads) -> int:
    _kv_pair(cache, batch)
    return int(load().nvfp4_kv_attention_workspace_bytes(cache._ref, batch._ref, _int32("q_heads", q_heads)))


def nvfp4_kv_attention(cache, batch, Q, scale, out, lse=None, window=0, tree=None, workspace=None, stream=None):
    """Attention of the batch's new tokens over the cache: Q and out bfloat16
    [tokens, q_heads, head_dim], lse float32 [tokens, q_heads] or None, tree int64
    [tokens] (bit patterns) or None."""
    _kv_pair(cache, batch)
    heads = Q.shape[1] if isinstance(Q, torch.Tensor) and Q.dim() == 3 else 0
    qs = _rows("Q", Q, cache, batch, heads, _BF16[:1])
    os_ = _rows("out", out, cache, batch, heads, _BF16[:1])
    if lse is not None:
        _flat("lse", lse, cache, torch.float32, batch.tokens * heads)
    if tree is not None:
        _flat("tree", tree, cache, torch.int64, batch.tokens)
    nbytes = 0
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != cache._index:
            raise ValueError("workspace must be contiguous, on %s" % cache.device)
        nbytes = workspace.numel() * workspace.element_size()
    _check(load().nvfp4_kv_attention(cache._ref, batch._ref, Q.data_ptr(), qs, heads, float(scale),
                                     _int32("window", window),
                                     None if tree is None else tree.data_ptr(), out.data_ptr(), os_,
                                     None if lse is None else lse.data_ptr(),
                                     workspace.data_ptr() if nbytes else None, nbytes, _kv_stream(stream, cache)),
           "nvfp4_kv_attention")


# ------------------------------------------------------------ rotary positions

def _device_of(name, t, dtype, index=None):
    """The GPU of a contiguous tensor of a type, the same as an earlier one's."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s tensor" % (name, dtype))
    at = t.get_device()
    if at < 0:
        raise ValueError("%s must be in GPU memory (is on %s)" % (name, t.device))
    if index is not None and at != index:
        raise ValueError("%s is on %s, other arguments on cuda:%d" % (name, t.device, index))
    return at


def _call_stream(stream, index):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(index)
        return torch.cuda.current_stream(index).cuda_stream
    return int(stream)


def _token_stride(name, t, shape, index):
    """Check a [tokens, heads, dim] tensor whose tokens may be strided (the heads of a
    token are not); its token stride in elements."""
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    token, head, element = t.stride()
    tokens, heads, dim = shape
    if tokens and (element != 1 or (heads > 1 and head != dim)):
        raise ValueError("%s: the heads of a token must be contiguous" % name)
    if t.get_device() != index:
        raise ValueError("%s is on %s, the positions on cuda:%d" % (name, t.device, index))
    return token if tokens > 1 else heads * dim


_rope_rows = struct.Struct("QQqqii")         # struct nvfp4_rope_rows of nvfp4.h


def nvfp4_rope(rows, positions, freqs, axis=None, adjacent=False, factor=1.0, stream=None):
    """Rotate rows by their tokens' positions: rows is a list of (in, out) pairs of
    [tokens, heads, head_dim] tensors (all inputs of one type, bfloat16 or float32; out of
    either; a pair of the same tensor is rotated in place), positions int32 [axes, tokens]
    or [tokens], freqs float64 [pairs] (radians for each position), axis uint8 [pairs] or
    None (all pairs follow the first axis)."""
    index = _device_of("positions", positions, torch.int32)
    _device_of("freqs", freqs, torch.float64, index)
    pairs = freqs.numel()
    if axis is not None:
        _device_of("axis", axis, torch.uint8, index)
        if axis.numel() != pairs:
            raise ValueError("axis has %d elements, freqs %d" % (axis.numel(), pairs))
    packed, dtype, first = b"", None, None
    for row in rows:
        if not (isinstance(row, (tuple, list)) and len(row) == 2 and isinstance(row[0], torch.Tensor) and
                isinstance(row[1], torch.Tensor) and row[0].dim() == 3):
            raise ValueError("rows must be a list of (in, out) pairs of [tokens, heads, head_dim] tensors")
        x, out = row
        shape = x.shape
        if first is None:
            first, dtype = shape, x.dtype
            if dtype not in _KV_DTYPE:
                raise ValueError("rows: dtype %s, expected bfloat16 or float32" % dtype)
        elif shape[0] != first[0] or shape[2] != first[2] or x.dtype is not dtype:
            raise ValueError("rows: %s %s beside %s %s" % (tuple(shape), x.dtype, tuple(first), dtype))
        if out.dtype not in _KV_DTYPE:
            raise ValueError("rows: out is %s, expected bfloat16 or float32" % out.dtype)
        packed += _rope_rows.pack(x.data_ptr(), out.data_ptr(), _token_stride("rows in", x, shape, index),
                                  _token_stride("rows out", out, shape, index), shape[1], _KV_DTYPE[out.dtype])
    if first is None:
        raise ValueError("rows is empty")
    tokens, _, dim = first
    if dim > 1024 or pairs > 512:        # before they are cut to 32 bits
        raise NVFP4Error(-2, "nvfp4_rope")
    axes = positions.shape
    if not 1 <= len(axes) <= 2 or axes[-1] != tokens:
        raise ValueError("positions has shape %s, expected ([axes,] %d)" % (tuple(axes), tokens))
    status = (_lib or load()).nvfp4_rope(
        packed, len(packed) // _rope_rows.size, _KV_DTYPE[dtype], tokens, dim, 2 * pairs, 1 if adjacent else 0,
        positions.data_ptr(), axes[0] if len(axes) == 2 else 1, freqs.data_ptr(),
        None if axis is None else axis.data_ptr(), float(factor), _call_stream(stream, index))
    if status:
        raise NVFP4Error(status, "nvfp4_rope")


# ------------------------------------- eviction by gathered attention weight

def _weights(name, t, cache, batch):
    """Check a [seqs, heads, width] tensor of weights; its width."""
    shape = t.shape if isinstance(t, torch.Tensor) else ()
    if not (len(shape) == 3 and shape[0] == batch._seqs and shape[1] == cache.heads and t.dtype is torch.float32 and
            t.is_contiguous() and t.get_device() == cache._index):
        raise ValueError("%s must be a contiguous float32 tensor [%d, %d, width] on %s" % (
            name, batch._seqs, cache.heads, cache.device))
    return shape[2]


def nvfp4_kv_weights(cache, batch, Q, scale, lse, weights, decay=1.0, window=0, tree=None, stream=None):
    """Gather the attention that the cache's keys receive from the batch's new tokens: Q,
    scale, window and tree as nvfp4_kv_attention took them, lse as it gave it; weights
    float32 [seqs, heads, width], width at least the tokens that the page table can name."""
    _kv_pair(cache, batch)
    heads = Q.shape[1] if isinstance(Q, torch.Tensor) and Q.dim() == 3 else 0
    qs = _rows("Q", Q, cache, batch, heads, _BF16[:1])
    _flat("lse", lse, cache, torch.float32, batch.tokens * heads)
    width = _weights("weights", weights, cache, batch)
    if tree is not None:
        _flat("tree", tree, cache, torch.int64, batch.tokens)
    _check((_lib or load()).nvfp4_kv_weights(cache._ref, batch._ref, Q.data_ptr(), qs, heads, float(scale),
                                   _int32("window", window), None if tree is None else tree.data_ptr(),
                                   lse.data_ptr(), float(decay), weights.data_ptr(), width,
                                   _kv_stream(stream, cache)), "nvfp4_kv_weights")


def nvfp4_kv_evict(cache, batch, weights, budget, kept, left, weights_out=None, first=0, recent=0, stream=None):
    """Cut sequences that hold more than `budget` tokens (the batch's `past`) down to it:
    of each head the first `first`, the last `recent` and the keys of the largest weights
    stay, and move to the front.  kept int32 [seqs, heads, budget], left int32 [seqs] (may
    be the batch's past), weights_out as weights, or None: in place."""
    _kv_pair(cache, batch)
    seqs, budget = batch._seqs, _int32("budget", budget)
    width = _weights("weights", weights, cache, batch)
    if weights_out is not None and _weights("weights_out", weights_out, cache, batch) != width:
        raise ValueError("weights_out is %d wide, weights %d" % (weights_out.shape[2], width))
    _flat("kept", kept, cache, torch.int32, seqs * cache.heads * max(budget, 0))
    _flat("left", left, cache, torch.int32, seqs)
    _check((_lib or load()).nvfp4_kv_evict(cache._ref, batch._ref, budget, _int32("first", first), _int32("recent", recent),
                                 weights.data_ptr(), (weights if weights_out is None else weights_out).data_ptr(),
                                 width, kept.data_ptr(), left.data_ptr(), _kv_stream(stream, cache)),
           "nvfp4_kv_evict")


# ---------------------------------------------------------- log probabilities

def nvfp4_logprobs_workspace_bytes(n: int, vocab: int, top: int) -> int:
    return int(load().nvfp4_logprobs_workspace_bytes(int(n), int(vocab), _int32("top", top)))


def _second(name, t, n, dtype, index):
    """The second extent of a contiguous [n, ...] tensor."""
    _device_of(name, t, dtype, index)
    shape = t.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError("%s must be a %s tensor [%d, ...]" % (name, dtype, n))
    return _int32("the extent of %s" % name, shape[1])


def _row_values(name, t, n, index):
    if t is None:
        return None
    _device_of(name, t, torch.float32, index)
    if t.numel() < n:
        raise ValueError("%s holds %d values, the call needs %d" % (name, t.numel(), n))
    return t.data_ptr()


def nvfp4_logprobs(logits, tokens=None, logp=None, lse=None, entropy=None, top_logp=None, top_index=None, scale=1.0,
                   workspace=None, stream=None):
    """Log probabilities of logits [n, vocab] (float32 or bfloat16; rows may be strided):
    logp float32 [n, given] of tokens int32 [n, given], lse and entropy float32 [n], and
    the likeliest tokens top_index int32 [n, top] with top_logp float32 [n, top].  What is
    None is not computed."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits: expected a torch.Tensor, got %r" % type(logits))
    dtype = _KV_DTYPE.get(logits.dtype)
    if dtype is None or logits.dim() != 2:
        raise ValueError("logits must be a float32 or bfloat16 tensor [n, vocab]")
    n, vocab = logits.shape
    stride, element = logits.stride()
    if vocab > 1 and element != 1:
        raise ValueError("the logits of a row must be contiguous")
    index = logits.get_device()
    if index < 0:
        raise ValueError("logits must be in GPU memory (is on %s)" % logits.device)
    if (tokens is None) != (logp is None) or (top_logp is None) != (top_index is None):
        raise ValueError("tokens and logp, and top_logp and top_index, come together")
    given = top = nbytes = 0
    if tokens is not None:
        given = _second("tokens", tokens, n, torch.int32, index)
        if _second("logp", logp, n, torch.float32, index) != given:
            raise ValueError("logp must have the shape of tokens, %s" % (tuple(tokens.shape),))
    if top_index is not None:
        top = _second("top_index", top_index, n, torch.int32, index)
        if _second("top_logp", top_logp, n, torch.float32, index) != top:
            raise ValueError("top_logp must have the shape of top_index, %s" % (tuple(top_index.shape),))
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != index:
            raise ValueError("workspace must be contiguous, on %s" % logits.device)
        nbytes = workspace.numel() * workspace.element_size()
    status = (_lib or load()).nvfp4_logprobs(
        dtype, logits.data_ptr(), n, vocab, stride if n > 1 else vocab, float(scale),
        tokens.data_ptr() if given else None, given, logp.data_ptr() if given else None,
        _row_values("lse", lse, n, index), _row_values("entropy", entropy, n, index), top,
        top_logp.data_ptr() if top else None, top_index.data_ptr() if top else None,
        workspace.data_ptr() if nbytes else None, nbytes, _call_stream(stream, index))
    if status:
        raise NVFP4Error(status, "nvfp4_logprobs")
