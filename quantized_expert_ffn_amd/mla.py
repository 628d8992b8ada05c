"""Binding of the latent-attention entry points (include/coli_mla.h).

Argument marshalling only: each function has the name of the C entry point
it calls, takes sizes and strides from the tensors, checks that they fit each
other, and raises ColiError on a non-zero return.  coli_moe_status() reads
the workspace's device status.

The checks and the call itself run in a CPython module (csrc/mla_bind.cpp),
since most of these kernels take less time than the same checks here; what
does not fit there comes back here, where the checks say what it is.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import torch

from . import _lib, LIB_PATH, ColiError

COLI_BF16, COLI_FP16 = 0, 1
COLI_KV_PLAIN, COLI_KV_E4M3 = 0, 1
COLI_ROPE_PAIRS, COLI_ROPE_HALVES = 0, 1
COLI_MLA_ROPE = 64
COLI_MLA_MAX_ROWS, COLI_MLA_MAX_BATCH, COLI_MLA_MAX_LENGTH = 16384, 4096, 2 ** 31 - 256

MLA_EXPORTS = ("coli_mla_row_bytes", "coli_mla_workspace_bytes", "coli_mla_append", "coli_mla_project",
               "coli_mla_decode", "coli_mla_expand", "coli_mla_prefill")

_TYPES = {torch.bfloat16: COLI_BF16, torch.float16: COLI_FP16, COLI_BF16: COLI_BF16, COLI_FP16: COLI_FP16}
_OF = {COLI_BF16: torch.bfloat16, COLI_FP16: torch.float16}


class coli_mla_dims(ctypes.Structure):
    _fields_ = [
        ("n_heads", ctypes.c_int32), ("rank", ctypes.c_int32), ("nope", ctypes.c_int32), ("v_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32), ("dtype", ctypes.c_int32), ("kv_format", ctypes.c_int32),
        ("rope_style", ctypes.c_int32), ("norm_eps", ctypes.c_float), ("softmax_scale", ctypes.c_float),
    ]


_P, _SZ, _I32, _I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64
_D = ctypes.POINTER(coli_mla_dims)
_sigs = {
    "coli_mla_row_bytes": (_SZ, [_D]),
    "coli_mla_workspace_bytes": (_SZ, [_D, _I32, _I32, _I32]),
    "coli_mla_append": (ctypes.c_int, [_D, _I32, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _I32,
                                       _P, _SZ, _P]),
    "coli_mla_project": (ctypes.c_int, [_I32, _I32, _I32, _I32, _I32, _P, _I64, _I64, _P, _P, _P]),
    "coli_mla_decode": (ctypes.c_int, [_D, _I32, _I32, _P, _P, _P, _P, _I32, _P, _I32, _P, _I32, _P, _P, _P, _SZ,
                                       _P]),
    "coli_mla_expand": (ctypes.c_int, [_D, _I32, _I32, _P, _P, _I32, _P, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "coli_mla_prefill": (ctypes.c_int, [_D, _I32, _I32, _I32, _P, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _P,
                                        _P, _I32, _I32, _P, _P, _P, _SZ, _P]),
}
for _name, (_res, _args) in _sigs.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


# ---------------------------------------------------------------- marshalling
def make_mla_dims(n_heads: int, rank: int, nope: int, v_dim: int, page_size: int, dtype=torch.bfloat16,
                  kv_format: int = COLI_KV_PLAIN, rope_style: int = COLI_ROPE_PAIRS, norm_eps: float = 1e-6,
                  softmax_scale: float | None = None) -> coli_mla_dims:
    """coli_mla_dims; softmax_scale defaults to (nope + 64) ** -0.5."""
    if dtype not in _TYPES:
        raise TypeError(f"dtype {dtype}: expected torch.bfloat16 or torch.float16")
    if softmax_scale is None:
        softmax_scale = (nope + COLI_MLA_ROPE) ** -0.5
    return coli_mla_dims(n_heads, rank, nope, v_dim, page_size, _TYPES[dtype], kv_format, rope_style, norm_eps,
                         softmax_scale)


def _check(rc, where):
    if rc:
        raise ColiError(rc, where)


def _arg(t, dtype, shape, what):
    """Address of a contiguous device tensor of this type and shape."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, dtype, shape, what)
    raise ValueError(f"{what}: must be contiguous")


def _refuse(t, dtype, shape, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{what}: must be a device tensor")


def _strided(t, dtype, shape, what):
    """Address and the first two strides of a device tensor [tokens, heads, width] whose last dimension is dense."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda):
        _refuse(t, dtype, shape, what)
    a, b, c = t.stride()
    if c != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    # the stride of a dimension of one element is never used
    return t.data_ptr(), a if shape[0] > 1 else 0, b if shape[1] > 1 else 0


def _distinct(t, strides, what):
    """An output's elements must not share an address."""
    n, h, width = t.shape
    ts, hs = strides
    if n and h and not ((h == 1 or hs >= width) and (n == 1 or ts >= (h - 1) * hs + width)
                        or (n == 1 or ts >= width) and (h == 1 or hs >= (n - 1) * ts + width)):
        raise ValueError(f"{what}: strides overlap")


def _ws(ws):
    n = ws.numel()
    return _arg(ws, torch.uint8, (n,), "ws"), n


def _load_bind():
    path = os.path.join(os.path.dirname(LIB_PATH), "_mla_bind.so")
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m quantized_expert_ffn_amd.build`")
    spec = importlib.util.spec_from_file_location("_mla_bind", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


_bind = _load_bind()
_at = ctypes.addressof


def _handle(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def _stream(stream, t):
    return torch.cuda.current_stream(t.device).cuda_stream if stream is None else _handle(stream)


def _columns(t, what):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{what}: expected a tensor of two dimensions")
    return t.shape[1]


def _pages(d, pages, kv_scale):
    if d.kv_format == COLI_KV_E4M3:
        dtype, row = torch.uint8, d.rank + 2 * COLI_MLA_ROPE
    else:
        dtype, row = _OF[d.dtype], d.rank + COLI_MLA_ROPE
    n, page = pages.shape[0], d.page_size
    at = _arg(pages, dtype, (n, page, row), "pages")
    if kv_scale is not None:
        kv_scale = _arg(kv_scale, torch.float32, (n * page,), "kv_scale")
    return at, kv_scale, n


# ---------------------------------------------------------------- entry points
def coli_mla_row_bytes(dims) -> int:
    return int(_lib.coli_mla_row_bytes(ctypes.byref(dims)))


def coli_mla_workspace_bytes(dims, batch: int = 0, n_q: int = 1, max_kv: int = 0) -> int:
    """Raises ColiError(COLI_EINVAL) for sizes that no call takes."""
    n = int(_lib.coli_mla_workspace_bytes(ctypes.byref(dims), batch, n_q, max_kv))
    if n == 0:
        raise ColiError(-1, "coli_mla_workspace_bytes")
    return n


def coli_mla_append(dims, kv_a, norm_w, positions, slots, inv_freq, q_pe, q_pe_out, pages, kv_scale, ws, stream=None):
    """norm_w None: the latent is stored as it is.  q_pe and q_pe_out (both may be None): [n, n_heads, 64] views with
    strides of their own; they may be the same tensor."""
    rc = _bind.append(_at(dims), kv_a, norm_w, positions, slots, inv_freq, q_pe, q_pe_out, pages, kv_scale, ws, _handle(stream))
    if rc != 1:
        return _check(rc, "coli_mla_append")
    d, n = dims, kv_a.shape[0]
    dt = _OF[d.dtype]
    q = o = (None, 0, 0)
    if q_pe is not None:
        q = _strided(q_pe, dt, (n, d.n_heads, COLI_MLA_ROPE), "q_pe")
    if q_pe_out is not None:
        o = _strided(q_pe_out, dt, (n, d.n_heads, COLI_MLA_ROPE), "q_pe_out")
        _distinct(q_pe_out, o[1:], "q_pe_out")
    at, scale, n_pages = _pages(d, pages, kv_scale)
    _check(_lib.coli_mla_append(
        ctypes.byref(d), n, _arg(kv_a, dt, (n, d.rank + COLI_MLA_ROPE), "kv_a"),
        None if norm_w is None else _arg(norm_w, dt, (d.rank,), "norm_w"),
        _arg(positions, torch.int32, (n,), "positions"), _arg(slots, torch.int64, (n,), "slots"),
        _arg(inv_freq, torch.float64, (COLI_MLA_ROPE // 2,), "inv_freq"), *q, *o, at, scale, n_pages, *_ws(ws),
        _stream(stream, kv_a)), "coli_mla_append")


def coli_mla_project(x, w, out, stream=None):
    """out[t, h] = w[h] x[t, h]: x [n, heads, n_in] (a view with strides of its own), w [heads, n_out, n_in], out
    [n, heads, n_out]."""
    rc = _bind.project(x, w, out, _handle(stream))
    if rc != 1:
        return _check(rc, "coli_mla_project")
    if x.dtype not in _TYPES:
        raise TypeError(f"x: dtype {x.dtype}, expected torch.bfloat16 or torch.float16")
    n, heads, n_in = x.shape
    n_out = w.shape[1]
    _check(_lib.coli_mla_project(
        _TYPES[x.dtype], n, heads, n_in, n_out, *_strided(x, x.dtype, (n, heads, n_in), "x"),
        _arg(w, x.dtype, (heads, n_out, n_in), "w"), _arg(out, x.dtype, (n, heads, n_out), "out"),
        _stream(stream, x)), "coli_mla_project")


def coli_mla_decode(dims, q_lat, q_pe, pages, kv_scale, table, kv_lens, max_kv, out, lse, ws, stream=None):
    """q_lat [batch * n_q, n_heads, rank]; the batch is kv_lens'.  lse may be None."""
    rc = _bind.decode(_at(dims), q_lat, q_pe, pages, kv_scale, table, kv_lens, max_kv, out, lse, ws, _handle(stream))
    if rc != 1:
        return _check(rc, "coli_mla_decode")
    d, dt, batch, rows = dims, _OF[dims.dtype], kv_lens.shape[0], q_lat.shape[0]
    if batch and (rows % batch or not rows):
        raise ValueError(f"q_lat: {rows} rows for {batch} sequences")
    at, scale, n_pages = _pages(d, pages, kv_scale)
    width = _columns(table, "table")
    _check(_lib.coli_mla_decode(
        ctypes.byref(d), batch, rows // batch if batch else 1, _arg(q_lat, dt, (rows, d.n_heads, d.rank), "q_lat"),
        _arg(q_pe, dt, (rows, d.n_heads, COLI_MLA_ROPE), "q_pe"), at, scale, n_pages,
        _arg(table, torch.int32, (batch, width), "table"), width, _arg(kv_lens, torch.int32, (batch,), "kv_lens"),
        max_kv, _arg(out, dt, (rows, d.n_heads, d.rank), "out"),
        None if lse is None else _arg(lse, torch.float32, (rows, d.n_heads), "lse"), *_ws(ws),
        _stream(stream, q_lat)), "coli_mla_decode")


def coli_mla_expand(dims, pages, kv_scale, table, cu_k, w, kv, k_pe, ws, stream=None):
    rc = _bind.expand(_at(dims), pages, kv_scale, table, cu_k, w, kv, k_pe, ws, _handle(stream))
    if rc != 1:
        return _check(rc, "coli_mla_expand")
    d, dt, n, wide = dims, _OF[dims.dtype], kv.shape[0], dims.nope + dims.v_dim
    batch = cu_k.shape[0] - 1
    at, scale, n_pages = _pages(d, pages, kv_scale)
    width = _columns(table, "table")
    _check(_lib.coli_mla_expand(
        ctypes.byref(d), batch, n, at, scale, n_pages, _arg(table, torch.int32, (batch, width), "table"),
        width, _arg(cu_k, torch.int32, (batch + 1,), "cu_k"), _arg(w, dt, (d.n_heads, wide, d.rank), "w"),
        _arg(kv, dt, (n, d.n_heads, wide), "kv"), _arg(k_pe, dt, (n, COLI_MLA_ROPE), "k_pe"), *_ws(ws),
        _stream(stream, kv)), "coli_mla_expand")


def coli_mla_prefill(dims, q, k_nope, k_pe, v, cu_q, cu_k, max_q, causal, out, lse, ws, stream=None):
    """q, k_nope and v are views with strides of their own (k_nope and v as coli_mla_expand leaves them: kv[..., :nope]
    and kv[..., nope:]).  lse may be None."""
    rc = _bind.prefill(_at(dims), q, k_nope, k_pe, v, cu_q, cu_k, max_q, causal, out, lse, ws, _handle(stream))
    if rc != 1:
        return _check(rc, "coli_mla_prefill")
    d, dt, n, m = dims, _OF[dims.dtype], q.shape[0], k_nope.shape[0]
    batch = cu_q.shape[0] - 1
    _check(_lib.coli_mla_prefill(
        ctypes.byref(d), batch, n, m, *_strided(q, dt, (n, d.n_heads, d.nope + COLI_MLA_ROPE), "q"),
        *_strided(k_nope, dt, (m, d.n_heads, d.nope), "k_nope"), _arg(k_pe, dt, (m, COLI_MLA_ROPE), "k_pe"),
        *_strided(v, dt, (m, d.n_heads, d.v_dim), "v"), _arg(cu_q, torch.int32, (batch + 1,), "cu_q"),
        _arg(cu_k, torch.int32, (batch + 1,), "cu_k"), max_q, int(bool(causal)),
        _arg(out, dt, (n, d.n_heads, d.v_dim), "out"),
        None if lse is None else _arg(lse, torch.float32, (n, d.n_heads), "lse"), *_ws(ws),
        _stream(stream, q)), "coli_mla_prefill")
