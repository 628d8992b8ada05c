"""Binding of the latent-attention entry points (include/coli_mla.h).

Argument marshalling only: each function has the name of the C entry point
it calls, takes sizes and strides from the tensors, checks that they fit each
other, and raises ColiError on a non-zero return.  coli_moe_status() reads
the workspace's device status.

The checks and the call itself run in a CPython module (csrc/mla_bind.cpp),
since most of these kernels take less time than the same checks here; what
does not fit there comes back here, where the checks say what it is.  The
module makes the tensors' device current for the call.
"""
from __future__ import annotations

import ctypes
import importlib.util
import operator
import os

import torch

from . import _lib, LIB_PATH, ColiError

COLI_BF16, COLI_FP16, COLI_F32 = 0, 1, 2
COLI_KV_PLAIN, COLI_KV_E4M3 = 0, 1
COLI_ROPE_PAIRS, COLI_ROPE_HALVES = 0, 1
COLI_MLA_ROPE = 64
COLI_MLA_MAX_ROWS, COLI_MLA_MAX_BATCH, COLI_MLA_MAX_LENGTH = 16384, 4096, 2 ** 31 - 256
COLI_MLA_MAX_SHARED_ROWS = 1 << 20

MLA_EXPORTS = ("coli_mla_row_bytes", "coli_mla_workspace_bytes", "coli_mla_append", "coli_mla_project",
               "coli_mla_decode", "coli_mla_expand", "coli_mla_prefill", "coli_mla_shared_workspace_bytes",
               "coli_mla_decode_shared", "coli_mla_debug_shared_path")

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
    "coli_mla_shared_workspace_bytes": (_SZ, [_D, _I32, _I32, _I32, _I32]),
    "coli_mla_decode_shared": (ctypes.c_int, [_D, _I32, _I32, _P, _P, _P, _P, _I32, _P, _I32, _I32, _P, _I32, _P, _I32, _P,
                                              _P, _P, _SZ, _P]),
    "coli_mla_debug_shared_path": (ctypes.c_int, [_I32]),
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


class _Refused:
    """The arguments of a call that the module below refused, one after the other: raises at the first that does not fit.
    Nothing is launched from here."""

    def __init__(self, where):
        self.where, self.device = where, None

    def tensor(self, t, dtype, shape, what):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: expected a torch tensor")
        if t.dtype != dtype:
            raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        if not t.is_cuda:
            raise ValueError(f"{what}: must be a device tensor")
        if self.device is None:
            self.device = t.device
        if t.device != self.device:
            raise ValueError(f"{what}: on device {t.device}, expected device {self.device} as the others")

    def dense(self, t, dtype, shape, what):
        self.tensor(t, dtype, shape, what)
        if not t.is_contiguous():
            raise ValueError(f"{what}: must be contiguous")

    def view(self, t, dtype, shape, what):
        """[tokens, heads, width] with strides of its own, the last dimension dense."""
        self.tensor(t, dtype, shape, what)
        if t.stride(2) != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")

    def pages(self, d, pages, kv_scale):
        if d.kv_format == COLI_KV_E4M3:
            dtype, row = torch.uint8, d.rank + 2 * COLI_MLA_ROPE
        else:
            dtype, row = _OF[d.dtype], d.rank + COLI_MLA_ROPE
        n = self.size(pages, 3, 0, "pages")
        self.dense(pages, dtype, (n, d.page_size, row), "pages")
        if kv_scale is not None:
            self.dense(kv_scale, torch.float32, (n * d.page_size,), "kv_scale")

    def rows(self, t, dtypes, shape, what):
        """[rows, width] with a stride of its own, the last dimension dense, of one of some types."""
        self.size(t, 2, 0, what)
        if t.dtype not in dtypes:
            raise TypeError(f"{what}: dtype {t.dtype}, expected one of {', '.join(str(d) for d in dtypes)}")
        self.tensor(t, t.dtype, shape, what)
        if t.shape[1] > 1 and t.stride(1) != 1:
            raise ValueError(f"{what}: the last dimension must be contiguous")

    def workspace(self, ws):
        self.dense(ws, torch.uint8, (self.size(ws, 1, 0, "ws"),), "ws")

    @staticmethod
    def size(t, dims, dim, what):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: expected a torch tensor")
        if t.dim() != dims:
            raise ValueError(f"{what}: {t.dim()} dimensions, expected {dims}")
        return t.shape[dim]

    @staticmethod
    def number(n, what):
        if not -2 ** 31 <= operator.index(n) < 2 ** 31:
            raise ValueError(f"{what}: {n} does not fit 32 bits")

    def end(self):
        raise ValueError(f"{self.where}: arguments refused")


def _distinct(t, strides, what):
    """An output's elements must not share an address."""
    n, h, width = t.shape
    ts, hs = strides
    if n and h and not ((h == 1 or hs >= width) and (n == 1 or ts >= (h - 1) * hs + width)
                        or (n == 1 or ts >= width) and (h == 1 or hs >= (n - 1) * ts + width)):
        raise ValueError(f"{what}: strides overlap")


class _Bind:
    """csrc/mla_bind.cpp's module, loaded by its first call: it is built against torch's headers, and the rest of the
    package does without it."""

    def __getattr__(self, name):
        global _bind
        path = os.path.join(os.path.dirname(LIB_PATH), "_mla_bind.so")
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with `python quantized_expert_ffn_amd/build.py` "
                              "(or __graft_entry__.build())")
        spec = importlib.util.spec_from_file_location("_mla_bind", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        _bind = mod
        return getattr(mod, name)


_bind = _Bind()


def _at(dims):
    if not isinstance(dims, coli_mla_dims):
        raise TypeError(f"dims: {type(dims).__name__}, expected coli_mla_dims")
    return ctypes.addressof(dims)



_MISFIT = 1   # the module's answer to arguments that do not fit


def _handle(stream, t):
    """A stream of t's device, or its raw handle, as a handle; None: the device's current one."""
    if stream is None:
        return None
    if not isinstance(stream, int):
        if not hasattr(stream, "cuda_stream"):
            raise TypeError(f"stream: {type(stream).__name__}, expected a torch stream or a handle")
        if isinstance(t, torch.Tensor) and stream.device != t.device:
            raise ValueError(f"stream: of device {stream.device}, the tensors' is {t.device}")
        return stream.cuda_stream
    if not 0 <= stream < 2 ** 64:
        raise ValueError(f"stream: {stream} is no handle")
    return stream


def _sequences(no, cu, what):
    n = no.size(cu, 1, 0, what)
    if n < 1:
        raise ValueError(f"{what}: needs an offset more than sequences")
    return n - 1


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
    rc = _bind.append(_at(dims), kv_a, norm_w, positions, slots, inv_freq, q_pe, q_pe_out, pages, kv_scale, ws, _handle(stream, kv_a))
    if rc == _MISFIT:
        no, d, dt = _Refused("coli_mla_append"), dims, _OF[dims.dtype]
        n = no.size(kv_a, 2, 0, "kv_a")
        no.pages(d, pages, kv_scale)
        no.dense(kv_a, dt, (n, d.rank + COLI_MLA_ROPE), "kv_a")
        if norm_w is not None:
            no.dense(norm_w, dt, (d.rank,), "norm_w")
        no.dense(positions, torch.int32, (n,), "positions")
        no.dense(slots, torch.int64, (n,), "slots")
        no.dense(inv_freq, torch.float64, (COLI_MLA_ROPE // 2,), "inv_freq")
        if q_pe is not None:
            no.view(q_pe, dt, (n, d.n_heads, COLI_MLA_ROPE), "q_pe")
        if q_pe_out is not None:
            no.view(q_pe_out, dt, (n, d.n_heads, COLI_MLA_ROPE), "q_pe_out")
            _distinct(q_pe_out, q_pe_out.stride()[:2], "q_pe_out")
        no.workspace(ws)
        no.end()
    _check(rc, "coli_mla_append")


def coli_mla_project(x, w, out, stream=None):
    """out[t, h] = w[h] x[t, h]: x [n, heads, n_in] (a view with strides of its own), w [heads, n_out, n_in], out
    [n, heads, n_out]."""
    rc = _bind.project(x, w, out, _handle(stream, x))
    if rc == _MISFIT:
        no = _Refused("coli_mla_project")
        n, heads, n_in, n_out = *(no.size(x, 3, i, "x") for i in range(3)), no.size(w, 3, 1, "w")
        if x.dtype not in _OF.values():
            raise TypeError(f"x: dtype {x.dtype}, expected torch.bfloat16 or torch.float16")
        no.view(x, x.dtype, (n, heads, n_in), "x")
        no.dense(w, x.dtype, (heads, n_out, n_in), "w")
        no.dense(out, x.dtype, (n, heads, n_out), "out")
        no.end()
    _check(rc, "coli_mla_project")


def coli_mla_decode(dims, q_lat, q_pe, pages, kv_scale, table, kv_lens, max_kv, out, lse, ws, stream=None):
    """q_lat [batch * n_q, n_heads, rank]; the batch is kv_lens'.  lse may be None."""
    rc = _bind.decode(_at(dims), q_lat, q_pe, pages, kv_scale, table, kv_lens, max_kv, out, lse, ws, _handle(stream, q_lat))
    if rc == _MISFIT:
        no, d, dt = _Refused("coli_mla_decode"), dims, _OF[dims.dtype]
        batch, rows = no.size(kv_lens, 1, 0, "kv_lens"), no.size(q_lat, 3, 0, "q_lat")
        if batch and (rows % batch or not rows):
            raise ValueError(f"q_lat: {rows} rows for {batch} sequences")
        no.pages(d, pages, kv_scale)
        no.dense(q_lat, dt, (rows, d.n_heads, d.rank), "q_lat")
        no.dense(q_pe, dt, (rows, d.n_heads, COLI_MLA_ROPE), "q_pe")
        no.dense(table, torch.int32, (batch, no.size(table, 2, 1, "table")), "table")
        no.dense(kv_lens, torch.int32, (batch,), "kv_lens")
        no.number(max_kv, "max_kv")
        no.dense(out, dt, (rows, d.n_heads, d.rank), "out")
        if lse is not None:
            no.dense(lse, torch.float32, (rows, d.n_heads), "lse")
        no.workspace(ws)
        no.end()
    _check(rc, "coli_mla_decode")


def coli_mla_shared_workspace_bytes(dims, batch: int, n_q: int, prefix_len: int, max_kv: int) -> int:
    """Raises ColiError(COLI_EINVAL) for sizes that no call takes."""
    n = int(_lib.coli_mla_shared_workspace_bytes(ctypes.byref(dims), batch, n_q, prefix_len, max_kv))
    if n == 0:
        raise ColiError(-1, "coli_mla_shared_workspace_bytes")
    return n


def coli_mla_decode_shared(dims, q_lat, q_pe, pages, kv_scale, prefix_table, prefix_len, table, kv_lens, max_kv, out, lse,
                           ws, stream=None):
    """coli_mla_decode for sequences that begin with the prefix_len tokens of prefix_table [pages]; table and kv_lens are of
    their own tokens.  lse may be None."""
    rc = _bind.decode_shared(_at(dims), q_lat, q_pe, pages, kv_scale, prefix_table, prefix_len, table, kv_lens, max_kv, out,
                             lse, ws, _handle(stream, q_lat))
    if rc == _MISFIT:
        no, d, dt = _Refused("coli_mla_decode_shared"), dims, _OF[dims.dtype]
        batch, rows = no.size(kv_lens, 1, 0, "kv_lens"), no.size(q_lat, 3, 0, "q_lat")
        if batch and (rows % batch or not rows):
            raise ValueError(f"q_lat: {rows} rows for {batch} sequences")
        no.pages(d, pages, kv_scale)
        no.dense(q_lat, dt, (rows, d.n_heads, d.rank), "q_lat")
        no.dense(q_pe, dt, (rows, d.n_heads, COLI_MLA_ROPE), "q_pe")
        no.dense(prefix_table, torch.int32, (no.size(prefix_table, 1, 0, "prefix_table"),), "prefix_table")
        no.number(prefix_len, "prefix_len")
        no.dense(table, torch.int32, (batch, no.size(table, 2, 1, "table")), "table")
        no.dense(kv_lens, torch.int32, (batch,), "kv_lens")
        no.number(max_kv, "max_kv")
        no.dense(out, dt, (rows, d.n_heads, d.rank), "out")
        if lse is not None:
            no.dense(lse, torch.float32, (rows, d.n_heads), "lse")
        no.workspace(ws)
        no.end()
    _check(rc, "coli_mla_decode_shared")


def coli_mla_debug_shared_path(path: int) -> None:
    _check(_lib.coli_mla_debug_shared_path(int(path)), "coli_mla_debug_shared_path")


def coli_mla_expand(dims, pages, kv_scale, table, cu_k, w, kv, k_pe, ws, stream=None):
    rc = _bind.expand(_at(dims), pages, kv_scale, table, cu_k, w, kv, k_pe, ws, _handle(stream, kv))
    if rc == _MISFIT:
        no, d, dt, wide = _Refused("coli_mla_expand"), dims, _OF[dims.dtype], dims.nope + dims.v_dim
        n, batch = no.size(kv, 3, 0, "kv"), _sequences(no, cu_k, "cu_k")
        no.pages(d, pages, kv_scale)
        no.dense(table, torch.int32, (batch, no.size(table, 2, 1, "table")), "table")
        no.dense(cu_k, torch.int32, (batch + 1,), "cu_k")
        no.dense(w, dt, (d.n_heads, wide, d.rank), "w")
        no.dense(kv, dt, (n, d.n_heads, wide), "kv")
        no.dense(k_pe, dt, (n, COLI_MLA_ROPE), "k_pe")
        no.workspace(ws)
        no.end()
    _check(rc, "coli_mla_expand")


def coli_mla_prefill(dims, q, k_nope, k_pe, v, cu_q, cu_k, max_q, causal, out, lse, ws, stream=None):
    """q, k_nope and v are views with strides of their own (k_nope and v as coli_mla_expand leaves them: kv[..., :nope]
    and kv[..., nope:]).  lse may be None."""
    rc = _bind.prefill(_at(dims), q, k_nope, k_pe, v, cu_q, cu_k, max_q, causal, out, lse, ws, _handle(stream, q))
    if rc == _MISFIT:
        no, d, dt = _Refused("coli_mla_prefill"), dims, _OF[dims.dtype]
        n, m, batch = no.size(q, 3, 0, "q"), no.size(k_nope, 3, 0, "k_nope"), _sequences(no, cu_q, "cu_q")
        no.view(q, dt, (n, d.n_heads, d.nope + COLI_MLA_ROPE), "q")
        no.view(k_nope, dt, (m, d.n_heads, d.nope), "k_nope")
        no.dense(k_pe, dt, (m, COLI_MLA_ROPE), "k_pe")
        no.view(v, dt, (m, d.n_heads, d.v_dim), "v")
        no.dense(cu_q, torch.int32, (batch + 1,), "cu_q")
        no.dense(cu_k, torch.int32, (batch + 1,), "cu_k")
        no.number(max_q, "max_q")
        bool(causal)
        no.dense(out, dt, (n, d.n_heads, d.v_dim), "out")
        if lse is not None:
            no.dense(lse, torch.float32, (n, d.n_heads), "lse")
        no.workspace(ws)
        no.end()
    _check(rc, "coli_mla_prefill")
