"""Binding of the 8-bit products (include/coli_w8.h), in the manner of mla.py: the checks and the call run in the CPython
module, and what does not fit there is named here."""
from __future__ import annotations

import ctypes

import torch

from . import _lib, mla
from .mla import _handle, _MISFIT, _Refused, _check

COLI_W8_MAX_K, COLI_W8_MAX_ROWS = 65536, 1 << 24

W8_EXPORTS = ("coli_w8_quantize", "coli_w8_linear")

_FLOATS = (torch.bfloat16, torch.float16, torch.float32)

_P, _I32, _I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
_sigs = {
    "coli_w8_quantize": [_I32, _I32, _I32, _P, _I64, _P, _P, _P],
    "coli_w8_linear": [_I32, _I32, _I32, _I32, _P, _I64, _P, _P, _P, _P, _P, _I64, _P],
}
for _name, _args in _sigs.items():
    _f = getattr(_lib, _name)
    _f.restype = ctypes.c_int
    _f.argtypes = _args


def coli_w8_quantize(x, codes, scale, stream=None):
    """x [tokens, k] of bfloat16, float16 or float32, rows at a stride of their own, as int8 codes [tokens, k] and float32
    scale [tokens]."""
    rc = mla._bind.quantize(x, codes, scale, _handle(stream, x))
    if rc == _MISFIT:
        no = _Refused("coli_w8_quantize")
        n, k = (no.size(x, 2, i, "x") for i in range(2))
        no.rows(x, _FLOATS, (n, k), "x")
        no.dense(codes, torch.int8, (n, k), "codes")
        no.dense(scale, torch.float32, (n,), "scale")
        no.end()
    _check(rc, "coli_w8_quantize")


def coli_w8_linear(codes, scale, w, w_scale, bias, out, stream=None):
    """out[t, o] = scale[t] w_scale[o] sum_k codes[t, k] w[o, k] (+ bias[o]): codes int8 [tokens, k] and out [tokens, n_out]
    of bfloat16, float16 or float32 at strides of their own, w int8 [n_out, k]; bias float32 [n_out] or None."""
    rc = mla._bind.linear(codes, scale, w, w_scale, bias, out, _handle(stream, codes))
    if rc == _MISFIT:
        no = _Refused("coli_w8_linear")
        n, k, n_out = *(no.size(codes, 2, i, "codes") for i in range(2)), no.size(w, 2, 0, "w")
        no.rows(codes, (torch.int8,), (n, k), "codes")
        no.dense(scale, torch.float32, (n,), "scale")
        no.dense(w, torch.int8, (n_out, k), "w")
        no.dense(w_scale, torch.float32, (n_out,), "w_scale")
        if bias is not None:
            no.dense(bias, torch.float32, (n_out,), "bias")
        no.rows(out, _FLOATS, (n, n_out), "out")
        if n > 1 and out.stride(0) < n_out:
            raise ValueError("out: rows overlap")
        no.end()
    _check(rc, "coli_w8_linear")
