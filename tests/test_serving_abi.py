"""8-bit products, expert selection and shared decode: the library exports what its headers declare, and refuses bad
arguments on the host, before it looks for a device."""
import ctypes
import os
import re

import pytest
import torch

import quantized_expert_ffn_amd as q
from tests.test_mla_abi import _dims, _on

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20   # an address that is never followed: every call here is refused first


def test_names_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "coli_w8.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(coli_w8_\w+)\s*\(", text)))
    assert sorted(q.W8_EXPORTS) == declared
    lib = ctypes.CDLL(q.LIB_PATH)
    for n in declared:
        assert hasattr(lib, n) and callable(getattr(q, n))


def quantize(dt=0, n=3, k=64, x=P, ts=64, codes=P, scale=P):
    return q._lib.coli_w8_quantize(dt, n, k, x, ts, codes, scale, None)


def linear(dt=0, n=3, k=64, o=5, codes=P, cs=64, scale=P, w=P, ws=P, bias=None, out=P, os_=5):
    return q._lib.coli_w8_linear(dt, n, k, o, codes, cs, scale, w, ws, bias, out, os_, None)


@pytest.mark.parametrize("call,bads", [
    (quantize, [dict(dt=3), dict(dt=-1), dict(n=-1), dict(n=(1 << 24) + 1), dict(k=0), dict(k=8), dict(k=72), dict(k=65552),
                dict(x=None), dict(codes=None), dict(scale=None), dict(x=P + 8), dict(codes=P + 4), dict(scale=P + 2),
                dict(ts=-8), dict(ts=68), dict(dt=2, ts=66), dict(ts=(1 << 36) + 8)]),
    (linear, [dict(dt=3), dict(n=-1), dict(n=(1 << 24) + 1), dict(k=0), dict(k=24), dict(k=65552), dict(o=0),
              dict(o=(1 << 24) + 1, os_=1 << 30), dict(codes=None), dict(scale=None), dict(w=None), dict(ws=None), dict(out=None),
              dict(codes=P + 8), dict(w=P + 4), dict(scale=P + 2), dict(ws=P + 1), dict(bias=P + 2), dict(out=P + 1),
              dict(dt=2, out=P + 2), dict(cs=-16), dict(cs=40), dict(cs=(1 << 36) + 16), dict(os_=4), dict(os_=(1 << 36) + 1)])])
def test_w8_bad_arguments_are_refused(call, bads):
    for bad in bads:
        assert call(**bad) == q.COLI_EINVAL, bad
        assert q.coli_moe_last_error()
    assert call(n=0) == q.COLI_OK


def select(d, n=3, dt=2, logits=P, ts=16, bias=P, idx=P, w=P, ws=P, wsb=256):
    return q._lib.coli_moe_select(ctypes.byref(d) if d else None, n, dt, logits, ts, bias, idx, w, ws, wsb, None)


def test_select_bad_arguments_are_refused():
    d = q.make_select_dims(16, 4, 4, 2)
    for bad in (dict(n=-1), dict(n=65537), dict(dt=3), dict(logits=None), dict(idx=None), dict(w=None), dict(ws=None), dict(ts=-1),
                dict(ts=-16), dict(ts=(1 << 32) + 1), dict(logits=P + 2), dict(dt=0, logits=P + 1), dict(bias=P + 2), dict(idx=P + 2),
                dict(w=P + 1), dict(ws=P + 8)):
        assert select(d, **bad) == q.COLI_EINVAL, bad
    assert select(None) == q.COLI_EINVAL
    assert select(d, wsb=255) == q.COLI_EWORKSPACE
    assert select(d, n=0) == q.COLI_OK


@pytest.mark.parametrize("field,value", [
    ("n_experts", 0), ("n_experts", 1025), ("n_experts", 17), ("top_k", 0), ("top_k", 9), ("top_k", 33), ("n_group", 0), ("n_group", 3),
    ("n_group", 65), ("topk_group", 0), ("topk_group", 5), ("scoring", 2), ("scoring", -1), ("group_score", 2),
    ("norm_topk_prob", 2), ("routed_scaling_factor", float("nan")), ("routed_scaling_factor", float("inf"))])
def test_select_dims_are_checked(field, value):
    d = q.make_select_dims(16, 4, 4, 2)
    setattr(d, field, value)
    assert select(d) == q.COLI_EINVAL
    assert field.split("_")[0] in q.coli_moe_last_error() or field == "n_experts"


def shared(d, batch=2, n_q=1, ql=P, qp=P, pages=P, scale=None, n_pages=4, ptable=P, pwidth=2, plen=90, table=P, width=2, lens=P,
           max_kv=90, out=P, lse=P, ws=P, wsb=1 << 40):
    return q._lib.coli_mla_decode_shared(ctypes.byref(d), batch, n_q, ql, qp, pages, scale, n_pages, ptable, pwidth, plen, table,
                                         width, lens, max_kv, out, lse, ws, wsb, None)


def test_shared_bad_arguments_are_refused():
    for bad in (dict(batch=-1), dict(batch=4097), dict(n_q=0), dict(n_q=4000), dict(batch=4000, n_q=60), dict(max_kv=-1),
                dict(batch=4000, max_kv=1 << 30), dict(plen=-1), dict(plen=2 ** 31 - 255), dict(plen=97), dict(pwidth=0),
                dict(pwidth=1), dict(ptable=None), dict(ql=None), dict(qp=None), dict(table=None), dict(lens=None), dict(out=None),
                dict(ql=P + 2), dict(qp=P + 2), dict(out=P + 2), dict(width=0), dict(width=1), dict(max_kv=97), dict(pages=None),
                dict(pages=P + 8), dict(scale=P), dict(n_pages=0), dict(ws=None), dict(ws=P + 8)):
        assert shared(_dims(), **bad) == q.COLI_EINVAL, bad
    assert shared(_dims(), wsb=4096) == q.COLI_EWORKSPACE
    assert shared(_dims(), batch=0) == q.COLI_OK
    d = _dims()
    d.rank = 100
    assert shared(d) == q.COLI_EINVAL
    assert shared(_dims(kv_format=q.COLI_KV_E4M3)) == q.COLI_EINVAL   # no kv_scale


def test_shared_path_is_one_of_three():
    for path in (-1, 3):
        assert q._lib.coli_mla_debug_shared_path(path) == q.COLI_EINVAL
    assert q._lib.coli_mla_debug_shared_path(0) == q.COLI_OK


def test_shared_workspace_grows_with_each_size():
    """A workspace serves every smaller call."""
    for heads in (1, 5, 32, 64, 128):
        d = _dims(n_heads=heads)
        sizes = [(b, n, p, k) for b in (1, 3, 16, 64) for n in (1, 2, 9) for p in (0, 1, 33, 5000, 100000) for k in (0, 1, 200, 9000)]
        need = {s: q.coli_mla_shared_workspace_bytes(d, *s) for s in sizes}
        for s in sizes:
            for t in sizes:
                if all(a <= b for a, b in zip(s, t)):
                    assert need[s] <= need[t], (s, t)
    for bad in ((-1, 1, 5, 5), (1, 0, 5, 5), (4000, 60, 5, 5), (1, 1, -1, 5), (1, 1, 5, -1), (1, 1, 2 ** 31 - 1, 5)):
        with pytest.raises(q.ColiError):
            q.coli_mla_shared_workspace_bytes(_dims(), *bad)


# ---------------------------------------------------------------- the binding
def _calls(index):
    i32, f32, i8, bf = torch.int32, torch.float32, torch.int8, torch.bfloat16

    def t(name, *shape, dtype=bf):
        return _on(index.get(name, 0), *shape, dtype=dtype)
    return {
        "quantize": (q.coli_w8_quantize, dict(x=t("x", 3, 64), codes=t("codes", 3, 64, dtype=i8), scale=t("scale", 3, dtype=f32))),
        "linear": (q.coli_w8_linear, dict(
            codes=t("codes", 3, 64, dtype=i8), scale=t("scale", 3, dtype=f32), w=t("w", 5, 64, dtype=i8),
            w_scale=t("w_scale", 5, dtype=f32), bias=t("bias", 5, dtype=f32), out=t("out", 3, 5))),
        "select": (q.coli_moe_select, dict(
            dims=q.make_select_dims(16, 4, 4, 2), logits=t("logits", 3, 16), bias=t("bias", 16, dtype=f32),
            topk_idx=t("topk_idx", 3, 4, dtype=i32), topk_w=t("topk_w", 3, 4, dtype=f32), ws=t("ws", 256, dtype=torch.uint8))),
        "shared": (q.coli_mla_decode_shared, dict(
            dims=_dims(), q_lat=t("q_lat", 2, 5, 512), q_pe=t("q_pe", 2, 5, 64), pages=t("pages", 4, 48, 576), kv_scale=None,
            prefix_table=t("prefix_table", 2, dtype=i32), prefix_len=90, table=t("table", 2, 2, dtype=i32),
            kv_lens=t("kv_lens", 2, dtype=i32), max_kv=90, out=t("out", 2, 5, 512), lse=t("lse", 2, 5, dtype=f32),
            ws=t("ws", 1 << 20, dtype=torch.uint8))),
    }


NAMES = sorted(_calls({}))


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_tensors_of_two_devices(name, monkeypatch):
    launches = []
    for entry in ("coli_w8_quantize", "coli_w8_linear", "coli_moe_select", "coli_mla_decode_shared"):
        monkeypatch.setattr(q._lib, entry, lambda *a, entry=entry: launches.append(entry) or 0)
    call, args = _calls({})[name]
    for odd in [k for k, v in args.items() if isinstance(v, torch.Tensor)]:
        call, args = _calls({odd: 1})[name]
        with pytest.raises(ValueError, match="device cuda"):
            call(**args, stream=0)
    call, args = _calls({})[name]   # fits by what it says, though not for the quick way
    with pytest.raises(ValueError, match="refused"):
        call(**args, stream=0)
    assert not launches


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_types_and_shapes(name):
    """Each tensor in turn of another type, then with a row or value more."""
    call, args = _calls({})[name]
    for k, v in args.items():
        if isinstance(v, torch.Tensor):
            wrong = torch.zeros(v.shape, dtype=torch.float64)
            with pytest.raises(TypeError, match=k):
                call(**{**args, k: wrong}, stream=0)
            with pytest.raises(TypeError):
                call(**{**args, k: [1, 2]}, stream=0)
            if k not in ("ws", "prefix_table"):   # any length; too few are the library's to refuse
                longer = torch.zeros((*v.shape[:-1], v.shape[-1] + 1), dtype=v.dtype)
                with pytest.raises(ValueError):
                    call(**{**args, k: longer}, stream=0)


@pytest.mark.parametrize("name", NAMES)
def test_binding_refuses_streams_that_do_not_fit(name):
    call, args = _calls({})[name]

    class Other:
        cuda_stream, device = 7, torch.device("cuda", 1)
    for bad, error in ((-5, ValueError), (1 << 70, ValueError), (Other(), ValueError), ("7", TypeError)):
        with pytest.raises(error, match="stream"):
            call(**args, stream=bad)


def test_binding_takes_its_own_dims_only():
    for name, what in (("select", "coli_select_dims"), ("shared", "coli_mla_dims")):
        call, args = _calls({})[name]
        for other in (ctypes.c_int32(5), q.coli_moe_dims(), None, 7):
            with pytest.raises(TypeError, match=what):
                call(**{**args, "dims": other}, stream=0)


def test_binding_refuses_rows_that_overlap():
    out, x = _on(0, 64).as_strided((3, 5), (4, 1)), _on(0, 64, 3).t()
    out.index = x.index = 0
    _, args = _calls({})["linear"]
    with pytest.raises(ValueError, match="overlap"):
        q.coli_w8_linear(**{**args, "out": out}, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        q.coli_w8_quantize(x, args["codes"], args["scale"], stream=0)
