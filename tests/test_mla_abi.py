"""Latent attention: the library exports what include/coli_mla.h declares, and refuses bad arguments on the host,
before it looks for a device."""
import ctypes
import os
import re

import pytest
import torch

import quantized_expert_ffn_amd as q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20   # an address that is never followed: every call here is refused first


def test_names_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "coli_mla.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(coli_mla_\w+)\s*\(", text)))
    assert sorted(q.MLA_EXPORTS) == declared
    lib = ctypes.CDLL(q.LIB_PATH)
    for n in declared:
        assert hasattr(lib, n) and callable(getattr(q, n))


def _dims(**kw):
    base = dict(n_heads=5, rank=512, nope=128, v_dim=128, page_size=48)
    base.update(kw)
    return q.make_mla_dims(**base)


@pytest.mark.parametrize("field,value", [
    ("n_heads", 0), ("n_heads", 257), ("rank", 0), ("rank", 384), ("nope", 192), ("v_dim", 64), ("page_size", 0),
    ("page_size", 65537), ("dtype", 2), ("kv_format", 2), ("kv_format", -1), ("rope_style", 2), ("norm_eps", -1.0),
    ("norm_eps", float("nan")), ("softmax_scale", 0.0), ("softmax_scale", float("inf"))])
def test_dims_are_checked(field, value):
    d = _dims()
    setattr(d, field, value)
    assert q.coli_mla_row_bytes(d) == 0
    assert field.split("_")[0] in q.coli_moe_last_error()
    with pytest.raises(q.ColiError) as e:
        q.coli_mla_workspace_bytes(d, 0)
    assert e.value.code == q.COLI_EINVAL


def test_sizes():
    assert q.coli_mla_row_bytes(_dims()) == 1152
    assert q.coli_mla_row_bytes(_dims(rank=256, kv_format=q.COLI_KV_E4M3)) == 384
    assert q.coli_mla_workspace_bytes(_dims()) >= 256
    for bad in ((-1, 1, 0), (4097, 1, 0), (1, 0, 0), (1, 4000, 5), (1, 1, -1), (4000, 1, 1 << 30)):
        with pytest.raises(q.ColiError):
            q.coli_mla_workspace_bytes(_dims(), *bad)
    assert q.make_mla_dims(1, 512, 192, 256, 64).softmax_scale == pytest.approx(1 / 16)
    with pytest.raises(TypeError):
        q.make_mla_dims(1, 512, 192, 256, 64, dtype=torch.float32)


def _ref(d):
    return ctypes.byref(d)


CALLS = {
    "append": (lambda d, n=3, kv_a=P, g=P, pos=P, slots=P, freq=P, qp=P, qts=320, qhs=64, qo=P, ots=320, ohs=64, pages=P,
               scale=None, n_pages=4, ws=P, wsb=256:
               q._lib.coli_mla_append(_ref(d), n, kv_a, g, pos, slots, freq, qp, qts, qhs, qo, ots, ohs, pages, scale,
                                      n_pages, ws, wsb, None),
               [dict(n=-1), dict(kv_a=None), dict(pos=None), dict(slots=None), dict(freq=None), dict(qp=None),
                dict(qo=None), dict(kv_a=P + 8), dict(g=P + 2), dict(qp=P + 4), dict(qo=P + 4), dict(qts=-8),
                dict(qhs=63), dict(ots=4), dict(ohs=1), dict(pages=None), dict(pages=P + 8), dict(scale=P),
                dict(n_pages=0), dict(ws=None), dict(ws=P + 4)]),
    "decode": (lambda d, batch=2, n_q=1, ql=P, qp=P, pages=P, scale=None, n_pages=4, table=P, width=2, lens=P, max_kv=90,
               out=P, lse=P, ws=P, wsb=1 << 40:
               q._lib.coli_mla_decode(_ref(d), batch, n_q, ql, qp, pages, scale, n_pages, table, width, lens, max_kv,
                                      out, lse, ws, wsb, None),
               [dict(batch=-1), dict(batch=4097), dict(n_q=0), dict(n_q=4000), dict(max_kv=-1),
                dict(batch=4000, max_kv=1 << 30), dict(ql=None),
                dict(qp=None), dict(table=None), dict(lens=None), dict(out=None), dict(ql=P + 2), dict(qp=P + 2),
                dict(out=P + 2), dict(width=0), dict(width=1), dict(max_kv=97), dict(pages=None), dict(scale=P),
                dict(n_pages=-1), dict(ws=None)]),
    "expand": (lambda d, batch=2, rows=7, pages=P, scale=None, n_pages=4, table=P, width=2, cu=P, w=P, kv=P, kp=P, ws=P,
               wsb=256:
               q._lib.coli_mla_expand(_ref(d), batch, rows, pages, scale, n_pages, table, width, cu, w, kv, kp, ws, wsb,
                                      None),
               [dict(batch=-1), dict(rows=-1), dict(table=None), dict(cu=None), dict(w=None), dict(kv=None),
                dict(kp=None), dict(w=P + 2), dict(kv=P + 2), dict(kp=P + 2), dict(width=0), dict(pages=None),
                dict(scale=P), dict(n_pages=0), dict(ws=None)]),
    "prefill": (lambda d, batch=2, nq=7, nk=9, qq=P, qts=960, qhs=192, kn=P, kts=1280, khs=256, kp=P, v=P, vts=1280,
                vhs=256, cq=P, ck=P, max_q=5, causal=1, out=P, lse=P, ws=P, wsb=256:
                q._lib.coli_mla_prefill(_ref(d), batch, nq, nk, qq, qts, qhs, kn, kts, khs, kp, v, vts, vhs, cq, ck,
                                        max_q, causal, out, lse, ws, wsb, None),
                [dict(batch=-1), dict(nq=-1), dict(nk=-1), dict(max_q=-1), dict(causal=2), dict(qq=None), dict(kn=None),
                 dict(kp=None), dict(v=None), dict(cq=None), dict(ck=None), dict(out=None), dict(qq=P + 2),
                 dict(kn=P + 2), dict(kp=P + 2), dict(v=P + 2), dict(out=P + 2), dict(qts=4), dict(qhs=-8),
                 dict(kts=1), dict(khs=4), dict(vts=-8), dict(vhs=12), dict(ws=None), dict(kts=(1 << 23) + 8),
                 dict(vts=1 << 40), dict(batch=4096, max_q=1 << 30)]),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_bad_arguments_are_refused(name):
    call, bads = CALLS[name]
    for bad in bads:
        assert call(_dims(), **bad) == q.COLI_EINVAL, bad
    assert call(_dims(), wsb=0) == q.COLI_EWORKSPACE
    d = _dims()
    d.rank = 100
    assert call(d) == q.COLI_EINVAL
    e4m3 = _dims(kv_format=q.COLI_KV_E4M3)
    if name != "prefill":
        assert call(e4m3) == q.COLI_EINVAL   # no kv_scale


@pytest.mark.parametrize("name,empty", [("append", dict(n=0)), ("decode", dict(batch=0)), ("expand", dict(rows=0)),
                                        ("expand", dict(batch=0)), ("prefill", dict(nq=0)), ("prefill", dict(max_q=0)),
                                        ("prefill", dict(batch=0))])
def test_empty_calls_are_no_ops(name, empty):
    assert CALLS[name][0](_dims(), **empty) == q.COLI_OK


def test_lengths_end_before_32_bits_do():
    """Tiles are counted in 32 bits, from a length rounded up."""
    top = q.COLI_MLA_MAX_LENGTH
    assert top == 2 ** 31 - 256
    d = _dims(page_size=65536)
    assert q.coli_mla_workspace_bytes(d, 1, 1, top) >= q.coli_mla_workspace_bytes(d, 1, 1, 1 << 20)
    for n in (top + 1, 2 ** 31 - 1):
        with pytest.raises(q.ColiError) as e:
            q.coli_mla_workspace_bytes(d, 1, 1, n)
        assert e.value.code == q.COLI_EINVAL
        assert CALLS["decode"][0](d, batch=1, max_kv=n, width=32768) == q.COLI_EINVAL
        assert CALLS["expand"][0](d, rows=n) == q.COLI_EINVAL
        assert CALLS["prefill"][0](d, nq=n) == q.COLI_EINVAL
        assert CALLS["prefill"][0](d, nk=n) == q.COLI_EINVAL
    assert CALLS["prefill"][0](_dims(n_heads=16), batch=1, max_q=2 ** 31 - 1) == q.COLI_EINVAL   # 2^28 blocks


def test_project_arguments():
    def call(dt=0, n=3, h=5, a=128, b=512, x=P, ts=640, hs=128, w=P, out=P):
        return q._lib.coli_mla_project(dt, n, h, a, b, x, ts, hs, w, out, None)
    for bad in (dict(dt=2), dict(n=-1), dict(n=1 << 30), dict(h=0), dict(h=257), dict(a=96), dict(a=0), dict(a=1088), dict(b=32),
                dict(b=4160), dict(x=None), dict(w=None), dict(out=None), dict(x=P + 2), dict(w=P + 2),
                dict(out=P + 2), dict(ts=-8), dict(hs=4)):
        assert call(**bad) == q.COLI_EINVAL, bad
    assert call(n=0) == q.COLI_OK


def test_binding_refuses_what_does_not_fit():
    """Types, shapes and devices, on CPU tensors: nothing gets as far as the library."""
    d = _dims()
    bf = torch.bfloat16
    kv_a, ws = torch.zeros(3, 576, dtype=bf), torch.zeros(256, dtype=torch.uint8)
    pages = torch.zeros(4, 48, 576, dtype=bf)
    with pytest.raises(ValueError, match="device"):
        q.coli_mla_append(d, kv_a, None, None, None, None, None, None, pages, None, ws)
    with pytest.raises(TypeError, match="pages: dtype"):
        q.coli_mla_append(d, kv_a, None, None, None, None, None, None, pages.half(), None, ws)
    with pytest.raises(ValueError, match="pages: shape"):
        q.coli_mla_append(d, kv_a, None, None, None, None, None, None, pages[:, :, :512], None, ws)
    with pytest.raises(TypeError, match="x: dtype"):
        q.coli_mla_project(torch.zeros(1, 1, 64), torch.zeros(1, 64, 64), torch.zeros(1, 1, 64))
    with pytest.raises(ValueError, match="rows for"):
        q.coli_mla_decode(d, torch.zeros(3, 5, 512, dtype=bf), None, pages, None, None, torch.zeros(2, dtype=torch.int32),
                          5, None, None, ws)
    with pytest.raises(ValueError, match="overlap"):
        q.mla._distinct(torch.zeros(64, dtype=bf).expand(2, 5, 64), (0, 0), "o")
    q.mla._distinct(torch.zeros(2, 5, 64), (320, 64), "o")
    q.mla._distinct(torch.zeros(2, 5, 192)[..., 128:], (960, 192), "o")
    q.mla._distinct(torch.zeros(5, 2, 64).transpose(0, 1), (64, 128), "o")


class _On(torch.Tensor):
    """A CPU tensor that says it is on a device."""
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", getattr(self, "index", 0))


def _on(index, *shape, dtype=torch.bfloat16):
    t = torch.zeros(shape, dtype=dtype).as_subclass(_On)
    t.index = index
    return t


def _device_calls(d, index):
    """Arguments that fit, by entry point; `index` says the device of the tensor of that name, 0 for the others."""
    i32, f32 = torch.int32, torch.float32

    def t(name, *shape, dtype=torch.bfloat16):
        return _on(index.get(name, 0), *shape, dtype=dtype)
    pages, ws = t("pages", 4, 48, 576), t("ws", 1 << 20, dtype=torch.uint8)
    return {
        "append": (q.coli_mla_append, dict(
            dims=d, kv_a=t("kv_a", 3, 576), norm_w=t("norm_w", 512), positions=t("positions", 3, dtype=i32),
            slots=t("slots", 3, dtype=torch.int64), inv_freq=t("inv_freq", 32, dtype=torch.float64), q_pe=t("q_pe", 3, 5, 64),
            q_pe_out=t("q_pe_out", 3, 5, 64), pages=pages, kv_scale=None, ws=ws)),
        "project": (q.coli_mla_project, dict(x=t("x", 3, 5, 128), w=t("w", 5, 512, 128), out=t("out", 3, 5, 512))),
        "decode": (q.coli_mla_decode, dict(
            dims=d, q_lat=t("q_lat", 2, 5, 512), q_pe=t("q_pe", 2, 5, 64), pages=pages, kv_scale=None,
            table=t("table", 2, 2, dtype=i32), kv_lens=t("kv_lens", 2, dtype=i32), max_kv=90, out=t("out", 2, 5, 512),
            lse=t("lse", 2, 5, dtype=f32), ws=ws)),
        "expand": (q.coli_mla_expand, dict(
            dims=d, pages=pages, kv_scale=None, table=t("table", 2, 2, dtype=i32), cu_k=t("cu_k", 3, dtype=i32),
            w=t("w", 5, 256, 512), kv=t("kv", 7, 5, 256), k_pe=t("k_pe", 7, 64), ws=ws)),
        "prefill": (q.coli_mla_prefill, dict(
            dims=d, q=t("q", 7, 5, 192), k_nope=t("k_nope", 9, 5, 128), k_pe=t("k_pe", 9, 64), v=t("v", 9, 5, 128),
            cu_q=t("cu_q", 3, dtype=i32), cu_k=t("cu_k", 3, dtype=i32), max_q=5, causal=True, out=t("out", 7, 5, 128),
            lse=t("lse", 7, 5, dtype=f32), ws=ws)),
    }


@pytest.mark.parametrize("name", sorted(CALLS) + ["project"])
def test_binding_refuses_tensors_of_two_devices(name, monkeypatch):
    """Whatever the quick way refuses is refused, and never launched from here."""
    launches = []
    for entry in q.MLA_EXPORTS:
        if entry not in ("coli_mla_row_bytes", "coli_mla_workspace_bytes"):
            monkeypatch.setattr(q._lib, entry, lambda *a, entry=entry: launches.append(entry) or 0)
    call, args = _device_calls(_dims(), {})[name]
    tensors = [k for k, v in args.items() if isinstance(v, torch.Tensor)]
    for odd in tensors:
        call, args = _device_calls(_dims(), {odd: 1})[name]
        with pytest.raises(ValueError, match="device cuda"):
            call(**args, stream=0)
    call, args = _device_calls(_dims(), {})[name]   # fits by what it says, though not for the quick way
    with pytest.raises(ValueError, match="refused"):
        call(**args, stream=0)
    assert not launches


def test_binding_refuses_numbers_past_32_bits():
    for name, what in (("decode", "max_kv"), ("prefill", "max_q")):
        call, args = _device_calls(_dims(), {})[name]
        args[what] = (1 << 32) + 5
        with pytest.raises(ValueError, match=what):
            call(**args, stream=0)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_binding_takes_its_own_dims_only(name):
    call, args = _device_calls(_dims(), {})[name]
    for other in (ctypes.c_int32(5), q.coli_moe_dims(), None, 7):
        with pytest.raises(TypeError, match="coli_mla_dims"):
            call(**{**args, "dims": other}, stream=0)


@pytest.mark.parametrize("name", sorted(CALLS) + ["project"])
def test_binding_refuses_streams_that_do_not_fit(name):
    """A handle is an address; a stream is the tensors' device's."""
    call, args = _device_calls(_dims(), {})[name]

    class Other:
        cuda_stream, device = 7, torch.device("cuda", 1)
    for bad, error in ((-5, ValueError), (1 << 70, ValueError), (Other(), ValueError), ("7", TypeError), (1.5, TypeError)):
        with pytest.raises(error, match="stream"):
            call(**args, stream=bad)


def test_the_package_stands_without_the_attention_module(tmp_path):
    """The MoE layer needs the library alone; attention says what is missing and how to build it, by a command that works
    where the package does not import."""
    import shutil
    import subprocess
    import sys
    pkg = os.path.join(ROOT, "quantized_expert_ffn_amd")
    copy = tmp_path / "quantized_expert_ffn_amd"
    shutil.copytree(pkg, copy, ignore=shutil.ignore_patterns("csrc", "__pycache__", "*.o", "_mla_bind.so"))
    code = ("import torch, quantized_expert_ffn_amd as q\n"
            "assert not q.coli_moe_last_error() and q.coli_mla_row_bytes(q.make_mla_dims(1, 512, 128, 128, 16)) == 1152\n"
            "try:\n    q.coli_mla_project(torch.zeros(1, 1, 64), torch.zeros(1, 64, 64), torch.zeros(1, 1, 64))\n"
            "except ImportError as e:\n    print(e)\n")
    run = lambda: subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    r = run()
    assert r.returncode == 0, r.stderr
    os.remove(copy / "_build" / "libcolimoe.so")
    gone = run()
    assert gone.returncode != 0
    for text in (r.stdout, gone.stderr):
        named = re.search(r"`python (\S+)`", text)
        assert named and os.path.samefile(os.path.join(ROOT, named.group(1)), os.path.join(pkg, "build.py")), text
