"""Builds the HIP library quantized_expert_ffn_amd/_build/libcolimoe.so for gfx950,
and the CPython module _mla_bind.so beside it (host code that calls the library).

Floating-point flags are part of the layer's contract: no contraction of
a*b+c into fma unless written as fmaf, correctly rounded binary32 division,
denormals kept, and no packed-fp32 instructions.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libcolimoe.so")
BIND = os.path.join(OUT_DIR, "_mla_bind.so")
SOURCES = ["route.hip", "forward.hip", "down_rows.hip", "prefill.hip", "prefill_mx.hip", "layer.hip", "debug.hip",
           "api.hip", "mla_append.hip", "mla_gemm.hip", "mla_decode.hip", "mla_prefill.hip", "mla_api.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


# Per-source additions: the matrix-core kernels keep their products in
# ordinary VGPRs (the prefill's f32 epilogue reads every product once, the
# latent attention's softmax every score).
_VGPR_FORM = ["-mllvm", "-amdgpu-mfma-vgpr-form"]
EXTRA = {"prefill.hip": _VGPR_FORM, "mla_decode.hip": _VGPR_FORM, "mla_prefill.hip": _VGPR_FORM}


def _compile(src: str) -> str:
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *EXTRA.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    return obj


def _torch_paths():
    """Include folders of torch and of Python, and torch's library folder, without importing torch."""
    import importlib.util
    import sysconfig
    root = os.path.dirname(importlib.util.find_spec("torch").origin)
    inc = os.path.join(root, "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"]], os.path.join(root, "lib")


def _compile_bind() -> str:
    """The CPython module's object: host code only, with torch's headers."""
    obj = os.path.join(OUT_DIR, "mla_bind.o")
    incs, _ = _torch_paths()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           "-I", os.path.join(ROOT, "include"), *[a for i in incs for a in ("-isystem", i)], "-isystem", "/opt/rocm/include",
           "-c", os.path.join(CSRC, "mla_bind.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for mla_bind.cpp:\n%s\n%s" % (" ".join(cmd), r.stderr))
    return obj


def _link_bind(obj: str) -> None:
    _, lib = _torch_paths()
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = ["g++", "-shared", obj, "-o", tmp, LIB, "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, BIND)


def build(verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(_compile_bind)
        objs = list(ex.map(_compile, SOURCES))
        bind = bind.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-Wl,-soname,libcolimoe.so", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    _link_bind(bind)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
