"""What the latent-attention kernels were compiled to: properties that their sources rely on, read from the metadata and
the assembly text of this build."""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BUILT = os.path.join(ROOT, "quantized_expert_ffn_amd", "_build")
READELF = "/opt/rocm/llvm/bin/llvm-readelf"


def code_object(name, tmp_path):
    """The gfx950 code object inside a built host object."""
    fat = str(tmp_path / "fat")
    subprocess.run(["objcopy", "-O", "binary", "--only-section=.hip_fatbin", "--set-section-flags", ".hip_fatbin=alloc",
                    os.path.join(BUILT, name), fat], check=True)
    data = open(fat, "rb").read()
    magic = b"__CLANG_OFFLOAD_BUNDLE__"
    assert data.startswith(magic)
    n, at = struct.unpack_from("<Q", data, len(magic))[0], len(magic) + 8
    for _ in range(n):
        offset, size, length = struct.unpack_from("<QQQ", data, at)
        triple = data[at + 24:at + 24 + length].decode()
        at += 24 + length
        if triple.endswith("gfx950"):
            out = str(tmp_path / "code")
            open(out, "wb").write(data[offset:offset + size])
            return out
    raise AssertionError(f"{name}: no gfx950 code")


def kernels(name, tmp_path):
    """Fixed LDS bytes of each kernel of an object."""
    notes = subprocess.run([READELF, "--notes", code_object(name, tmp_path)], check=True, capture_output=True, text=True).stdout
    found = {}
    for entry in re.split(r"\n\s*- \.a", notes)[1:]:   # entries begin with .agpr_count or .args
        size, kernel = re.search(r"\.group_segment_fixed_size:\s*(\d+)", entry), re.search(r"\.symbol:\s*'?(\S+?)\.kd", entry)
        if size and kernel:
            found[kernel.group(1)] = int(size.group(1))
    return found


@pytest.mark.parametrize("name,count", [("mla_prefill.o", 8), ("mla_decode.o", 16), ("mla_gemm.o", 18)])
def test_dynamic_lds_begins_at_zero(name, count, tmp_path):
    """These kernels address LDS by byte offset from 0, so nothing may be placed before their dynamic allocation: a
    barrier that carries a value, for one, takes a word of the device library's."""
    found = {k: v for k, v in kernels(name, tmp_path).items() if "k_mla_join" not in k}
    assert len(found) >= count and all("k_mla_" in k for k in found), sorted(found)
    assert not {k: v for k, v in found.items() if v}


def test_assembly_names_what_it_writes():
    """Every assembly text that writes m0 or the condition code says so to the compiler."""
    csrc = os.path.join(ROOT, "quantized_expert_ffn_amd", "csrc")
    seen = 0
    for name in sorted(os.listdir(csrc)):
        for text in re.findall(r"\basm\s+volatile\s*\((.*?)\);", open(os.path.join(csrc, name)).read(), re.S):
            if re.search(r"\bs_\w+\s+m0\b", text):
                seen += 1
                clobbers = text.rsplit(":", 1)[1]
                assert '"m0"' in clobbers and '"memory"' in clobbers, (name, text)
                assert "s_add" not in text or '"scc"' in clobbers, (name, text)
    assert seen
