"""What the kernels of the 8-bit products and the shared-prefix decode were compiled to: a property that their sources rely
on, read from the metadata of this build."""
import pytest

from tests.test_mla_kernels import kernels


@pytest.mark.parametrize("name,kernel,count", [("mla_shared.o", "k_mla_shared", 8), ("w8_linear.o", "k_w8_split", 14),
                                               ("w8_linear.o", "k_w8_tiles", 9)])
def test_dynamic_lds_begins_at_zero(name, kernel, count, tmp_path):
    """These kernels address LDS by byte offset from 0, so nothing may be placed before their dynamic allocation."""
    found = {k: v for k, v in kernels(name, tmp_path).items() if kernel in k and "_join" not in k}
    assert len(found) >= count, sorted(found)
    assert not {k: v for k, v in found.items() if v}
