"""Quantisation of more tokens than one launch's grid holds: the last ones are done too."""
import pytest
import torch

from tests.gpu_util import q, say

pytestmark = pytest.mark.gpu


def test_quantize_more_tokens_than_a_grid():
    """2^22 + 3 tokens of 1024 threads each are more than 2^32 threads.  One row stands for all of them (stride 0)."""
    say("quantize, many tokens")
    assert torch.cuda.is_available(), "no GPU visible"
    n, k = (1 << 22) + 3, 16384
    if torch.cuda.mem_get_info()[0] < n * k + (8 << 30):
        pytest.skip("not enough free memory")
    x = torch.randn(1, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    codes, scale = torch.empty(n, k, dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda")
    one, s = torch.empty(1, k, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    q().coli_w8_quantize(x, one, s)
    q().coli_w8_quantize(x.expand(n, k), codes, scale)
    assert (scale == s).all()
    for at in (0, (1 << 21) - 1, 1 << 21, 1 << 22, n - 1):
        assert torch.equal(codes[at], one[0]), at
