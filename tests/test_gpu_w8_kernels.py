"""8-bit products through every kernel that tokens and channels choose, in all three types: splits of one to three tiles of
channels by two to five of tokens, whose sums meet in LDS in batches of which the last is partly filled, and the three sizes
of tiles, with one and with several of them a workgroup."""
import pytest
import torch

from tests import mla_ref as ref
from tests.gpu_util import q, say
from tests.test_gpu_w8 import BF, F32, FP, TINY, U, exact_sums, gen, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


def tolerance(p, bias, dtype):
    """Binary32 results are formed in binary64, product by product and then the sum, on both sides: eight roundings of 2^-53
    in all, and half a step of binary32.  16-bit ones are formed in binary32: three roundings of the product, one of the sum
    (2^-24 each), then half a step of the output's type."""
    want = p if bias is None else p + bias.double()
    if dtype == F32:
        return want, 2.0 ** -24 * want.abs() + 2.0 ** -50 * (p.abs() + want.abs()) + 2.0 ** -149
    f32 = 3.01 * ref.U32 * p.abs() + 1.01 * ref.U32 * want.abs() + 4 * 2.0 ** -149
    return want, f32 + 1.01 * U[dtype] * want.abs() + TINY[dtype]


def check(n, k, n_out, dtype, with_bias, seed):
    g = gen(seed)
    codes, scale, w, w_scale = inputs(g, n, k, n_out, full=True)
    bias = torch.randn(n_out, generator=g, device="cuda") if with_bias else None
    out = torch.full((n + 1, n_out), 7.0, dtype=dtype, device="cuda")
    q().coli_w8_linear(codes, scale, w, w_scale, bias, out[:n])
    want, tol = tolerance(exact_sums(codes, w) * scale.double()[:, None] * w_scale.double(), bias, dtype)
    ref.close(out[:n], want, tol, "out")
    assert (out[n] == 7).all(), "written behind the last token"


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("n_out", [8192, 8193, 12289, 16384, 16385, 19393])
@pytest.mark.parametrize("n", [33, 40, 64, 65, 90, 96, 97, 120, 128, 129, 133, 160])
def test_linear_of_every_split(dtype, n_out, n):
    """One tile of 32 channels a workgroup up to 8192 of them, two up to 16384, three beyond, by two to five tiles of tokens:
    rings that go round and end inside a step."""
    say("linear, split", dtype, n, n_out)
    check(n, 1424, n_out, dtype, (n + n_out) % 2 == 0, n + n_out)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("k", [16, 144, 4096])
def test_linear_of_every_split_short_and_long(dtype, k):
    """Sums shorter than a step, of two steps, and of many."""
    for n, n_out in ((1, 2048), (32, 2049), (40, 8200), (64, 17000), (90, 16000), (133, 8193), (160, 16385)):
        say("linear, split", dtype, n, k, n_out)
        check(n, k, n_out, dtype, n % 2 == 1, n + k)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("n,n_out", [
    (161, 2000), (300, 6144), (500, 6143),             # 128 x 64: fewer than CUs, and more
    (700, 9000), (1001, 6143), (3190, 6130),           # 256 x 128, and several a workgroup
    (2050, 6100), (2048, 6144), (8192, 6143)])         # 256 x 256, and several a workgroup
@pytest.mark.parametrize("k", [16, 272, 1040])
def test_linear_of_every_tile(dtype, n, n_out, k):
    say("linear, tiles", dtype, n, k, n_out)
    check(n, k, n_out, dtype, (n + k // 16) % 2 == 0, n + k)


@pytest.mark.parametrize("n", [1, 40, 133, 300, 1024, 2048])
def test_linear_rounds_binary32_once(n):
    """A bias that takes away nearly all of the first token's product: what is left of it is 2^-24 of the product and less,
    which an intermediate result in binary32 would not hold."""
    say("linear, rounded once", n)
    k, n_out = 512, 6144
    codes, scale, w, w_scale = inputs(gen(n), n, k, n_out)
    p = exact_sums(codes, w) * scale.double()[:, None] * w_scale.double()
    bias = -p[0].float()
    out = torch.empty(n, n_out, device="cuda")
    q().coli_w8_linear(codes, scale, w, w_scale, bias, out)
    want, tol = tolerance(p, bias, F32)
    assert (want[0].abs() <= 2.0 ** -24 * p[0].abs()).all() and (want[0] != 0).any()
    ref.close(out, want, tol, "out")
