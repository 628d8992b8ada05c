"""8-bit products on the GPU against their formulas: codes against exact quotients, products against exact sums."""
import math

import pytest
import torch

from tests import mla_ref as ref
from tests.gpu_util import q, say

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
NAN, INF = float("nan"), float("inf")
U = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -133, FP: 2.0 ** -24, F32: 2.0 ** -149}


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes_of(x, scale):
    """Codes by the scale as it is held, in 64 bits: torch.round takes ties to even, and 53 bits tell every quotient of two
    24-bit numbers from the half-integers (they differ by 2^-26 of it at least)."""
    s = scale.double()[:, None]
    return torch.where(s > 0, x.double() / torch.where(s > 0, s, 1.0), 0.0).round().clamp(-127, 127).to(torch.int8)


def run_quantize(x):
    n, k = x.shape
    codes = torch.full((n + 1, k), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((n + 1,), 7.0, device="cuda")
    q().coli_w8_quantize(x, codes[:n], scale[:n])
    assert (codes[n] == 99).all() and scale[n] == 7, "written behind the last token"
    return codes[:n], scale[:n]


def check_quantize(x):
    codes, scale = run_quantize(x)
    # one division, rounded once: 64 bits hold the quotient of two binary32 numbers well enough to round it again
    top = x.double().abs().amax(-1)
    want = (top / torch.tensor(127.0, dtype=torch.float64, device="cuda")).float()
    assert torch.equal(scale.isnan(), ~top.isfinite())   # a value that is not finite (binary16 has some here): NaN
    assert torch.equal(scale[top.isfinite()], want[top.isfinite()])
    assert torch.equal(codes, codes_of(x, scale))
    return codes, scale


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("n,k", [(1, 16), (1, 6144), (3, 48), (2, 4096), (5, 4112), (131, 1536), (2, 8192), (3, 8208),
                                 (2, 16384), (1, 65536), (1000, 112), (40, 240), (70, 1024), (9, 1040)])
def test_quantize(dtype, n, k):
    say("quantize", dtype, n, k)
    g = gen(n + k)
    x = torch.randn(n, k, generator=g, device="cuda") * torch.exp(3 * torch.randn(n, 1, generator=g, device="cuda"))
    check_quantize(x.to(dtype))


@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_quantize_ties_and_ends(dtype):
    """A scale that is a power of two puts half-integers on the border, all of them; signs, zeros, one value in a row."""
    say("quantize ties", dtype)
    k = 512
    x = torch.zeros(6, k, dtype=dtype, device="cuda")
    half = (torch.arange(254, device="cuda") - 126.5)
    x[0, :254], x[0, 254] = half.to(dtype), 127.0
    x[1, :254], x[1, 300] = (half / 32).to(dtype), -127.0 / 32
    x[2, 77] = -3.0
    x[4] = 1.5
    x[5, ::2], x[5, 1::2] = 127.0, 0.5
    codes, scale = check_quantize(x)
    assert scale[0] == 1 and scale[1] == 1 / 32 and scale[3] == 0 and not codes[3].any() and codes[2, 77] == -127
    assert (codes[0, :254] % 2 == 0).all() or dtype == BF   # bf16 does not hold the larger halves


def test_quantize_far_scales():
    """Scales below the normal numbers, and next to binary32's largest."""
    say("quantize far")
    g = gen(4)
    rows = [torch.randn(64, generator=g, device="cuda") * v for v in (1e-44, 1e-41, 1e-38, 1e-36, 1e-20, 1e37)]
    rows += [torch.full((64,), v, device="cuda") for v in (2.0 ** -149, 60 * 2.0 ** -149, 190 * 2.0 ** -149, 3.4e38)]
    check_quantize(torch.stack(rows))
    check_quantize((torch.randn(3, 64, generator=g, device="cuda") * 2.0 ** -130).to(BF))
    check_quantize((torch.randn(3, 64, generator=g, device="cuda") * 2.0 ** -23).to(FP))


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("k", [64, 6144])
def test_quantize_what_is_not_finite_stays_in_its_token(dtype, k):
    say("quantize nonfinite", dtype, k)
    x = torch.randn(5, k, generator=gen(3), device="cuda").to(dtype)
    x[1, 17], x[2, k - 1], x[3, 0] = NAN, INF, -INF
    codes, scale = run_quantize(x)
    assert scale[1:4].isnan().all() and not codes[1:4].any()
    keep = [0, 4]
    assert torch.equal(codes[keep], codes_of(x[keep], scale[keep])) and scale[keep].isfinite().all()


def test_quantize_strides():
    say("quantize strides")
    for dtype in (BF, F32):
        whole = torch.randn(9, 1024, generator=gen(8), device="cuda").to(dtype)
        for x in (whole[:, 16:528], whole[::2, :512], whole[:1].expand(4, -1), whole[:, 512:]):
            check_quantize(x)
    with pytest.raises(q().ColiError, match="token_stride"):
        run_quantize(torch.zeros(3, 70, device="cuda")[:, :64])
    with pytest.raises(q().ColiError, match="aligned"):
        run_quantize(torch.zeros(3, 80, device="cuda")[:, 1:65])


# ---------------------------------------------------------------- linear
def inputs(g, n, k, n_out, full=False):
    low = -128 if full else -127
    codes = torch.randint(-127, 128, (n, k), generator=g, device="cuda").to(torch.int8)
    w = torch.randint(low, 128, (n_out, k), generator=g, device="cuda").to(torch.int8)
    scale = torch.rand(n, generator=g, device="cuda") * 0.02 + 0.001
    w_scale = (torch.rand(n_out, generator=g, device="cuda") + 0.1) / (127 * math.sqrt(k))
    return codes, scale, w, w_scale


def exact_sums(codes, w):
    total = torch.zeros(codes.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for a in range(0, codes.shape[1], 512):   # sums of 512 products of codes are below 2^24
        total += codes[:, a:a + 512].float() @ w[:, a:a + 512].float().t()
    return total


def check_linear(codes, scale, w, w_scale, bias, out):
    q().coli_w8_linear(codes, scale, w, w_scale, bias, out)
    p = exact_sums(codes, w) * scale.double()[:, None] * w_scale.double()
    b = 0.0 if bias is None else bias.double()
    want = p + b
    # three roundings of the product, one of the sum with the bias, then the output's
    f32 = 3.01 * ref.U32 * p.abs() + 1.01 * ref.U32 * want.abs() + 4 * 2.0 ** -149
    u = 0.0 if out.dtype == F32 else U[out.dtype]
    ref.close(out, want, f32 + 1.01 * u * want.abs() + TINY[out.dtype], "out")


SHAPES = [  # tokens, k, n_out
    (1, 16, 1), (1, 6144, 256), (2, 48, 33), (1, 4096, 4099), (3, 1040, 1000), (4, 16384, 320), (7, 512, 31),
    (15, 272, 129), (16, 2048, 512), (17, 144, 257), (32, 6144, 96), (33, 128, 128), (61, 2064, 640), (64, 64, 63),
    (65, 160, 65), (100, 1536, 2112), (129, 112, 259), (255, 1024, 511), (256, 256, 1000), (300, 720, 770), (513, 384, 4097),
    (1034, 192, 300), (2050, 1536, 576), (1, 65536, 40), (90, 65536, 96)]


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("n,k,n_out", SHAPES)
def test_linear(dtype, n, k, n_out):
    say("linear", dtype, n, k, n_out)
    g = gen(n + k + n_out)
    codes, scale, w, w_scale = inputs(g, n, k, n_out, full=True)
    bias = torch.randn(n_out, generator=g, device="cuda") if (n + n_out) % 2 else None
    out = torch.full((n + 1, n_out), 7.0, dtype=dtype, device="cuda")
    check_linear(codes, scale, w, w_scale, bias, out[:n])
    assert (out[n] == 7).all(), "written behind the last token"


@pytest.mark.parametrize("n,k,n_out", [(4096, 512, 4096), (3001, 1024, 5003), (8192, 128, 1030)])
def test_linear_of_many_tiles(n, k, n_out):
    """More tiles than run at once, the last ones partly filled."""
    test_linear(BF, n, k, n_out)


@pytest.mark.parametrize("n", [1, 5, 40, 300])
def test_linear_extreme_codes(n):
    """The largest sums 32 bits have to hold: 2^16 products of 127 or -127 with -128."""
    say("linear extremes", n)
    k, n_out = 65536, 70
    codes = torch.full((n, k), 127, dtype=torch.int8, device="cuda")
    codes[::2] = -127
    w = torch.full((n_out, k), -128, dtype=torch.int8, device="cuda")
    out = torch.empty(n, n_out, device="cuda")
    check_linear(codes, torch.ones(n, device="cuda"), w, torch.ones(n_out, device="cuda"), None, out)
    assert (out[0] == 127 * 128 * k).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [3, 40, 300])
def test_linear_strides(dtype, n):
    """Codes out of wider rows, results into wider rows whose other elements stay."""
    say("linear strides", dtype, n)
    g = gen(n)
    k, n_out = 320, 515
    codes, scale, w, w_scale = inputs(g, n, k, n_out)
    wide = torch.full((n, 512), -128, dtype=torch.int8, device="cuda")
    wide[:, 96:416] = codes
    for off, width in ((0, 515), (1, 517), (8, 1024)):
        out = torch.full((n, width), 7.0, dtype=dtype, device="cuda")
        check_linear(wide[:, 96:416], scale, w, w_scale, None, out[:, off:off + n_out])
        rest = torch.ones(width, dtype=torch.bool, device="cuda")
        rest[off:off + n_out] = False
        assert (out[:, rest] == 7).all()
    check_linear(codes[:1].expand(n, -1), scale, w, w_scale, None, torch.empty(n, n_out, dtype=dtype, device="cuda"))


@pytest.mark.parametrize("n", [2, 33, 200])
def test_linear_passes_on_a_token_of_nan(n):
    say("linear nan", n)
    g = gen(n)
    codes, scale, w, w_scale = inputs(g, n, 256, 300)
    codes[1], scale[1] = 0, NAN
    out = torch.empty(n, 300, dtype=BF, device="cuda")
    q().coli_w8_linear(codes, scale, w, w_scale, None, out)
    assert out[1].isnan().all() and out.isnan().sum() == 300


def test_linear_on_another_stream_and_replayed():
    """A captured quantize and linear, replayed over new inputs, give what eager calls give."""
    say("w8 graph")
    m, g = q(), gen(6)
    for n in (1, 50, 400):
        k, n_out = 1024, 777
        _, _, w, w_scale = inputs(g, 1, k, n_out)
        x = torch.randn(n, k, generator=g, device="cuda")
        codes, scale = torch.empty(n, k, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
        out, side = torch.empty(n, n_out, device="cuda"), torch.cuda.Stream()

        def step(stream=None):
            m.coli_w8_quantize(x, codes, scale, stream=stream)
            m.coli_w8_linear(codes, scale, w, w_scale, None, out, stream=stream)
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        side.synchronize()
        first = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, first)
            x.copy_(torch.randn(n, k, generator=g, device="cuda"))
            step()
            first = out.clone()


def test_quantized_product_is_near_the_plain_one():
    """Together: the product of quantised activations and weights against the same in 64 bits.  Each value is off by half a
    step, amax / 254, at most; their errors are apart from each other, so a sum's stays within 6 of its deviations."""
    say("w8 together")
    n, k, n_out = 70, 1024, 600
    g = gen(12)
    x, wf = torch.randn(n, k, generator=g, device="cuda"), torch.randn(n_out, k, generator=g, device="cuda")
    codes, scale = check_quantize(x)
    w, w_scale = check_quantize(wf)
    out = torch.empty(n, n_out, device="cuda")
    q().coli_w8_linear(codes, scale, w, w_scale, None, out)
    want = x.double() @ wf.double().t()
    dev = ((scale.double() ** 2 / 12)[:, None] * wf.double().square().sum(1) + (w_scale.double() ** 2 / 12) * x.double().square().sum(1)[:, None]).sqrt()
    assert ((out.double() - want).abs() <= 6 * dev).all()
