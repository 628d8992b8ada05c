"""Calls of the serving step's operators that stand at an edge: queries that are not finite, pages and lengths that are not
there where blocks of rows are of one sequence, pages named twice, calls on several streams at once."""
import pytest
import torch

from tests import mla_ref as ref
from tests.gpu_util import q, say, status
from tests.test_gpu_mla import BF, NAN, cache, dims, gen, ok, randn
from tests.test_gpu_shared import path, reference, workspace  # noqa: F401  (path: every test here that takes it, both ways)

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("value", [NAN, INF])
def test_shared_query_that_is_not_finite_reaches_no_other(fp8, heads, value):
    say("shared bad query", fp8, heads, value)
    g, page, prefix, lens = gen(heads), 16, 200, [33, 0, 70]
    pages, scale, table = cache(g, lens + [prefix], 512, BF, fp8, page)
    d = dims(heads, 512, BF, fp8, page, scale=0.07)
    q_lat, q_pe = randn(g, 3, heads, 512, dtype=BF), randn(g, 3, heads, 64, dtype=BF)
    kv, ws = torch.tensor(lens, dtype=torch.int32, device="cuda"), workspace(d, 3, 1, prefix, 70)

    def run():
        out = torch.empty(3, heads, 512, dtype=BF, device="cuda")
        q().coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, table[3].contiguous(), prefix, table[:3].contiguous(), kv, 70, out,
                                   None, ws)
        ok(ws)
        return out
    clean = run()
    q_lat[1, 5, 100] = value
    q_lat[1, 5, 101] = value   # products of both signs: no score of this query is finite
    out = run()
    rest = torch.ones(3, heads, dtype=torch.bool, device="cuda")
    rest[1, 5] = False
    assert clean.isfinite().all() and torch.equal(out[rest], clean[rest])


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_reports_bad_pages_and_lengths_of_whole_blocks(fp8):
    """Blocks of rows of one sequence read its own tokens too: what is not there sets the status, and nothing is read."""
    say("shared bad pages, whole blocks", fp8)
    g, page = gen(4), 16
    d = dims(64, 256, BF, fp8, page, scale=0.07)
    pages, scale, table = cache(g, [30, 40, 100], 256, BF, fp8, page)
    q_lat, q_pe = randn(g, 4, 64, 256, dtype=BF), randn(g, 4, 64, 64, dtype=BF)
    out, prefix = torch.empty(4, 64, 256, dtype=BF, device="cuda"), table[2, :7].contiguous()
    ws = workspace(d, 2, 2, 100, 48)

    def call(prefix_table=prefix, own=table[:2, :3].contiguous(), lens=(30, 40)):
        q().coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, prefix_table, 100, own,
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), 48, out, None, ws)
        return status(ws)
    assert call() == 0
    for bad in (-1, pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        broken = prefix.clone()
        broken[6] = bad
        assert call(prefix_table=broken) == q().COLI_EINVAL
        broken = table[:2, :3].contiguous()
        broken[1, 2] = bad
        assert call(own=broken) == q().COLI_EINVAL
    assert call(lens=(30, 49)) == q().COLI_EINVAL and call(lens=(-1, 40)) == q().COLI_EINVAL
    assert call(lens=(2 ** 31 - 1, 40)) == q().COLI_EINVAL and call(lens=(-2 ** 31, 40)) == q().COLI_EINVAL
    assert call() == 0


@pytest.mark.parametrize("heads,n_q", [(16, 1), (64, 2)])
def test_shared_pages_named_twice(heads, n_q, path):  # noqa: F811
    """A page may stand in the prefix twice, and be a page of two sequences as well."""
    say("shared pages twice", heads, n_q, path)
    g, page = gen(6), 16
    pages, _, _ = cache(g, [64], 256, BF, False, page, spare=0)
    prefix_table = torch.tensor([1, 1, 0, 3, 1], dtype=torch.int32, device="cuda")
    own = torch.tensor([[1, 2], [1, 1]], dtype=torch.int32, device="cuda")
    d, lens, prefix = dims(heads, 256, BF, page=page, scale=0.07), [20, 32], 75
    q_lat, q_pe = randn(g, 2 * n_q, heads, 256, dtype=BF), randn(g, 2 * n_q, heads, 64, dtype=BF)
    ws, out = workspace(d, 2, n_q, prefix, 32), torch.empty(2 * n_q, heads, 256, dtype=BF, device="cuda")
    pages = torch.nan_to_num(pages)
    q().coli_mla_decode_shared(d, q_lat, q_pe, pages, None, prefix_table, prefix, own,
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 32, out, None, ws)
    ok(ws)
    lat, key = ref.rows_of(pages, None, 256, BF)
    want, _, mag, smag = reference(q_lat, q_pe, lat, key, prefix_table, prefix, own, lens, n_q, page, d.softmax_scale)
    ref.close(out, want, ref.attend_tol(want, mag, smag, 320, prefix + 32, BF)[0], "out")


def test_products_and_selection_on_four_streams():
    """Calls of all sizes beside one another give what they give alone."""
    say("four streams")
    m, g = q(), gen(21)
    d = m.make_select_dims(160, 6, 8, 3)
    work = []
    for n, k, n_out in ((1, 6144, 2048), (61, 1024, 6144), (133, 512, 4097), (700, 768, 1030)):
        x = torch.randn(n, k, generator=g, device="cuda")
        w = torch.randint(-127, 128, (n_out, k), generator=g, device="cuda").to(torch.int8)
        w_scale, logits = torch.rand(n_out, generator=g, device="cuda"), torch.randn(7 * n, 160, generator=g, device="cuda")
        work.append((x, w, w_scale, logits))

    def run(x, w, w_scale, logits):
        codes, scale = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
        out = torch.empty(len(x), len(w), device="cuda")
        idx, weights = torch.empty(len(logits), 6, dtype=torch.int32, device="cuda"), torch.empty(len(logits), 6, device="cuda")
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        m.coli_w8_quantize(x, codes, scale)
        m.coli_w8_linear(codes, scale, w, w_scale, None, out)
        m.coli_moe_select(d, logits, None, idx, weights, ws)
        return codes, scale, out, idx, weights
    alone = [run(*a) for a in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for _ in range(3):
        got = []
        for a, stream in zip(work, streams):
            with torch.cuda.stream(stream):
                got.append(run(*a))
        torch.cuda.synchronize()
        for g_, w_ in zip(got, alone):
            assert all(torch.equal(a, b) for a, b in zip(g_, w_))
