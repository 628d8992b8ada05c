"""Decode behind a shared prefix on the GPU against the formulas in 64 bits (tests/mla_ref.py): rows that fill blocks or do
not, prefixes that end anywhere, sequences without tokens of their own, masks that reach into the prefix or leave a query
nothing, poisoned places that nothing may read, both cache formats and both types."""
import pytest
import torch

from tests import mla_ref as ref
from tests.gpu_util import q, say, status
from tests.test_gpu_mla import BF, FP, NAN, _outlier, cache, dims, gen, ok, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


@pytest.fixture(params=["together", "apart"], autouse=True)
def path(request, device):
    """Every test with the prefix read once for blocks of rows of all sequences, and by each sequence for itself."""
    q().coli_mla_debug_shared_path({"together": 1, "apart": 2}[request.param])
    yield request.param
    q().coli_mla_debug_shared_path(0)


def workspace(d, *sizes):
    ws = torch.zeros(q().coli_mla_shared_workspace_bytes(d, *sizes), dtype=torch.uint8, device="cuda")
    ws[256:] = 0xff   # stale partial results
    return ws


def reference(q_lat, q_pe, lat, key, prefix_table, prefix, table, lens, n_q, page, scale):
    n, h, rank = q_lat.shape
    out = torch.zeros(n, h, rank, dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full((n, h), -float("inf"), dtype=torch.float64, device="cuda")
    smag = torch.zeros_like(lse)
    before = ref.slots_of(prefix_table[None], 0, prefix, page)
    for b, m in enumerate(lens):
        at = torch.cat([before, ref.slots_of(table, b, m, page)])
        for j in range(n_q):
            seen = prefix + m - n_q + 1 + j
            if seen > 0:
                r = b * n_q + j
                c, k = lat[at[:seen]], key[at[:seen]]
                x, xp = q_lat[r].double(), q_pe[r].double()
                out[r], lse[r], mag[r] = ref.attend((x @ c.t() + xp @ k.t()) * scale, c)
                smag[r] = ((x.abs() @ c.abs().t() + xp.abs() @ k.abs().t()) * scale).amax(-1)
    return out, lse, mag, smag


def run(g, prefix, lens, n_q, heads, rank, dtype, fp8, page, poison=None, spread=1.0, max_kv=None, with_lse=True):
    pages, scale, table = cache(g, lens + [prefix], rank, dtype, fp8, page)
    need = -(-prefix // page)
    prefix_table, own = table[-1, :need].contiguous(), table[:-1].contiguous()
    d = dims(heads, rank, dtype, fp8, page, scale=192 ** -0.5)
    n = len(lens) * n_q
    q_lat, q_pe = (spread * randn(g, n, heads, rank)).to(dtype), randn(g, n, heads, 64, dtype=dtype)
    if poison:
        poison(pages, scale, table)
    top = max(lens + [0]) if max_kv is None else max_kv
    ws = workspace(d, len(lens), n_q, prefix, top)
    out = torch.full((n + 1, heads, rank), NAN, dtype=dtype, device="cuda")
    out[n] = 7
    lse = torch.full((n, heads), NAN, device="cuda")
    q().coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, prefix_table, prefix, own,
                               torch.tensor(lens, dtype=torch.int32, device="cuda"), top, out[:n], lse if with_lse else None, ws)
    ok(ws)
    assert (out[n] == 7).all(), "written behind the last row"
    lat, key = ref.rows_of(pages, scale, rank, dtype)
    want, wl, mag, smag = reference(q_lat, q_pe, lat, key, prefix_table, prefix, own, lens, n_q, page, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, rank + 64, prefix + max(lens + [1]), dtype)
    if fp8 and dtype == FP:   # binary16 weights end: see test_gpu_mla._decode_and_compare
        tol = tol + (prefix + sum(lens)) * 2.0 ** -23 * mag.amax(-1, keepdim=True)
    ref.close(out[:n], want, tol, "out")
    if with_lse:
        ref.close(lse, wl, tl, "lse")
    return out[:n], lse


CASES = [  # prefix, own lengths, n_q, heads, page
    (1, [1], 1, 1, 1), (31, [0], 1, 1, 16), (32, [5, 0, 33], 1, 5, 16), (33, [64, 1], 1, 16, 48), (100, [0, 0], 2, 3, 48),
    (65, [3, 7, 2], 4, 16, 16), (500, [129, 1, 63, 65, 0], 1, 64, 128), (1023, [20, 1, 300], 1, 128, 64), (777, [9, 40], 7, 5, 64),
    (2000, [31] * 9, 1, 33, 16), (64, [2, 2, 2], 4, 1, 16), (2, [0, 1, 4], 5, 6, 1), (96, [0, 3], 8, 16, 7)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rank,fp8", [(512, False), (512, True), (256, False), (256, True)])
@pytest.mark.parametrize("prefix,lens,n_q,heads,page", CASES)
def test_shared(dtype, rank, fp8, prefix, lens, n_q, heads, page):
    say("shared", dtype, rank, fp8, prefix, lens, n_q, heads, page)
    run(gen(prefix + rank), prefix, lens, n_q, heads, rank, dtype, fp8, page)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix,batch,n_q,heads", [(20011, 3, 1, 16), (9001, 1, 1, 128), (3000, 40, 1, 64), (700, 60, 4, 128),
                                                    (129, 130, 3, 5), (33, 4, 33, 256)])
def test_shared_many_rows_and_splits(fp8, prefix, batch, n_q, heads):
    """From one block of rows over a prefix that is shared out to every CU, to more blocks than CUs."""
    say("shared many", fp8, prefix, batch, n_q, heads)
    g = torch.Generator().manual_seed(batch)
    lens = [int(v) for v in torch.randint(0, 90, (batch,), generator=g)]
    run(gen(batch), prefix, lens, n_q, heads, 512 if heads > 64 else 256, BF, fp8, 16)


@pytest.mark.parametrize("dtype,fp8", [(BF, False), (FP, False), (BF, True), (FP, True)])
@pytest.mark.parametrize("prefix,lens,n_q,heads", [
    (1, [1], 1, 128), (31, [0, 0, 5], 1, 256), (700, [300, 0, 1, 33, 64], 2, 64), (64, [40] * 70, 1, 128), (9000, [5000, 3], 1, 128),
    (50, [2, 0, 31, 900], 4, 32), (3, [0, 1, 2, 3, 4], 8, 16), (100, [129, 7], 128, 1), (96, [257, 300, 31], 16, 128)])
def test_shared_blocks_of_one_sequence(dtype, fp8, prefix, lens, n_q, heads):
    """Rows of a sequence that fill blocks: its own tokens follow the prefix's there."""
    say("shared whole", dtype, fp8, prefix, lens, n_q, heads)
    run(gen(prefix + len(lens)), prefix, lens, n_q, heads, 512 if len(lens) < 6 else 256, dtype, fp8, 48)


def test_shared_many_sequences():
    """Own tokens in the plan of more than 64 sequences, whole and in parts."""
    say("shared sequences")
    g = torch.Generator().manual_seed(3)
    lens = [int(v) for v in torch.randint(0, 40, (150,), generator=g)]
    lens[70], lens[140] = 5000, 777
    run(gen(3), 70, lens, 1, 20, 256, FP, False, 16)
    run(gen(3), 70, lens, 2, 32, 256, BF, True, 16)
    run(gen(3), 70, lens, 2, 64, 256, BF, True, 16)


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_peaked_scores(fp8):
    """Scores of hundreds: the running maximum rises by steps that underflow the older weights."""
    say("shared peaked", fp8)
    run(gen(8), 1300, [700, 30], 2, 16, 512, BF, fp8, 16, spread=12.0)
    run(gen(8), 1300, [700, 30], 1, 40, 256, FP, fp8, 16, spread=12.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,n_q", [(5, 4), (64, 4), (24, 4)])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_shared_masked_tokens_may_hold_anything(fp8, heads, n_q, value):
    """The last tokens of the prefix are not finite: a query whose sequence begins so late does not see them."""
    say("shared poisoned", fp8, heads, n_q, value)
    page, prefix, rank, lens = 16, 77, 512, [1, 0, 3]

    def poison(pages, scale, table):
        flat = pages.view(-1, pages.shape[-1])
        s = ref.slots_of(table, len(lens), prefix, page)[-1]
        if fp8:
            flat[s, :rank] = 0x7f
            scale[s] = value
        else:
            flat[s] = value
    out, lse = run(gen(4), prefix, lens, n_q, heads, rank, BF, fp8, page, poison)
    out, lse = out.view(3, n_q, heads, rank), lse.view(3, n_q, heads)
    for b, m in enumerate(lens):
        clean = max(0, n_q - 1 - m)   # queries that end before the prefix's last token
        assert out[b, :clean].isfinite().all() and lse[b, :clean].isfinite().all() and out[b, clean:].isnan().any(-1).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,n_q", [(5, 4), (64, 4)])
def test_shared_unseen_drafts_may_hold_anything(fp8, heads, n_q):
    """The last own token is not finite: the queries before it do not see it."""
    for value in (NAN, float("inf")):
        say("shared poisoned drafts", fp8, heads, n_q, value)
        page, prefix, rank, lens = 16, 40, 512, [77, 4, 33]

        def poison(pages, scale, table):
            flat = pages.view(-1, pages.shape[-1])
            for b, n in enumerate(lens):
                s = ref.slots_of(table, b, n, page)[-1]
                if fp8:
                    flat[s, :rank] = 0x7f
                    scale[s] = value
                else:
                    flat[s] = value
        out, lse = run(gen(4), prefix, lens, n_q, heads, rank, BF, fp8, page, poison)
        out, lse = out.view(3, n_q, heads, rank), lse.view(3, n_q, heads)
        assert out[:, :-1].isfinite().all() and lse[:, :-1].isfinite().all() and out[:, -1].isnan().any(-1).all()


def test_shared_queries_that_see_nothing():
    say("shared nothing")
    for fp8 in (False, True):
        out, lse = run(gen(6), 2, [0, 1], 5, 7, 256, BF, fp8, 16)
        assert (out.view(2, 5, 7, 256)[0, :3] == 0).all() and (lse.view(2, 5, 7)[0, :3] == -float("inf")).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("times,down", [(2.0 ** 16, 60.0), (2.0 ** 26, 18.0), (2.0 ** 100, 800.0), (2.0 ** -40, 0.0), (0.0, -5.0)])
def test_shared_scale_of_one_token(dtype, times, down):
    """One token's scale far from the others', in the prefix's first and in a later tile."""
    say("shared scale of one", dtype, times, down)
    for at in (3, 66):
        change = _outlier(at, 256, 16, [100, 333], times, down, dtype)   # of both the sequence and the prefix
        g = gen(16)
        pages, scale, table = cache(g, [100, 333], 256, dtype, True, 16)
        change(pages, scale, table)
        q_lat, q_pe = randn(g, 1, 16, 256, dtype=dtype), torch.ones(1, 16, 64, dtype=dtype, device="cuda")
        q_lat[..., 0] = 0
        d = dims(16, 256, dtype, True, 16, scale=192 ** -0.5)
        ws = workspace(d, 1, 1, 333, 100)
        out, lse = torch.full((1, 16, 256), NAN, dtype=dtype, device="cuda"), torch.full((1, 16), NAN, device="cuda")
        q().coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, table[1].contiguous(), 333, table[:1, :7].contiguous(),
                                   torch.tensor([100], dtype=torch.int32, device="cuda"), 100, out, lse, ws)
        ok(ws)
        lat, key = ref.rows_of(pages, scale, 256, dtype)
        want, wl, mag, smag = reference(q_lat, q_pe, lat, key, table[1], 333, table[:1], [100], 1, 16, d.softmax_scale)
        tol, tl = ref.attend_tol(want, mag, smag, 320, 433, dtype)
        if dtype == FP:   # a weight below the least normal number of binary16: see test_gpu_mla._decode_and_compare
            tol = tol + 433 * 2.0 ** -23 * mag.amax(-1, keepdim=True)
        ref.close(out, want, tol, "out")
        ref.close(lse, wl, tl, "lse")


def test_shared_prefix_alone_and_none():
    """max_kv = 0 reads no page of the sequences; prefix_len = 0 is coli_mla_decode, bit for bit."""
    say("shared alone")
    for fp8 in (False, True):
        run(gen(1), 300, [0, 0, 0], 1, 16, 512, BF, fp8, 16, max_kv=0)
        run(gen(1), 300, [0, 5, 0], 1, 16, 512, BF, fp8, 16, with_lse=False)
        g, lens = gen(2), [40, 0, 133]
        pages, scale, table = cache(g, lens, 512, FP, fp8, 16)
        d = dims(16, 512, FP, fp8, 16, scale=0.07)
        q_lat, q_pe = randn(g, 3, 16, 512, dtype=FP), randn(g, 3, 16, 64, dtype=FP)
        kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
        got, want = (torch.full((3, 16, 512), NAN, dtype=FP, device="cuda") for _ in range(2))
        ws = workspace(d, 3, 1, 0, 133)
        q().coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, torch.zeros(0, dtype=torch.int32, device="cuda"), 0, table, kv, 133,
                                   got, None, ws)
        q().coli_mla_decode(d, q_lat, q_pe, pages, scale, table, kv, 133, want, None, ws)
        ok(ws)
        assert torch.equal(got, want)


def test_shared_agrees_with_decode():
    """Where the prefix ends with a page, the same queries over one table a sequence."""
    say("shared against decode")
    g, page, prefix, lens, heads = gen(5), 16, 160, [33, 0, 100], 16
    for fp8 in (False, True):
        pages, scale, table = cache(g, lens + [prefix], 512, BF, fp8, page)
        d = dims(heads, 512, BF, fp8, page, scale=0.07)
        q_lat, q_pe = randn(g, 3, heads, 512, dtype=BF), randn(g, 3, heads, 64, dtype=BF)
        whole = torch.cat([table[-1:, :10].expand(3, -1), table[:-1]], 1).contiguous()
        total = torch.tensor([prefix + n for n in lens], dtype=torch.int32, device="cuda")
        a, b = (torch.empty(3, heads, 512, dtype=BF, device="cuda") for _ in range(2))
        la, lb = (torch.empty(3, heads, device="cuda") for _ in range(2))
        ws = torch.zeros(q().coli_mla_workspace_bytes(d, 3, 1, 260), dtype=torch.uint8, device="cuda")
        q().coli_mla_decode(d, q_lat, q_pe, pages, scale, whole, total, 260, a, la, ws)
        ok(ws)
        ws = workspace(d, 3, 1, prefix, 100)
        q().coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, table[-1, :10].contiguous(), prefix, table[:-1].contiguous(),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), 100, b, lb, ws)
        ok(ws)
        # each is within half a step of bf16 of its weights, and rounded: 4 half-steps of what values reach apart
        lat, _ = ref.rows_of(pages, scale, 512, BF)
        reach = lat[torch.cat([ref.slots_of(table, i, n, page) for i, n in enumerate(lens + [prefix])])].abs().amax()
        assert ((a - b).abs() <= 4 * ref.U[BF] * reach).all() and ((la - lb).abs() <= 1e-4).all()


def test_shared_reports_bad_pages_and_lengths():
    """Ids and lengths outside what the call was given set the status; nothing outside the arrays is read."""
    say("shared bad pages")
    g, page = gen(3), 16
    d = dims(5, 256, BF, page=page, scale=0.07)
    pages, _, table = cache(g, [30, 40, 100], 256, BF, False, page)
    q_lat, q_pe = randn(g, 2, 5, 256, dtype=BF), randn(g, 2, 5, 64, dtype=BF)
    out, prefix = torch.empty(2, 5, 256, dtype=BF, device="cuda"), table[2, :7].contiguous()
    ws = workspace(d, 2, 1, 100, 48)

    def call(prefix_table=prefix, own=table[:2, :3].contiguous(), lens=(30, 40)):
        q().coli_mla_decode_shared(d, q_lat, q_pe, pages, None, prefix_table, 100, own,
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
    assert call() == 0


def test_shared_far_pages():
    """Byte offsets past 32 bits in a long cache."""
    say("shared far pages")
    g, page, rank, n = gen(2), 64, 512, 500
    n_pages = (1 << 32) // (page * 1152) + 40
    d = dims(16, rank, BF, page=page, scale=0.07)
    pages = torch.empty(n_pages, page, 576, dtype=BF, device="cuda")
    pages[n_pages - 9:] = randn(g, 9, page, 576, dtype=BF)
    prefix_table = torch.arange(n_pages - 1, n_pages - 9, -1, dtype=torch.int32, device="cuda")
    own = torch.full((1, 1), n_pages - 9, dtype=torch.int32, device="cuda")
    q_lat, q_pe = randn(g, 1, 16, rank, dtype=BF), randn(g, 1, 16, 64, dtype=BF)
    ws = workspace(d, 1, 1, n, 60)
    out, lse = torch.zeros(1, 16, rank, dtype=BF, device="cuda"), torch.zeros(1, 16, device="cuda")
    q().coli_mla_decode_shared(d, q_lat, q_pe, pages, None, prefix_table, n, own, torch.tensor([60], dtype=torch.int32, device="cuda"),
                               60, out, lse, ws)
    ok(ws)
    lat, key = ref.rows_of(pages[n_pages - 9:], None, rank, BF)
    near = n_pages - 9
    want, wl, mag, smag = reference(q_lat, q_pe, lat, key, prefix_table - near, n, own - near, [60], 1, page, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, 576, n + 60, BF)
    ref.close(out, want, tol, "out")
    ref.close(lse, wl, tl, "lse")


def test_shared_replayed():
    """A captured call, replayed while lengths and queries change in place, gives what eager calls give, bit for bit; a
    workspace for larger calls serves."""
    say("shared graph")
    m, g, page, prefix, lens, heads = q(), gen(11), 16, 333, [20, 0, 70, 5], 16
    for fp8 in (False, True):
        pages, scale, table = cache(g, [96] * 4 + [prefix], 512, BF, fp8, page)
        d = dims(heads, 512, BF, fp8, page, scale=0.07)
        q_lat, q_pe = randn(g, 4, heads, 512, dtype=BF), randn(g, 4, heads, 64, dtype=BF)
        kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
        own, prefix_table = table[:4, :6].contiguous(), table[4].contiguous()
        out, lse = torch.empty(4, heads, 512, dtype=BF, device="cuda"), torch.empty(4, heads, device="cuda")
        ws, side = workspace(d, 9, 2, 2000, 500), torch.cuda.Stream()

        def step(stream=None):
            m.coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, prefix_table, prefix, own, kv, 96, out, lse, ws, stream=stream)
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(4):
            kv.copy_(torch.tensor([(n + 7 * i) % 97 for n in lens], dtype=torch.int32))
            q_lat.copy_(randn(g, 4, heads, 512, dtype=BF))
            step()
            want = out.clone(), lse.clone()
            out.fill_(NAN)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        ok(ws)
