"""Shared decode as it comes, with the library's own choice of how the prefix is read, on both sides of that choice; and call
after call, bit for bit, whatever the workspace held before."""
import pytest
import torch

from tests import mla_ref as ref
from tests.gpu_util import q, say
from tests.test_gpu_mla import BF, FP, NAN, cache, dims, gen, ok, randn
from tests.test_gpu_shared import reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


@pytest.fixture(autouse=True)
def restored(device):
    q().coli_mla_debug_shared_path(0)
    yield
    q().coli_mla_debug_shared_path(0)


def make(g, prefix, lens, n_q, heads, rank, dtype, fp8, page):
    pages, scale, table = cache(g, lens + [prefix], rank, dtype, fp8, page)
    d, n = dims(heads, rank, dtype, fp8, page, scale=192 ** -0.5), len(lens) * n_q
    q_lat, q_pe = randn(g, n, heads, rank, dtype=dtype), randn(g, n, heads, 64, dtype=dtype)
    prefix_table, own = table[-1, :-(-prefix // page)].contiguous(), table[:-1].contiguous()
    kv, top = torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens)
    need = q().coli_mla_shared_workspace_bytes(d, len(lens), n_q, prefix, top)

    def call(fill=0xff):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        out = torch.full((n, heads, rank), NAN, dtype=dtype, device="cuda")
        lse = torch.full((n, heads), NAN, device="cuda")
        q().coli_mla_decode_shared(d, q_lat, q_pe, pages, scale, prefix_table, prefix, own, kv, top, out, lse, ws)
        ok(ws)
        return out, lse

    def compare(out, lse):
        lat, key = ref.rows_of(pages, scale, rank, dtype)
        want, wl, mag, smag = reference(q_lat, q_pe, lat, key, prefix_table, prefix, own, lens, n_q, page, d.softmax_scale)
        tol, tl = ref.attend_tol(want, mag, smag, rank + 64, prefix + top, dtype)
        if fp8 and dtype == FP:   # binary16 weights end: see test_gpu_mla._decode_and_compare
            tol = tol + (prefix + sum(lens)) * 2.0 ** -23 * mag.amax(-1, keepdim=True)
        ref.close(out, want, tol, "out")
        ref.close(lse, wl, tl, "lse")
    return call, compare


# prefix, batch, n_q, heads, rank, E4M3, and how the prefix is read: 1 once for all, 2 by each sequence
CHOICES = [(2000, 4, 1, 16, 512, False, 2), (9000, 48, 1, 16, 512, False, 1), (300, 40, 1, 64, 512, False, 2),
           (33000, 16, 2, 64, 512, False, 1), (3000, 8, 1, 128, 256, False, 2), (1000, 6, 1, 16, 512, True, 2),
           (9000, 64, 1, 16, 512, True, 1), (20000, 64, 1, 5, 256, True, 1), (2000, 5, 4, 32, 512, True, 2)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("prefix,batch,n_q,heads,rank,fp8,way", CHOICES)
def test_shared_by_choice(dtype, prefix, batch, n_q, heads, rank, fp8, way):
    say("shared, by choice", dtype, prefix, batch, n_q, heads, rank, fp8)
    lens = [(37 * b) % 90 for b in range(batch)]
    call, compare = make(gen(prefix), prefix, lens, n_q, heads, rank, dtype, fp8, 16)
    out, lse = call()
    compare(out, lse)
    q().coli_mla_debug_shared_path(way)
    forced = call()
    assert torch.equal(out, forced[0]) and torch.equal(lse, forced[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix,batch,n_q,heads", [(2047, 8, 1, 16), (1500, 9, 1, 128), (700, 33, 2, 5), (333, 1, 1, 64)])
def test_shared_repeats_itself(fp8, prefix, batch, n_q, heads):
    """No sum depends on which workgroup is first, nor on what lay in the workspace."""
    say("shared, repeated", fp8, prefix, batch, n_q, heads)
    call, _ = make(gen(heads), prefix, [(53 * b) % 300 for b in range(batch)] if batch > 1 else [7], n_q, heads, 512, BF, fp8, 64)
    for way in (0, 1, 2):
        q().coli_mla_debug_shared_path(way)
        first = call()
        for fill in (0xff, 0, 0x3c, 0x80, 0x7f):
            again = call(fill)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]), (way, fill)
