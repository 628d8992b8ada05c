"""Latent attention on the GPU against the formulas in 64 bits (tests/mla_ref.py): odd sizes, empty sequences, masks
that leave a row nothing, pages that end anywhere, strides, poisoned places that nothing may read, both cache formats
and both types."""
import math

import pytest
import torch

from tests import mla_ref as ref
from tests.gpu_util import q, say, status

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def dims(heads=5, rank=512, dtype=BF, fp8=False, page=48, halves=False, nope=128, v=128, eps=1e-6, scale=None):
    m = q()
    return m.make_mla_dims(heads, rank, nope, v, page, dtype, m.COLI_KV_E4M3 if fp8 else m.COLI_KV_PLAIN,
                           m.COLI_ROPE_HALVES if halves else m.COLI_ROPE_PAIRS, eps, scale)


def workspace(d, *sizes):
    return torch.zeros(q().coli_mla_workspace_bytes(d, *sizes), dtype=torch.uint8, device="cuda")


def ok(ws):
    assert status(ws) == 0, q().coli_moe_last_error()


def cache(g, lens, rank, dtype, fp8, page, spare=3, width=None):
    """A pool whose every place outside the sequences holds NaN, and the sequences' pages in no order."""
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + spare
    table = torch.full((len(lens), max(1, width or max(need))), -7, dtype=torch.int32, device="cuda")
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    lat, key = randn(g, n_pages, page, rank), randn(g, n_pages, page, ref.ROPE).to(dtype)
    used = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        if n:
            used.view(-1)[ref.slots_of(table, b, n, page)] = True
    if fp8:
        s = lat.abs().amax(-1) / 448 * (0.25 + torch.rand(n_pages, page, generator=g, device="cuda"))
        codes = (lat / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes[~used] = 0x7f
        key[~used] = NAN
        s[~used] = NAN
        pages = torch.cat([codes, key.contiguous().view(torch.uint8)], -1).contiguous()
        return pages, s.reshape(-1).contiguous(), table
    pages = torch.cat([lat.to(dtype), key], -1)
    pages[~used] = NAN
    return pages.contiguous(), None, table


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rank,fp8,halves,with_norm", [(512, False, False, True), (512, True, True, True),
                                                       (256, True, False, True), (256, False, True, False),
                                                       (512, True, False, False)])
@pytest.mark.parametrize("n,heads", [(1, 1), (3, 5), (131, 16), (40, 128)])
def test_append(dtype, rank, fp8, halves, with_norm, n, heads):
    say("append", dtype, rank, fp8, halves, with_norm, n, heads)
    g = gen(n + rank)
    page = 7
    n_pages = n // page + 3
    d = dims(heads, rank, dtype, fp8, page, halves)
    kv_a = randn(g, n, rank + 64, dtype=dtype)
    kv_a[0, :rank] = 0   # a latent of zeros: scale 0, codes 0
    gain = (1 + 0.1 * randn(g, rank)).to(dtype) if with_norm else None
    positions = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    positions[-1] = 2 ** 31 - 1
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:n].long()
    if n > 2:
        slots[1] = -1
    freq = 10000.0 ** (-torch.arange(0, 64, 2, device="cuda", dtype=torch.float64) / 64)
    whole = randn(g, n, heads, 192, dtype=dtype)
    q_pe = whole[..., 128:]
    out = torch.full((n, heads, 64), NAN, dtype=dtype, device="cuda")
    row = q().coli_mla_row_bytes(d)
    raw = torch.randint(0, 255, (n_pages, page, row), generator=g, device="cuda", dtype=torch.uint8)
    pages = raw.clone() if fp8 else raw.clone().view(dtype)
    scale = torch.full((n_pages * page,), 5.0, device="cuda") if fp8 else None
    ws = workspace(d)
    q().coli_mla_append(d, kv_a, gain, positions, slots, freq, q_pe, out, pages, scale, ws)
    ok(ws)
    u = ref.U[dtype]
    rot_tol = lambda want, x: 1.01 * u * want.abs() + 16 * ref.U32 * x.double().abs().amax(-1, keepdim=True) * 2 + ref.TINY[dtype]
    want = ref.rotate(q_pe, positions, freq, halves)
    ref.close(out, want, rot_tol(want, q_pe), "q_pe")
    keep = slots >= 0
    got = pages.view(torch.uint8).view(-1, row)
    others = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    others[slots[keep]] = False
    assert torch.equal(got[others], raw.view(-1, row)[others]), "a slot that is not the call's was written"
    lat, key = ref.rows_of(pages, scale, rank, dtype)
    want = ref.rotate(kv_a[:, rank:], positions, freq, halves)[keep]
    ref.close(key[slots[keep]], want, rot_tol(want, kv_a[keep, rank:]), "key")
    want = ref.norm(kv_a[:, :rank], gain, 1e-6)[keep]
    rel = (rank + 16) * ref.U32
    if fp8:
        top = want.abs().amax(-1)
        ref.close(scale[slots[keep]], top / 448, 2 * rel * top / 448, "scale")
        # half a step of a normal code, 2^-4 of it, or of the subnormals, 2^-10, in units of the scale
        ref.close(lat[slots[keep]], want, (2.0 ** -4 + 4 * rel) * want.abs() + (2.0 ** -10 + rel) * (top / 448)[:, None], "latent")
        assert (scale[others] == 5.0).all()
        if 0 in slots[keep][:0] or keep[0]:
            assert scale[slots[0]] == 0 and (got[slots[0], :rank] & 0x7f == 0).all()
    else:
        ref.close(lat[slots[keep]], want, (u * 1.01 + rel) * want.abs() + ref.TINY[dtype], "latent")


def test_append_in_place_and_without_queries():
    say("append in place")
    g, n, heads = gen(5), 9, 6
    d = dims(heads, 256, FP, page=16)
    kv_a, freq = randn(g, n, 320, dtype=FP), torch.rand(32, device="cuda", dtype=torch.float64)
    positions, slots = torch.arange(n, device="cuda", dtype=torch.int32) + 70000, torch.arange(n, device="cuda")
    whole = randn(g, n, heads, 192, dtype=FP)
    out = torch.zeros(n, heads, 64, dtype=FP, device="cuda")
    a, b = (torch.zeros(2, 16, 320, dtype=FP, device="cuda") for _ in range(2))
    ws = workspace(d)
    q().coli_mla_append(d, kv_a, None, positions, slots, freq, whole[..., 128:], out, a, None, ws)
    before = whole[..., :128].clone()
    q().coli_mla_append(d, kv_a, None, positions, slots, freq, whole[..., 128:], whole[..., 128:], b, None, ws)
    assert torch.equal(whole[..., 128:], out) and torch.equal(whole[..., :128], before) and torch.equal(a, b)
    b.zero_()
    q().coli_mla_append(d, kv_a, None, positions, slots, freq, None, None, b, None, ws)
    ok(ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("n,heads", [(1, 6), (9, 6), (9, 1)])
def test_append_query_layouts(n, heads, monkeypatch):
    """Rotated queries go to any layout whose runs of 64 lie apart, heads outermost too; others are refused."""
    say("append layouts", n, heads)
    m, g = q(), gen(5)
    for entry in m.MLA_EXPORTS[2:]:   # the checks alone launch
        monkeypatch.setattr(m._lib, entry, None)
    d = dims(heads, 256, BF, page=16)
    kv_a, freq, q_pe = randn(g, n, 320, dtype=BF), torch.rand(32, device="cuda", dtype=torch.float64), randn(g, n, heads, 64, dtype=BF)
    positions, slots = torch.arange(n, device="cuda", dtype=torch.int32), torch.arange(n, device="cuda")
    pages, ws = torch.zeros(2, 16, 320, dtype=BF, device="cuda"), workspace(d)

    def run(out):
        m.coli_mla_append(d, kv_a, None, positions, slots, freq, q_pe, out, pages, None, ws)
        ok(ws)
        return out
    want = run(torch.empty(n, heads, 64, dtype=BF, device="cuda"))
    assert torch.equal(run(torch.empty(heads, n, 64, dtype=BF, device="cuda").transpose(0, 1)), want)
    assert torch.equal(run(torch.empty(heads, n + 3, 72, dtype=BF, device="cuda")[:, :n, :64].transpose(0, 1)), want)
    assert torch.equal(run(torch.empty(n, heads, 192, dtype=BF, device="cuda")[..., 128:]), want)
    if n * heads > 9:
        for strides in ((0, 64), (64, 0), (64, 64), (8, 64 * 9)):
            with pytest.raises(ValueError, match="overlap"):
                run(torch.empty(heads * n * 64, dtype=BF, device="cuda").as_strided((n, heads, 64), (*strides, 1)))
    empty = torch.empty(0, heads, 256, dtype=BF, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    m.coli_mla_decode(d, empty, empty[..., :64].contiguous(), pages, None, torch.empty(0, 1, dtype=torch.int32, device="cuda"),
                      lens, 5, empty, None, ws)


def test_append_reports_a_slot_behind_the_cache():
    say("append bad slot")
    d = dims(1, 256, page=4)
    pages = torch.zeros(2, 4, 320, dtype=BF, device="cuda")
    ws = workspace(d)
    freq = torch.zeros(32, device="cuda", dtype=torch.float64)
    q().coli_mla_append(d, torch.ones(2, 320, dtype=BF, device="cuda"), None,
                        torch.zeros(2, device="cuda", dtype=torch.int32), torch.tensor([8, 3], device="cuda"), freq, None,
                        None, pages, None, ws)
    assert status(ws) == q().COLI_EINVAL and "slot" in q().coli_moe_last_error()
    assert (pages.view(8, 320)[3] == 1).all() and pages.view(8, 320)[:3].abs().sum() == 0
    ok(ws)


def test_append_keeps_a_nan_visible():
    say("append nan")
    for fp8 in (False, True):
        d = dims(1, 256, FP, fp8, page=4)
        kv_a = torch.ones(2, 320, dtype=FP, device="cuda")
        kv_a[0, 17] = NAN
        pages = torch.zeros(2, 4, 384 if fp8 else 320, dtype=torch.uint8 if fp8 else FP, device="cuda")
        scale = torch.zeros(8, device="cuda") if fp8 else None
        ws = workspace(d)
        q().coli_mla_append(d, kv_a, torch.ones(256, dtype=FP, device="cuda"),
                            torch.zeros(2, device="cuda", dtype=torch.int32), torch.tensor([0, 1], device="cuda"),
                            torch.zeros(32, device="cuda", dtype=torch.float64), None, None, pages, scale, ws)
        ok(ws)
        lat, _ = ref.rows_of(pages, scale, 256, FP)
        assert lat[0].isnan().all() and not lat[1].isnan().any()


def test_append_scale_below_the_normal_numbers():
    """E4M3: a scale so small that its own rounding brings codes past 448, the largest (values of 655 steps of binary32's
    subnormals, a scale of 1.46 of them)."""
    say("append small scale")
    d = dims(1, 256, BF, True, page=4, eps=1e4)
    pages, scale, ws = torch.zeros(2, 4, 384, dtype=torch.uint8, device="cuda"), torch.zeros(8, device="cuda"), workspace(d)
    kv_a, gain = torch.ones(3, 320, dtype=BF, device="cuda"), torch.full((256,), 2.0 ** -133, dtype=BF, device="cuda")
    kv_a[1] = -1
    kv_a[2, 7] = NAN
    q().coli_mla_append(d, kv_a, gain, torch.zeros(3, device="cuda", dtype=torch.int32), torch.arange(3, device="cuda"),
                        torch.zeros(32, device="cuda", dtype=torch.float64), None, None, pages, scale, ws)
    ok(ws)
    lat, _ = ref.rows_of(pages, scale, 256, BF)
    assert (lat[0] == 448 * 2.0 ** -149).all() and (lat[1] == -448 * 2.0 ** -149).all() and lat[2].isnan().all()


# ---------------------------------------------------------------- project
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,heads,n_in,n_out", [
    (1, 1, 64, 64), (1, 5, 192, 512), (3, 64, 512, 128), (5, 16, 128, 256), (16, 7, 192, 512), (17, 5, 512, 256),
    (33, 3, 128, 512), (64, 2, 256, 128), (600, 2, 192, 512), (513, 3, 64, 192), (133, 9, 512, 128), (300, 5, 192, 512), (257, 1, 1024, 320), (129, 2, 64, 4096)])
def test_project(dtype, n, heads, n_in, n_out):
    say("project", dtype, n, heads, n_in, n_out)
    g = gen(n * heads)
    x = randn(g, n, heads, n_in + 64, dtype=dtype)[..., :n_in]   # the unrotated part of whole queries
    w = (randn(g, heads, n_out, n_in) / math.sqrt(n_in)).to(dtype)
    out = torch.full((n + 1, heads, n_out), 7.0, dtype=dtype, device="cuda")
    q().coli_mla_project(x, w, out[:n])
    xt, wt = x.double().transpose(0, 1), w.double().transpose(1, 2)
    want = torch.matmul(xt, wt).transpose(0, 1)
    mag = torch.matmul(xt.abs(), wt.abs()).transpose(0, 1)
    ref.close(out[:n], want, 1.01 * ref.U[dtype] * want.abs() + n_in * ref.U32 * mag + ref.TINY[dtype], "out")
    assert (out[n] == 7).all(), "written behind the last token"


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n,heads,n_in,n_out", [(300, 20, 192, 512), (517, 37, 64, 192), (259, 67, 512, 64), (513, 33, 512, 320),
                                                (770, 48, 256, 192), (40, 150, 1024, 320), (257, 96, 320, 512)])
def test_project_of_many_heads(dtype, n, heads, n_in, n_out):
    """Products of more tiles than run at once, whose last tokens and features do not fill a tile."""
    test_project(dtype, n, heads, n_in, n_out)


# ---------------------------------------------------------------- decode
def run_decode(g, lens, n_q, heads, rank, dtype, fp8, page, poison=None, spread=1.0, max_kv=None, with_lse=True):
    pages, scale, table = cache(g, lens, rank, dtype, fp8, page)
    d = dims(heads, rank, dtype, fp8, page, scale=192 ** -0.5)
    n = len(lens) * n_q
    q_lat, q_pe = (spread * randn(g, n, heads, rank)).to(dtype), randn(g, n, heads, 64, dtype=dtype)
    if poison:
        poison(pages, scale, table)
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    top = max(lens) if max_kv is None else max_kv
    ws = workspace(d, len(lens), n_q, top)
    ws[256:] = 0xff   # stale partial results
    out = torch.full((n, heads, rank), NAN, dtype=dtype, device="cuda")
    lse = torch.full((n, heads), NAN, device="cuda")
    q().coli_mla_decode(d, q_lat, q_pe, pages, scale, table, kv_lens, top, out, lse if with_lse else None, ws)
    ok(ws)
    lat, key = ref.rows_of(pages, scale, rank, dtype)
    want, wl, mag, smag = ref.decode(q_lat, q_pe, lat, key, table, lens, n_q, page, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, rank + 64, max(lens + [1]), dtype)
    ref.close(out, want, tol, "out")
    if with_lse:
        ref.close(lse, wl, tl, "lse")
    return out, lse


DECODE = [  # lens, n_q, heads, page
    ([1], 1, 1, 1), ([1, 0, 2], 1, 5, 16), ([0, 0], 2, 3, 48), ([33, 1, 64], 4, 16, 16), ([63, 65, 129, 0, 7], 1, 64, 48),
    ([1023], 1, 16, 16), ([5, 300, 2], 7, 5, 64), ([777, 31, 1500], 1, 128, 64), ([200, 90], 3, 33, 128),
    ([4000, 17], 2, 32, 1), ([2500], 4, 64, 64)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rank,fp8", [(512, False), (512, True), (256, False), (256, True)])
@pytest.mark.parametrize("lens,n_q,heads,page", DECODE)
def test_decode(dtype, rank, fp8, lens, n_q, heads, page):
    say("decode", dtype, rank, fp8, lens, n_q, heads, page)
    run_decode(gen(sum(lens) + rank), lens, n_q, heads, rank, dtype, fp8, page)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,n_q", [(16, 1), (64, 1), (128, 2)])
def test_decode_many_splits(fp8, heads, n_q):
    """Work shared out over the whole GPU: one long sequence among short ones."""
    lens = [20011, 1, 0, 640, 64, 63, 9000, 129]
    say("decode splits", fp8, heads, n_q)
    run_decode(gen(3), lens, n_q, heads, 512, BF, fp8, 64)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch,n_q,heads,top", [(100, 1, 3, 200), (62, 33, 256, 40), (300, 2, 20, 70)])
def test_decode_many_sequences(fp8, batch, n_q, heads, top):
    """More sequences than a wavefront has lanes, and so many rows that one workgroup goes through all sequences."""
    say("decode many", fp8, batch, n_q, heads)
    g = torch.Generator().manual_seed(batch)
    lens = [int(v) for v in torch.randint(0, top + 1, (batch,), generator=g)]
    run_decode(gen(batch), lens, n_q, heads, 256, BF, fp8, 16)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_peaked_scores(fp8):
    """Scores of hundreds: one key takes all, the running maximum rises by steps that underflow the older weights."""
    say("decode peaked", fp8)
    run_decode(gen(8), [700, 1300], 2, 16, 512, BF, fp8, 16, spread=12.0)
    run_decode(gen(8), [700, 1300], 1, 40, 256, FP, fp8, 16, spread=12.0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,n_q", [(5, 4), (64, 4)])
def test_decode_masked_tokens_may_hold_anything(fp8, heads, n_q):
    """The last token of a sequence is NaN (then infinite): the earlier queries do not see it."""
    for value in (NAN, float("inf")):
        say("decode poisoned", fp8, heads, n_q, value)
        page, lens, rank = 16, [77, 300], 512

        def poison(pages, scale, table):
            flat = pages.view(-1, pages.shape[-1])
            for b, n in enumerate(lens):
                s = ref.slots_of(table, b, n, page)[-1]
                if fp8:
                    flat[s, :rank] = 0x7f
                    scale[s] = value
                else:
                    flat[s] = value
        out, lse = run_decode(gen(4), lens, n_q, heads, rank, BF, fp8, page, poison)
        for b in range(2):
            assert out[b * n_q:(b + 1) * n_q - 1].isfinite().all() and lse[b * n_q:(b + 1) * n_q - 1].isfinite().all()
            assert out[(b + 1) * n_q - 1].isnan().any()


def test_decode_scales_far_apart():
    """E4M3 scales over ten powers of two, fp16 activations."""
    say("decode scales")

    def poison(pages, scale, table):
        scale *= torch.exp2(torch.arange(scale.numel(), device="cuda") % 11 - 5.0)
    run_decode(gen(9), [400, 90], 2, 16, 512, FP, True, 16, poison)
    run_decode(gen(9), [400, 90], 1, 64, 512, BF, True, 16, poison)


def _outlier(at, rank, page, lens, times, down, dtype):
    """Token `at` of each sequence: a scale of `times` and a latent of one column, which it has alone and no query looks
    at, and a key that lowers its score by about `down`."""
    def change(pages, scale, table):
        flat = pages.view(-1, pages.shape[-1])
        flat[:, 0] = 0
        for b, n in enumerate(lens):
            s = int(ref.slots_of(table, b, n, page)[at])
            flat[s, 1:rank] = 0
            flat[s, 0] = 0x7e   # 448
            scale[s] = times / 448
            flat[s, rank:].view(dtype)[:] = -down / (64 * 192 ** -0.5)
    return change


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("heads,n_q", [(16, 1), (64, 1), (16, 4)])
@pytest.mark.parametrize("times,down", [(2.0 ** 16, 60.0), (2.0 ** 26, 60.0), (2.0 ** 26, 18.0), (2.0 ** 100, 800.0),
                                        (2.0 ** 100, 104.0), (2.0 ** -40, 0.0), (0.0, -5.0)])
def test_decode_scale_of_one_token(dtype, heads, n_q, times, down):
    """One token's scale far from the others': a token of no weight takes nothing from them, one whose small weight times
    its scale counts is counted, one whose weight times its scale is nothing leaves the others their precision."""
    say("decode scale of one", dtype, heads, n_q, times, down)
    rank, page, lens = 256, 16, [70, 333]
    for at in (3, 66):   # in a sequence's first tile, in a later one
        g = gen(heads)
        pages, scale, table = cache(g, lens, rank, dtype, True, page)
        _outlier(at, rank, page, lens, times, down, dtype)(pages, scale, table)
        n = len(lens) * n_q
        q_lat, q_pe = randn(g, n, heads, rank, dtype=dtype), torch.ones(n, heads, 64, dtype=dtype, device="cuda")
        q_lat[..., 0] = 0
        _decode_and_compare(q_lat, q_pe, pages, scale, table, lens, n_q, page, dtype)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("heads,n_q", [(5, 4), (64, 2)])
def test_decode_scale_of_an_unseen_token(dtype, heads, n_q):
    """The last draft token's scale is 2^26 times the others': the queries before it have the bits they have without."""
    say("decode unseen scale", dtype, heads, n_q)
    rank, page, lens = 512, 16, [77, 300]
    outs = []
    for times in (1.0, 2.0 ** 26):
        g = gen(7)
        pages, scale, table = cache(g, lens, rank, dtype, True, page)
        for b, n in enumerate(lens):
            scale[ref.slots_of(table, b, n, page)[-1]] *= times
        n = len(lens) * n_q
        q_lat, q_pe = randn(g, n, heads, rank, dtype=dtype), randn(g, n, heads, 64, dtype=dtype)
        d = dims(heads, rank, dtype, True, page, scale=192 ** -0.5)
        ws = workspace(d, len(lens), n_q, max(lens))
        out, lse = torch.full((n, heads, rank), NAN, dtype=dtype, device="cuda"), torch.full((n, heads), NAN, device="cuda")
        q().coli_mla_decode(d, q_lat, q_pe, pages, scale, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens),
                            out, lse, ws)
        ok(ws)
        outs.append((out.view(len(lens), n_q, heads, rank)[:, :-1], lse.view(len(lens), n_q, heads)[:, :-1]))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("power", [-134, -120, 60])
@pytest.mark.parametrize("lens,heads,n_q", [([40, 333], 5, 2), ([9000], 64, 1)])
def test_decode_small_and_large_scales(power, lens, heads, n_q):
    """All scales at the ends of binary32's range, below its normal numbers too; keys alone make the scores."""
    say("decode scales at the ends", power, lens, heads)
    rank, page = 512, 64
    g = gen(heads)
    pages, scale, table = cache(g, lens, rank, BF, True, page)
    scale *= 2.0 ** (power / 2)
    scale *= 2.0 ** (power / 2)
    n = len(lens) * n_q
    q_lat, q_pe = torch.zeros(n, heads, rank, dtype=BF, device="cuda"), randn(g, n, heads, 64, dtype=BF)
    _decode_and_compare(q_lat, q_pe, pages, scale, table, lens, n_q, page, BF)


def _decode_and_compare(q_lat, q_pe, pages, scale, table, lens, n_q, page, dtype):
    n, heads, rank = q_lat.shape
    d = dims(heads, rank, dtype, scale is not None, page, scale=192 ** -0.5)
    ws = workspace(d, len(lens), n_q, max(lens))
    ws[256:] = 0xff   # stale partial results
    out, lse = torch.full((n, heads, rank), NAN, dtype=dtype, device="cuda"), torch.full((n, heads), NAN, device="cuda")
    q().coli_mla_decode(d, q_lat, q_pe, pages, scale, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens),
                        out, lse, ws)
    ok(ws)
    lat, key = ref.rows_of(pages, scale, rank, dtype)
    want, wl, mag, smag = ref.decode(q_lat, q_pe, lat, key, table, lens, n_q, page, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, rank + 64, max(lens), dtype)
    # a weight below the least normal number of binary16 is off by up to half a step of it, 2^-25 of the row's largest
    # weight times scale (which is at least 2^-2 of the unit), times a code of up to 448
    if scale is not None and dtype == FP:
        tol = tol + sum(lens) * 2.0 ** -23 * mag.amax(-1, keepdim=True)
    ref.close(out, want, tol, "out")
    ref.close(lse, wl, tl, "lse")


def test_decode_far_pages():
    """Byte offsets past 32 bits in a long cache."""
    say("decode far pages")
    g, page, rank, n = gen(2), 64, 512, 500
    n_pages = (1 << 32) // (page * 1152) + 40
    d = dims(16, rank, BF, page=page, scale=0.07)
    pages = torch.empty(n_pages, page, 576, dtype=BF, device="cuda")
    table = torch.arange(n_pages - 1, n_pages - 9, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    pages[n_pages - 8:] = randn(g, 8, page, 576, dtype=BF)
    q_lat, q_pe = randn(g, 1, 16, rank, dtype=BF), randn(g, 1, 16, 64, dtype=BF)
    ws = workspace(d, 1, 1, n)
    out, lse = torch.zeros(1, 16, rank, dtype=BF, device="cuda"), torch.zeros(1, 16, device="cuda")
    q().coli_mla_decode(d, q_lat, q_pe, pages, None, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, out,
                        lse, ws)
    ok(ws)
    near = table - (n_pages - 8)
    lat, key = ref.rows_of(pages[n_pages - 8:], None, rank, BF)
    want, wl, mag, smag = ref.decode(q_lat, q_pe, lat, key, near, [n], 1, page, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, 576, n, BF)
    ref.close(out, want, tol, "out")
    ref.close(lse, wl, tl, "lse")
    # expand out of the same far pages
    kv, k_pe = torch.zeros(n, 16, 256, dtype=BF, device="cuda"), torch.zeros(n, 64, dtype=BF, device="cuda")
    w = randn(g, 16, 256, rank, dtype=BF)
    q().coli_mla_expand(d, pages, None, table, ref.cumulative([n], "cuda"), w, kv, k_pe, ws)
    ok(ws)
    at = ref.slots_of(near, 0, n, page)
    want = (lat[at] @ w.double().flatten(0, 1).t()).view(n, 16, 256)
    mag = (lat[at].abs() @ w.double().abs().flatten(0, 1).t()).view(n, 16, 256)
    ref.close(kv, want, 1.01 * ref.U[BF] * want.abs() + rank * ref.U32 * mag, "kv")
    assert torch.equal(k_pe.double(), key[at])


def test_decode_without_lse_and_repeated():
    """The same bits on a second call and on a stream of its own; no lse asked for."""
    say("decode repeated")
    lens = [3000, 64, 0, 700]
    a, _ = run_decode(gen(6), lens, 1, 32, 512, BF, False, 64, with_lse=False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b, _ = run_decode(gen(6), lens, 1, 32, 512, BF, False, 64)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)
    run_decode(gen(6), lens, 1, 32, 512, BF, False, 64, max_kv=3008)   # a bound that no sequence reaches


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_reports_bad_pages_and_lengths(fp8):
    """Kernels check page ids and lengths themselves and stay inside the cache."""
    say("decode bad pages", fp8)
    g = gen(1)
    d = dims(5, 256, BF, fp8, 16)
    m = q()
    ws = workspace(d, 2, 1, 40)
    q_lat, q_pe = randn(g, 2, 5, 256, dtype=BF), randn(g, 2, 5, 64, dtype=BF)
    out, lse = torch.zeros_like(q_lat), torch.zeros(2, 5, device="cuda")
    for change in ("page", "negative page", "length", "negative length", "none"):
        pages, scale, table = cache(g, [40, 33], 256, BF, fp8, 16)
        kv_lens = torch.tensor([40, 33], dtype=torch.int32, device="cuda")
        if change == "page":
            table[1, 2] = pages.shape[0]
        elif change == "negative page":
            table[0, 1] = -1
        elif change == "length":
            kv_lens[0] = 41
        elif change == "negative length":
            kv_lens[1] = -3
        m.coli_mla_decode(d, q_lat, q_pe, pages, scale, table, kv_lens, 40, out, lse, ws)
        if change == "none":
            ok(ws)
        else:
            assert status(ws) == m.COLI_EINVAL and "page" in m.coli_moe_last_error(), change


# ---------------------------------------------------------------- expand
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rank,fp8", [(512, False), (512, True), (256, False), (256, True)])
@pytest.mark.parametrize("lens,heads,page,nope", [([1], 1, 1, 128), ([0, 3, 0, 70, 1], 5, 16, 192), ([333, 1, 0, 700], 3, 48, 192),
                                                  ([130], 32, 64, 128), ([257, 255], 1, 128, 192), ([2000, 48], 16, 64, 192)])
def test_expand(dtype, rank, fp8, lens, heads, page, nope):
    say("expand", dtype, rank, fp8, lens, heads, page, nope)
    g = gen(sum(lens) + heads)
    v = 128 if nope == 128 else 256
    pages, scale, table = cache(g, lens, rank, dtype, fp8, page)
    d = dims(heads, rank, dtype, fp8, page, nope=nope, v=v)
    w = (randn(g, heads, nope + v, rank) / math.sqrt(rank)).to(dtype)
    n = sum(lens)
    kv = torch.full((n + 2, heads, nope + v), 7.0, dtype=dtype, device="cuda")
    k_pe = torch.full((n + 2, 64), 7.0, dtype=dtype, device="cuda")
    ws = workspace(d)
    q().coli_mla_expand(d, pages, scale, table, ref.cumulative(lens, "cuda"), w, kv, k_pe, ws)
    ok(ws)
    lat, key = ref.rows_of(pages, scale, rank, dtype)
    at = torch.cat([ref.slots_of(table, b, m, page) for b, m in enumerate(lens)])
    wf = w.double().flatten(0, 1).t()
    want, mag = (lat[at] @ wf).view(n, heads, -1), (lat[at].abs() @ wf.abs()).view(n, heads, -1)
    ref.close(kv[:n], want, 1.01 * ref.U[dtype] * want.abs() + (rank + 4) * ref.U32 * mag + ref.TINY[dtype], "kv")
    assert torch.equal(k_pe[:n].double(), key[at])
    assert (kv[n:] == 7).all() and (k_pe[n:] == 7).all(), "written behind the last row"


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rank,fp8", [(512, False), (512, True), (256, False), (256, True)])
@pytest.mark.parametrize("lens,heads,page,nope", [([333, 1, 0, 700], 37, 48, 192), ([129, 62], 64, 16, 128), ([300], 64, 64, 192),
                                                  ([2000, 49, 0], 33, 1, 128), ([95, 2], 128, 64, 128)])
def test_expand_of_many_heads(dtype, rank, fp8, lens, heads, page, nope):
    """Products of more tiles than run at once."""
    test_expand(dtype, rank, fp8, lens, heads, page, nope)


@pytest.mark.parametrize("fp8", [False, True])
def test_expand_and_prefill_of_many_sequences(fp8):
    """A hundred sequences, every third of them empty."""
    say("expand many", fp8)
    g = gen(6)
    lens = [0 if i % 3 == 1 else 1 + 7 * i % 23 for i in range(100)]
    heads, rank, page, n = 3, 256, 16, sum(lens)
    pages, scale, table = cache(g, lens, rank, BF, fp8, page)
    d = dims(heads, rank, BF, fp8, page)
    w = (randn(g, heads, 256, rank) / 16).to(BF)
    kv, k_pe = torch.full((n, heads, 256), NAN, dtype=BF, device="cuda"), torch.full((n, 64), NAN, dtype=BF, device="cuda")
    ws, cu = workspace(d), ref.cumulative(lens, "cuda")
    q().coli_mla_expand(d, pages, scale, table, cu, w, kv, k_pe, ws)
    lat, key = ref.rows_of(pages, scale, rank, BF)
    at = torch.cat([ref.slots_of(table, b, m, page) for b, m in enumerate(lens)])
    wf = w.double().flatten(0, 1).t()
    want, mag = (lat[at] @ wf).view(n, heads, -1), (lat[at].abs() @ wf.abs()).view(n, heads, -1)
    ref.close(kv, want, 1.01 * ref.U[BF] * want.abs() + (rank + 4) * ref.U32 * mag, "kv")
    assert torch.equal(k_pe.double(), key[at])
    qq = randn(g, n, heads, 192, dtype=BF)
    out, lse = torch.full((n, heads, 128), NAN, dtype=BF, device="cuda"), torch.full((n, heads), NAN, device="cuda")
    q().coli_mla_prefill(d, qq, kv[..., :128], k_pe, kv[..., 128:], cu, cu, max(lens), True, out, lse, ws)
    ok(ws)
    want, wl, mag, smag = ref.prefill(qq, kv[..., :128], k_pe, kv[..., 128:], lens, lens, True, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, 192, max(lens), BF)
    ref.close(out, want, tol, "out")
    ref.close(lse, wl, tl, "lse")


def test_expand_reports_bad_pages_and_offsets():
    say("expand bad pages")
    g = gen(1)
    m = q()
    d = dims(5, 256, BF, False, 16)
    pages, _, table = cache(g, [40, 33], 256, BF, False, 16)
    w = randn(g, 5, 256, 256, dtype=BF)
    kv, k_pe = torch.zeros(80, 5, 256, dtype=BF, device="cuda"), torch.zeros(80, 64, dtype=BF, device="cuda")
    ws = workspace(d)
    table[1, 2] = 1 << 20
    m.coli_mla_expand(d, pages, None, table, ref.cumulative([40, 33], "cuda"), w, kv, k_pe, ws)
    assert status(ws) == m.COLI_EINVAL
    table[1, 2] = 0
    m.coli_mla_expand(d, pages, None, table, ref.cumulative([49, 20], "cuda"), w, kv, k_pe, ws)   # behind the table
    assert status(ws) == m.COLI_EINVAL


@pytest.mark.parametrize("lens,tail", [([30, 20], 0), ([3] * 150, 7)])
def test_expand_reports_offsets_that_do_not_fit(lens, tail):
    """Offsets that begin behind or before 0, descend anywhere, or end behind the rows."""
    say("expand bad offsets", len(lens), tail)
    g, m, batch = gen(1), q(), len(lens)
    d = dims(2, 256, BF, False, 16)
    pages, _, table = cache(g, [64] * batch, 256, BF, False, 16)
    w = randn(g, 2, 256, 256, dtype=BF)
    rows = sum(lens) + tail
    kv, k_pe = torch.zeros(rows, 2, 256, dtype=BF, device="cuda"), torch.zeros(rows, 64, dtype=BF, device="cuda")
    ws, good = workspace(d), ref.cumulative(lens, "cuda")
    for what in ("good", "first", "before", "middle", "last descends", "last", "negative", "good"):
        cu = good.clone()
        if what == "first":
            cu[0] = 1
        elif what == "before":
            cu[0] = -3
        elif what == "middle":
            cu[batch // 2] = cu[batch] + 1
        elif what == "last descends":
            cu[batch] = cu[batch - 1] - 1
        elif what == "last":
            cu[batch] = rows + 1
        elif what == "negative":
            cu[batch] = -1
        m.coli_mla_expand(d, pages, None, table, cu, w, kv, k_pe, ws)
        if what == "good":
            ok(ws)
        else:
            assert status(ws) == m.COLI_EINVAL and "offset" in m.coli_moe_last_error(), what


# ---------------------------------------------------------------- prefill
def run_prefill(g, q_lens, k_lens, heads, nope, dtype, causal, spread=1.0, poison=None, packed=True):
    v_dim = 128 if nope == 128 else 256
    d = dims(heads, 512, dtype, nope=nope, v=v_dim)
    n, m = sum(q_lens), sum(k_lens)
    qq = (spread * randn(g, n, heads, nope + 64)).to(dtype)
    kv = randn(g, m, heads, nope + v_dim, dtype=dtype)
    k_pe = randn(g, m, 64, dtype=dtype)
    if not packed:   # strides of their own: heads outermost, an odd token stride
        qq = torch.empty(heads, n, nope + 72, dtype=dtype, device="cuda").copy_(torch.nn.functional.pad(qq, (0, 8)).transpose(0, 1))[..., :nope + 64].transpose(0, 1)
        kv = torch.empty(heads, m, nope + v_dim + 8, dtype=dtype, device="cuda").copy_(torch.nn.functional.pad(kv, (0, 8)).transpose(0, 1))[..., :nope + v_dim].transpose(0, 1)
    k_nope, v = kv[..., :nope], kv[..., nope:]
    if poison:
        poison(k_nope, k_pe, v)
    cu_q, cu_k = ref.cumulative(q_lens, "cuda"), ref.cumulative(k_lens, "cuda")
    out = torch.full((n + 1, heads, v_dim), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((n, heads), NAN, device="cuda")
    ws = workspace(d)
    q().coli_mla_prefill(d, qq, k_nope, k_pe, v, cu_q, cu_k, max(q_lens), causal, out[:n], lse, ws)
    ok(ws)
    want, wl, mag, smag = ref.prefill(qq, k_nope, k_pe, v, q_lens, k_lens, causal, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, nope + 64, max(k_lens + [1]), dtype)
    ref.close(out[:n], want, tol, "out")
    ref.close(lse, wl, tl, "lse")
    assert (out[n] == 7).all(), "written behind the last query"
    return out[:n], lse


PREFILL = [  # q_lens, k_lens, heads
    ([1], [1], 1), ([2, 0, 5], [2, 0, 5], 5), ([1, 77, 300], [1, 200, 300], 3), ([64, 65, 63], [64, 65, 63], 2),
    ([33], [1000], 5), ([130, 5], [129, 0], 3), ([513, 1, 128], [513, 700, 131], 1), ([700], [64], 2),
    ([300, 77], [300, 200], 128)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("nope", [128, 192])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,k_lens,heads", PREFILL)
def test_prefill(dtype, nope, causal, q_lens, k_lens, heads):
    say("prefill", dtype, nope, causal, q_lens, k_lens, heads)
    run_prefill(gen(sum(q_lens)), q_lens, k_lens, heads, nope, dtype, causal)


@pytest.mark.parametrize("nope", [128, 192])
def test_prefill_strides_and_peaked_scores(nope):
    say("prefill strides", nope)
    run_prefill(gen(1), [70, 130], [70, 150], 3, nope, BF, True, packed=False)
    run_prefill(gen(2), [700], [900], 2, nope, FP, True, spread=12.0)


@pytest.mark.parametrize("nope,heads", [(128, 2), (192, 2), (128, 256), (192, 256)])
def test_prefill_masked_keys_may_hold_anything(nope, heads):
    """Keys and values that a query does not see are NaN or infinite: inside its own tile and behind it."""
    n = 200
    for value in (NAN, float("inf"), -float("inf")):
        for at in (199, 130, 70):
            say("prefill poisoned", nope, heads, value, at)

            def poison(k_nope, k_pe, v):
                k_nope[at] = value
                v[at] = value
            out, lse = run_prefill(gen(at), [n], [n], heads, nope, BF, True, poison=poison)
            assert out[:at].isfinite().all() and lse[:at].isfinite().all()


@pytest.mark.parametrize("nope,heads", [(128, 2), (192, 2), (128, 256), (192, 256)])
def test_prefill_keeps_a_seen_nan_visible(nope, heads):
    """A value that is not finite reaches exactly the queries that see it, and its own column only."""
    def poison(k_nope, k_pe, v):
        v[70, 0, 5] = NAN
        v[90, 1, 7] = float("inf")
    say("prefill seen nan", nope)
    out, _ = run_prefill(gen(5), [200], [200], heads, nope, FP, True, poison=poison)
    assert out[70:, 0, 5].isnan().all() and out[90:, 1, 7].isinf().all()


@pytest.mark.parametrize("nope,heads", [(128, 2), (192, 2), (128, 256), (192, 256)])
@pytest.mark.parametrize("q_len,causal", [(1, True), (200, False), (1, False)])
@pytest.mark.parametrize("k_len", [200, 33])
def test_prefill_last_value_infinite(nope, heads, q_len, causal, k_len):
    """The last value of a tile that is not full is infinite, and every query sees it: the places behind it hold nothing."""
    say("prefill last value", nope, heads, q_len, causal, k_len)

    def poison(k_nope, k_pe, v):
        v[-1, 0, 5] = float("inf")
        v[-1, 1, 7] = -float("inf")
        v[-2, 1, 9] = NAN
    out, _ = run_prefill(gen(6), [q_len], [k_len], heads, nope, BF, causal, poison=poison)
    assert (out[:, 0, 5] == math.inf).all() and (out[:, 1, 7] == -math.inf).all()


def test_prefill_of_thousands_of_sequences():
    """One prompt of 4096 tokens among 4095 of one token each, 128 heads: more blocks by the longest prompt than one launch
    takes.  A token that sees itself alone gets its value."""
    say("prefill thousands")
    g, heads, at, long = gen(40), 128, 2500, 4096
    lens = [1] * 4096
    lens[at] = long
    n = sum(lens)
    d = dims(heads)
    qq, kv, k_pe = randn(g, n, heads, 192, dtype=BF), randn(g, n, heads, 256, dtype=BF), randn(g, n, 64, dtype=BF)
    out, lse = torch.full((n, heads, 128), NAN, dtype=BF, device="cuda"), torch.full((n, heads), NAN, device="cuda")
    cu, ws = ref.cumulative(lens, "cuda"), workspace(d)
    q().coli_mla_prefill(d, qq, kv[..., :128], k_pe, kv[..., 128:], cu, cu, long, True, out, lse, ws)
    ok(ws)
    one = torch.ones(n, dtype=torch.bool, device="cuda")
    one[at:at + long] = False
    assert torch.equal(out[one], kv[one][..., 128:])
    some, span = [0, 63, 127], slice(at, at + long)
    args = qq[span][:, some], kv[span][:, some, :128], k_pe[span], kv[span][:, some, 128:]
    want, wl, mag, smag = ref.prefill(*args, [long], [long], True, d.softmax_scale)
    tol, tl = ref.attend_tol(want, mag, smag, 192, long, BF)
    ref.close(out[span][:, some], want, tol, "out")
    ref.close(lse[span][:, some], wl, tl, "lse")


def test_prefill_reports_bad_offsets():
    say("prefill bad offsets")
    m = q()
    d = dims(2)
    qq, kv, k_pe = (torch.zeros(10, 2, 192, dtype=BF, device="cuda"), torch.zeros(10, 2, 256, dtype=BF, device="cuda"),
                    torch.zeros(10, 64, dtype=BF, device="cuda"))
    out, lse = torch.zeros(10, 2, 128, dtype=BF, device="cuda"), torch.zeros(10, 2, device="cuda")
    ws = workspace(d)
    for cu_q, cu_k, top in (([0, 11], [0, 10], 11), ([0, 10], [0, 11], 10), ([0, 10], [5, 3], 10), ([0, 10], [0, 10], 9),
                            ([-1, 4], [0, 10], 10)):
        m.coli_mla_prefill(d, qq, kv[..., :128], k_pe, kv[..., 128:], torch.tensor(cu_q, dtype=torch.int32, device="cuda"),
                           torch.tensor(cu_k, dtype=torch.int32, device="cuda"), top, True, out, lse, ws)
        assert status(ws) == m.COLI_EINVAL, (cu_q, cu_k, top)


def _lift_tol(tol, keys, v):
    """Weights of binary16 below its normal numbers are off by half a step, 2^-25, where the row's largest is at least
    2^5 (2^7, less a scale's fraction and the rounding of the reference): `keys` of them, on values of up to v."""
    return tol + keys * 2.0 ** -30 * v


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,n_q", [(64, 1), (256, 64)])
def test_decode_many_small_weights(fp8, heads, n_q):
    """binary16: one key takes nearly all, 60000 others 2^-25.5 of its weight each, which together are seen: shared out
    over the GPU, and so many rows that a workgroup goes through all tokens."""
    say("decode small weights", fp8, heads, n_q)
    n, page, rank = 60000, 64, 256
    pages = torch.zeros(n // page + 2, page, rank + 128 if fp8 else rank + 64, dtype=torch.uint8 if fp8 else FP, device="cuda")
    flat = pages.view(-1, pages.shape[-1])
    scale = torch.ones(flat.shape[0], device="cuda") if fp8 else None
    flat[:, 5] = 0x38 if fp8 else 1.0   # one
    flat[777, 5] = 0
    flat[777, rank:].view(FP)[:] = 25.5 * math.log(2) / (64 * 192 ** -0.5)
    table = torch.arange(pages.shape[0], dtype=torch.int32, device="cuda")[None].contiguous()
    q_lat, q_pe = torch.zeros(n_q, heads, rank, dtype=FP, device="cuda"), torch.ones(n_q, heads, 64, dtype=FP, device="cuda")
    d = dims(heads, rank, FP, fp8, page, scale=192 ** -0.5)
    ws = workspace(d, 1, n_q, n)
    out, lse = torch.full((n_q, heads, rank), NAN, dtype=FP, device="cuda"), torch.full((n_q, heads), NAN, device="cuda")
    q().coli_mla_decode(d, q_lat, q_pe, pages, scale, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, out, lse, ws)
    ok(ws)
    lat, key = ref.rows_of(pages, scale, rank, FP)
    want, wl, mag, smag = ref.decode(q_lat, q_pe, lat, key, table, [n], n_q, page, d.softmax_scale)
    assert 1e-3 < float(want[0, 0, 5]) < 2e-3
    tol, tl = ref.attend_tol(want, mag, smag, rank + 64, n, FP)
    ref.close(out, want, _lift_tol(tol, n, 1.0), "out")
    ref.close(lse, wl, tl, "lse")


@pytest.mark.parametrize("nope", [128, 192])
@pytest.mark.parametrize("heads", [2, 256])
def test_prefill_many_small_weights(nope, heads):
    """The same of prefill."""
    say("prefill small weights", nope, heads)
    n, v_dim = 60000 if heads == 2 else 20000, 128 if nope == 128 else 256
    d = dims(heads, 512, FP, nope=nope, v=v_dim)
    kv = torch.zeros(n, 1, nope + v_dim, dtype=FP, device="cuda")
    kv[:, :, nope + 5] = 1.0
    kv[777, :, nope + 5] = 0.0
    kv = kv.expand(n, heads, nope + v_dim)   # every head reads the same keys and values
    k_pe = torch.zeros(n, 64, dtype=FP, device="cuda")
    k_pe[777] = 25.5 * math.log(2) / (64 * d.softmax_scale)
    qq = torch.ones(1, heads, nope + 64, dtype=FP, device="cuda")
    cu_q, cu_k = ref.cumulative([1], "cuda"), ref.cumulative([n], "cuda")
    out, lse = torch.full((1, heads, v_dim), NAN, dtype=FP, device="cuda"), torch.full((1, heads), NAN, device="cuda")
    ws = workspace(d)
    q().coli_mla_prefill(d, qq, kv[..., :nope], k_pe, kv[..., nope:], cu_q, cu_k, 1, True, out, lse, ws)
    ok(ws)
    want, wl, mag, smag = ref.prefill(qq, kv[..., :nope], k_pe, kv[..., nope:], [1], [n], True, d.softmax_scale)
    assert 4e-4 < float(want[0, 0, 5]) < 2e-3
    tol, tl = ref.attend_tol(want, mag, smag, nope + 64, n, FP)
    ref.close(out, want, _lift_tol(tol, n, 1.0), "out")
    ref.close(lse, wl, tl, "lse")


# ---------------------------------------------------------------- together
def test_calls_run_on_the_current_stream_or_the_given_one():
    """Inputs that a stream writes late are seen by a call on that stream."""
    say("streams")
    g = gen(31)
    real, w = randn(g, 9, 4, 128, dtype=BF), randn(g, 4, 64, 128, dtype=BF)
    want = torch.empty(9, 4, 64, dtype=BF, device="cuda")
    q().coli_mla_project(real, w, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for given in (False, True):
        x, out = torch.zeros_like(real), torch.zeros_like(want)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            x.copy_(real)
            if not given:
                q().coli_mla_project(x, w, out)
        if given:
            q().coli_mla_project(x, w, out, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want), given


@pytest.mark.parametrize("fp8", [False, True])
def test_absorbed_form_is_the_expanded_form(fp8):
    """A prompt's last queries through project, decode, project equal the expanded form's: one cache, two ways."""
    say("forms", fp8)
    g, m = gen(12), q()
    n, heads, rank, nope, v = 150, 5, 512, 128, 128
    d = dims(heads, rank, FP, fp8, 16)
    pages, scale, table = cache(g, [n], rank, FP, fp8, 16)
    w = (randn(g, heads, nope + v, rank) / math.sqrt(rank)).to(FP)
    wk, wv = w[:, :nope].transpose(1, 2).contiguous(), w[:, nope:].contiguous()
    whole = randn(g, 3, heads, nope + 64, dtype=FP)
    ws = workspace(d, 1, 3, n)
    kv, k_pe = torch.empty(n, heads, nope + v, dtype=FP, device="cuda"), torch.empty(n, 64, dtype=FP, device="cuda")
    m.coli_mla_expand(d, pages, scale, table, ref.cumulative([n], "cuda"), w, kv, k_pe, ws)
    a, b = torch.empty(3, heads, v, dtype=FP, device="cuda"), torch.empty(3, heads, v, dtype=FP, device="cuda")
    la, lb = torch.empty(3, heads, device="cuda"), torch.empty(3, heads, device="cuda")
    m.coli_mla_prefill(d, whole, kv[..., :nope], k_pe, kv[..., nope:], ref.cumulative([3], "cuda"),
                       ref.cumulative([n], "cuda"), 3, True, a, la, ws)
    q_lat, o_lat = torch.empty(3, heads, rank, dtype=FP, device="cuda"), torch.empty(3, heads, rank, dtype=FP, device="cuda")
    m.coli_mla_project(whole[..., :nope], wk, q_lat)
    m.coli_mla_decode(d, q_lat, whole[..., nope:].contiguous(), pages, scale, table,
                      torch.tensor([n], dtype=torch.int32, device="cuda"), n, o_lat, lb, ws)
    m.coli_mla_project(o_lat, wv, b)
    ok(ws)
    # roundings on the way (u = 2^-11 each): keys, values, q_lat, weights twice, o_lat and both outputs; scores of
    # size S carry 2 u S into the weights.  Values and outputs are of size about one.
    s = float(la.abs().max()) + 1
    assert (la - lb).abs().max() <= 4 * s * 2.0 ** -11
    assert (a.float() - b.float()).abs().max() <= 2 * (4 * s + 8) * 2.0 ** -11


def test_graph_replays():
    """All five captured into one graph; every replay has the eager bits, with eager work between."""
    say("graph")
    g, m = gen(20), q()
    heads, rank, page, n = 5, 512, 16, 700
    d = dims(heads, rank, BF, False, page)
    pages, _, table = cache(g, [n, 60], rank, BF, False, page)
    freq = torch.rand(32, device="cuda", dtype=torch.float64)
    kv_a, whole = randn(g, 2, rank + 64, dtype=BF), randn(g, 2, heads, 192, dtype=BF)
    positions = torch.tensor([n - 1, 59], dtype=torch.int32, device="cuda")
    slots = torch.stack([ref.slots_of(table, 0, n, page)[-1], ref.slots_of(table, 1, 60, page)[-1]])
    lens = torch.tensor([n, 60], dtype=torch.int32, device="cuda")
    w = (randn(g, heads, 256, rank) / math.sqrt(rank)).to(BF)
    wk = w[:, :128].transpose(1, 2).contiguous()
    ws = workspace(d, 2, 1, n)
    cu_k, cu_q = ref.cumulative([n, 60], "cuda"), ref.cumulative([1, 1], "cuda")
    bufs = {"q_pe": torch.zeros(2, heads, 64, dtype=BF, device="cuda"), "q_lat": torch.zeros(2, heads, rank, dtype=BF, device="cuda"),
            "out": torch.zeros(2, heads, rank, dtype=BF, device="cuda"), "lse": torch.zeros(2, heads, device="cuda"),
            "kv": torch.zeros(n + 60, heads, 256, dtype=BF, device="cuda"), "k_pe": torch.zeros(n + 60, 64, dtype=BF, device="cuda"),
            "full": torch.zeros(2, heads, 128, dtype=BF, device="cuda"), "l2": torch.zeros(2, heads, device="cuda")}

    def step():
        t = bufs
        m.coli_mla_append(d, kv_a, None, positions, slots, freq, whole[..., 128:], t["q_pe"], pages, None, ws)
        m.coli_mla_project(whole[..., :128], wk, t["q_lat"])
        m.coli_mla_decode(d, t["q_lat"], t["q_pe"], pages, None, table, lens, n, t["out"], t["lse"], ws)
        m.coli_mla_expand(d, pages, None, table, cu_k, w, t["kv"], t["k_pe"], ws)
        m.coli_mla_prefill(d, whole, t["kv"][..., :128], t["k_pe"], t["kv"][..., 128:], cu_q, cu_k, 1, True, t["full"], t["l2"], ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        kv_a.copy_(randn(g, 2, rank + 64, dtype=BF))
        whole.copy_(randn(g, 2, heads, 192, dtype=BF))
        step()
        want = {k: t.clone() for k, t in bufs.items()}
        for t in bufs.values():
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, t in bufs.items():
            assert torch.equal(t, want[k]), (i, k)
    ok(ws)
