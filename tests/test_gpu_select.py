"""Expert selection from logits on the GPU against the rules of include/coli_moe.h in 64 bits, one token at a time."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_util import q, say, status

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def dims(E, K, groups=1, keep=1, softmax=False, top2=True, norm=True, rsf=2.5):
    m = q()
    return m.make_select_dims(E, K, groups, keep, m.COLI_SCORE_SOFTMAX if softmax else m.COLI_SCORE_SIGMOID,
                              m.COLI_GROUP_TOP2 if top2 else m.COLI_GROUP_MAX, norm, rsf)


def reference(d, logits, bias):
    """Indices and weights by sorting, in numpy's 64 bits."""
    x = logits.double().cpu().numpy()
    b = np.zeros(d.n_experts) if bias is None else bias.double().cpu().numpy()
    idx, w = np.empty((len(x), d.top_k), np.int32), np.empty((len(x), d.top_k))
    size = d.n_experts // d.n_group
    for t, l in enumerate(x):
        if d.scoring == q().COLI_SCORE_SOFTMAX:
            p = np.exp(l - l.max())
            score = p / math.fsum(p)
        else:
            score = 1.0 / (1.0 + np.exp(-l))
        choice = score + b
        best = []
        for g in range(d.n_group):
            top = sorted(choice[g * size:(g + 1) * size], reverse=True)
            best.append(sum(top[:2]) if d.group_score == q().COLI_GROUP_TOP2 else top[0])
        open_ = sorted(range(d.n_group), key=lambda g: (-best[g], g))[:d.topk_group]
        ranked = sorted((e for e in range(d.n_experts) if e // size in open_), key=lambda e: (-choice[e], e))[:d.top_k]
        s = score[ranked]
        idx[t], w[t] = ranked, (s / s.sum() if d.norm_topk_prob else s) * d.routed_scaling_factor
    return idx, w


def run(d, logits, bias):
    n = logits.shape[0]
    idx = torch.full((n + 1, d.top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((n + 1, d.top_k), 7.0, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q().coli_moe_select(d, logits, bias, idx[:n], w[:n], ws)
    assert status(ws) == 0, q().coli_moe_last_error()
    assert (idx[n] == -7).all() and (w[n] == 7).all(), "written behind the last token"
    return idx[:n].cpu().numpy(), w[:n].double().cpu().numpy()


def check(d, logits, bias):
    got, gw = run(d, logits, bias)
    idx, w = reference(d, logits, bias)
    assert np.array_equal(got, idx), (got[(got != idx).any(1)][:3], idx[(got != idx).any(1)][:3])
    # one rounding to binary32, and a few of 64 bits before it
    assert (np.abs(gw - w) <= 2.0 ** -24 * 1.001 * np.abs(w) + 2.0 ** -149).all()


SHAPES = [  # experts, top_k, groups, groups kept
    (1, 1, 1, 1), (2, 2, 1, 1), (5, 3, 1, 1), (5, 5, 5, 5), (5, 2, 5, 3), (16, 4, 4, 2), (60, 4, 1, 1), (64, 6, 8, 3), (64, 32, 2, 2),
    (64, 3, 64, 5), (96, 8, 3, 1), (128, 8, 1, 1), (160, 6, 8, 3), (256, 8, 8, 4), (256, 8, 1, 1), (256, 1, 16, 1), (257, 7, 1, 1),
    (384, 8, 1, 1), (512, 10, 16, 7), (1000, 32, 8, 2), (1024, 8, 64, 64), (1024, 16, 4, 1), (255, 9, 5, 2), (320, 20, 10, 10)]


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("softmax,top2,bias,norm", [(False, True, True, True), (True, False, False, False),
                                                    (False, False, False, True), (True, True, True, True)])
@pytest.mark.parametrize("E,K,groups,keep", SHAPES)
def test_select(dtype, softmax, top2, bias, norm, E, K, groups, keep):
    say("select", dtype, softmax, top2, bias, norm, E, K, groups, keep)
    g = gen(E + K)
    for n in (1, 3, 37):
        logits = (1.5 * torch.randn(n, E, generator=g, device="cuda")).to(dtype)
        b = 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None
        check(dims(E, K, groups, keep, softmax, top2, norm), logits, b)


@pytest.mark.parametrize("E,K,groups,keep", [(256, 8, 8, 4), (160, 6, 1, 1), (1024, 16, 8, 3)])
@pytest.mark.parametrize("n", [4099, 9000])
def test_select_many_tokens(E, K, groups, keep, n):
    """So many that another layout of lanes takes them; a part of them is checked one by one, and all against a batch of
    those few."""
    say("select many", E, K, groups, keep, n)
    g = gen(n)
    d, b = dims(E, K, groups, keep), 0.1 * torch.randn(E, generator=g, device="cuda")
    few = 1.5 * torch.randn(301, E, generator=g, device="cuda")
    idx, w = reference(d, few, b)
    at = torch.arange(n, device="cuda") % 301
    got, gw = run(d, few[at], b)
    at = at.cpu().numpy()
    assert np.array_equal(got, idx[at]) and (np.abs(gw - w[at]) <= 2.0 ** -24 * 1.001 * np.abs(w[at])).all()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 4)])
@pytest.mark.parametrize("n", [3, 5000])
def test_select_equal_choices(softmax, groups, keep, n):
    """Ties go to the lower group and expert: all equal, equal pairs, few distinct values."""
    say("select ties", softmax, groups, keep, n)
    g = gen(2)
    rows = [torch.zeros(256, device="cuda"), torch.arange(256, device="cuda") // 2 / 64.0,
            torch.randint(0, 3, (256,), generator=g, device="cuda").float(), -torch.ones(256, device="cuda"),
            (torch.arange(256, device="cuda") % 32 == 31).float(), torch.full((256,), 50.0, device="cuda")]
    few = torch.stack(rows)
    at = torch.arange(n, device="cuda") % 6
    for b in (None, torch.full((256,), 0.25, device="cuda")):
        for top2 in (False, True):
            d = dims(256, 8, groups, keep, softmax, top2)
            idx, w = reference(d, few, b)
            got, gw = run(d, few[at].contiguous(), b)
            assert np.array_equal(got, idx[at.cpu().numpy()])
            assert (np.abs(gw - w[at.cpu().numpy()]) <= 2.0 ** -24 * 1.001 * np.abs(w[at.cpu().numpy()])).all()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("n", [7, 6000])
def test_select_neighbours_that_binary32_merges(softmax, n):
    """Logits one binary32 step apart, far out where their sigmoids in binary32 are one number, and biases that bring
    choices within 2^-27 of each other, between experts and between groups."""
    say("select near", softmax, n)
    g = gen(9)
    base = torch.tensor([14.0, 12.0, 3.0, 0.25, -2.0, -9.0], device="cuda")
    step = torch.randperm(256, generator=g, device="cuda").to(torch.int32)
    few = torch.stack([(torch.full((256,), float(v), device="cuda").view(torch.int32) + step).view(torch.float32) for v in base])
    at = torch.arange(n, device="cuda") % 6
    for groups, keep in ((1, 1), (8, 4), (32, 5)):
        for top2 in (False, True):
            d = dims(256, 8, groups, keep, softmax, top2)
            idx, _ = reference(d, few, None)
            assert np.array_equal(run(d, few[at].contiguous(), None)[0], idx[at.cpu().numpy()])
    # choices meet: bias = 0.5 - score up to binary32's rounding of it
    l = torch.randn(256, generator=g, device="cuda")
    score = torch.softmax(l.double(), 0) if softmax else torch.sigmoid(l.double())
    b = (0.5 - score).float()
    for groups, keep in ((1, 1), (8, 4), (32, 5)):
        d = dims(256, 8, groups, keep, softmax, True)
        idx, _ = reference(d, l[None], b)
        assert (run(d, l[None].expand(n, -1).contiguous(), b)[0] == idx).all()


def test_select_wide_logits():
    """Scores from one to below the normal numbers; a shift of all logits far from zero."""
    say("select wide")
    g = gen(5)
    x = 40 * torch.randn(50, 64, generator=g, device="cuda")
    check(dims(64, 4, softmax=True), x.clamp(-600, 600), None)
    check(dims(64, 4, softmax=True, norm=False), x + 1e6, None)
    check(dims(64, 8), x.clamp(-20, 20), 0.1 * torch.randn(64, generator=g, device="cuda"))
    check(dims(64, 8, rsf=-1.0), x.clamp(-18, 18) - 2, None)
    check(dims(64, 8, rsf=0.0, norm=False), x.clamp(-18, 18), 1e6 * torch.randn(64, generator=g, device="cuda"))


def test_select_strides():
    say("select strides")
    for dtype in (BF, F32):
        whole = torch.randn(40, 300, generator=gen(1), device="cuda").to(dtype)
        for x in (whole[:, 3:163], whole[::3, :160], whole[:1, :160].expand(9, -1)):
            check(dims(160, 6, 8, 3), x, None)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [1, 5000])
def test_select_reports_what_is_not_finite(value, n):
    """The status says so, indices are distinct and in range all the same, and other tokens keep their routing."""
    say("select nonfinite", value, n)
    m, d = q(), dims(256, 8, 8, 4)
    x, b = torch.randn(n, 256, generator=gen(7), device="cuda"), torch.zeros(256, device="cuda")
    want = run(d, x, b)[0]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    idx, w = torch.empty(n, 8, dtype=torch.int32, device="cuda"), torch.empty(n, 8, device="cuda")
    poisoned = x.clone()
    poisoned[0] = value
    for logits, bias in ((poisoned, b), (x, b.clone().fill_(value))):
        m.coli_moe_select(d, logits, bias, idx, w, ws)
        assert status(ws) == m.COLI_ENONFINITE
        got = idx.cpu().numpy()
        assert ((got >= 0) & (got < 256)).all() and all(len(set(r)) == 8 for r in got[:50])
        if bias is b:
            assert np.array_equal(got[1:], want[1:])
    # scores of zero cannot be renormalised
    m.coli_moe_select(d, torch.full_like(x, -1000.0), None, idx, w, ws)
    assert status(ws) == m.COLI_ENONFINITE


def test_select_agrees_with_route():
    """Without groups, on the logits of coli_moe_route, the same experts, and weights but for binary32's sigmoid."""
    import synth
    from synth.device import upload_layer
    from tests.gpu_util import gpu_route, workspace
    say("select against route")
    m, S = q(), 9
    layer = upload_layer(synth.tiny_layer(seed=3, S=S), device="cuda:0")
    d = m.make_dims(synth.TINY)
    idx, w = gpu_route(d, layer, workspace(d, S))
    logits = torch.empty(S, synth.TINY.n_experts, device="cuda")
    m.coli_moe_debug_logits(d, layer["x"], layer["router_w"], logits)
    got, gw = run(dims(synth.TINY.n_experts, synth.TINY.top_k, norm=bool(synth.TINY.norm_topk_prob),
                       rsf=synth.TINY.routed_scaling_factor), logits, layer["bias"])
    assert np.array_equal(got, idx.cpu().numpy())
    assert np.allclose(gw, w.cpu().numpy(), rtol=1e-5, atol=0)


def test_select_replayed():
    say("select graph")
    m, g, d = q(), gen(1), dims(160, 6, 8, 3)
    for n in (1, 4100):
        x, b = torch.randn(n, 160, generator=g, device="cuda"), 0.1 * torch.randn(160, generator=g, device="cuda")
        idx, w = torch.empty(n, 6, dtype=torch.int32, device="cuda"), torch.empty(n, 6, device="cuda")
        ws, side = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        m.coli_moe_select(d, x, b, idx, w, ws, stream=side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.coli_moe_select(d, x, b, idx, w, ws)
        for _ in range(3):
            x.copy_(torch.randn(n, 160, generator=g, device="cuda"))
            m.coli_moe_select(d, x, b, idx, w, ws)
            want = idx.clone(), w.clone()
            idx.zero_()
            w.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(idx, want[0]) and torch.equal(w, want[1])
        assert status(ws) == 0
