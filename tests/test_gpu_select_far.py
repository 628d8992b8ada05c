"""Logits whose scores binary64 does not tell apart: choices are equal there, and go to the lower group and expert.  A bias
that is not given is one of zeros."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_select import dims, gen, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


def rows(E, softmax):
    """In an order that is not the experts'.  Scores a quarter of a binary64 step from where they would round the other way at
    least, so that how exp rounds its last bit does not count."""
    g = gen(E)

    def mixed(v):
        return v[torch.randperm(E, generator=g, device="cuda")]
    e = torch.arange(E, device="cuda", dtype=torch.float32)
    out = [mixed(e) * 1e-20,                          # scores of one half, or equal shares
           mixed(e) * 1e-20 - 3.0,
           mixed(torch.cat([e[:E // 2] * -1e-20, e[:E - E // 2] / 8]))]
    if softmax:
        far = mixed(-800.0 - e)                       # no share at all
        far[E // 3] = 0.0
        out += [far, mixed(torch.cat([e[:3] / 4, -900.0 - e[:E - 3]])), mixed(e / 8 + 300.0)]
    else:
        out += [mixed(e / 8 + 29.0),                  # from two steps below one to one itself
                mixed(e + 40.0), mixed(e / 8 + 10.0), mixed(-e * 3.0)]
    return torch.stack(out)


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("n", [7, 2051])
@pytest.mark.parametrize("E,K,groups,keep", [(256, 8, 1, 1), (256, 8, 8, 4), (160, 6, 8, 3), (60, 4, 5, 2), (64, 1, 1, 1), (64, 6, 32, 5),
                                             (512, 10, 16, 7)])
def test_select_scores_that_meet(softmax, top2, n, E, K, groups, keep):
    say("select far", softmax, top2, n, E, K, groups, keep)
    few = rows(E, softmax)
    at = torch.arange(n, device="cuda") * 3 % few.shape[0]
    zeros = torch.zeros(E, device="cuda")
    for norm in (False, True):
        d = dims(E, K, groups, keep, softmax, top2, norm)
        idx, w = reference(d, few, None)
        # a token whose experts have no share cannot be renormalised
        sound = np.isfinite(w).all(1)
        keep_rows = torch.from_numpy(sound).cuda()[at]
        logits = few[at][keep_rows]
        rows_at = at[keep_rows].cpu().numpy()
        for bias in (zeros, None):
            got, gw = run(d, logits, bias)
            wrong = (got != idx[rows_at]).any(1)
            assert not wrong.any(), (bias is None, sorted(set(rows_at[wrong])), got[wrong][:2], idx[rows_at][wrong][:2])
            assert (np.abs(gw - w[rows_at]) <= 2.0 ** -24 * 1.001 * np.abs(w[rows_at]) + 2.0 ** -149).all()


@pytest.mark.parametrize("top2", [False, True])
@pytest.mark.parametrize("n", [5, 2050])
@pytest.mark.parametrize("E,K,groups,keep", [(256, 8, 8, 4), (160, 6, 8, 3), (60, 4, 5, 2), (64, 6, 32, 5)])
def test_select_scores_of_zero_meet(top2, n, E, K, groups, keep):
    """Sigmoids below every number of binary64, of logits that rise with the expert: the first groups and experts, with a
    weight of zero.  Beside them tokens of which a few experts are not so low."""
    say("select zero", top2, n, E, K, groups, keep)
    e = torch.arange(E, device="cuda", dtype=torch.float32)
    few = torch.stack([e * 2 - 2400, e / 4 - 790, torch.where(e % 29 == 28, -e / 8, e - 1800), torch.where(e == E - 1, 3.0, e - 1800)])
    d = dims(E, K, groups, keep, False, top2, False)
    idx, w = reference(d, few, None)
    at = torch.arange(n, device="cuda") % 4
    rows_at = at.cpu().numpy()
    for bias in (torch.zeros(E, device="cuda"), None):
        got, gw = run(d, few[at], bias)
        wrong = (got != idx[rows_at]).any(1)
        assert not wrong.any(), (bias is None, sorted(set(rows_at[wrong])), got[wrong][:2], idx[rows_at][wrong][:2])
        assert (np.abs(gw - w[rows_at]) <= 2.0 ** -24 * 1.001 * np.abs(w[rows_at]) + 2.0 ** -149).all()
