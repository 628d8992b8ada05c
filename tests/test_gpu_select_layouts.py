"""Expert selection of many tokens, where sixteen lanes have one and four share a wavefront, against the rules in 64 bits: all
types, groups of any size, rows at odd places, tokens that are done over beside others that are not."""
import numpy as np
import pytest
import torch

from tests.gpu_util import say
from tests.test_gpu_select import BF, F32, FP, dims, gen, reference, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "no GPU visible"


def check(d, few, bias, n, lay=lambda x: x):
    """n tokens that repeat a few rows, in an order in which neighbours differ from wavefront to wavefront."""
    idx, w = reference(d, few, bias)
    at = torch.arange(n, device="cuda") * 7 % few.shape[0]
    got, gw = run(d, lay(few[at]), bias)
    at = at.cpu().numpy()
    wrong = (got != idx[at]).any(1)
    assert not wrong.any(), (int(wrong.sum()), got[wrong][:3], idx[at][wrong][:3])
    # one rounding to binary32, and a few of 64 bits before it
    assert (np.abs(gw - w[at]) <= 2.0 ** -24 * 1.001 * np.abs(w[at]) + 2.0 ** -149).all()


SHAPES = [  # experts, top_k, groups, groups kept
    (160, 6, 8, 3), (60, 4, 5, 2), (64, 6, 8, 3), (5, 2, 5, 3), (255, 9, 5, 2), (96, 8, 3, 1), (256, 8, 8, 4), (256, 8, 8, 1),
    (256, 10, 16, 2), (64, 10, 16, 16), (32, 3, 2, 1), (64, 8, 1, 1), (250, 5, 2, 1), (1, 1, 1, 1), (33, 10, 11, 7)]


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("softmax,top2,bias,norm", [(False, True, True, True), (True, False, False, False), (False, False, False, True),
                                                    (True, True, True, False), (True, True, False, True), (False, True, False, False)])
@pytest.mark.parametrize("E,K,groups,keep", SHAPES)
def test_select_sixteen_lanes(dtype, softmax, top2, bias, norm, E, K, groups, keep):
    say("select, sixteen lanes", dtype, softmax, top2, bias, norm, E, K, groups, keep)
    g = gen(E + K + groups)
    few = (1.5 * torch.randn(101, E, generator=g, device="cuda")).to(dtype)
    check(dims(E, K, groups, keep, softmax, top2, norm), few, 0.1 * torch.randn(E, generator=g, device="cuda") if bias else None, 2050)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("E,K,groups,keep", [(160, 6, 8, 3), (60, 4, 5, 2), (256, 8, 8, 4)])
def test_select_sixteen_lanes_strides(dtype, E, K, groups, keep):
    """Rows that begin at odd places, and further apart than they are long."""
    say("select, sixteen lanes, strides", dtype, E)
    few = (1.5 * torch.randn(101, E, generator=gen(E), device="cuda")).to(dtype)

    def lay(left, right):
        def at(x):
            whole = torch.full((x.shape[0], left + E + right), float("nan"), dtype=dtype, device="cuda")
            whole[:, left:left + E] = x
            return whole[:, left:left + E]
        return at
    b = 0.1 * torch.randn(E, generator=gen(1), device="cuda")
    for left, right in ((3, 0), (0, 5), (8, 8)):
        check(dims(E, K, groups, keep), few, b, 2051, lay(left, right))
        check(dims(E, K, groups, keep, True, False, False), few, None, 2051, lay(left, right))


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,K,groups,keep", [(160, 6, 8, 3), (60, 4, 5, 2), (255, 9, 5, 2), (256, 8, 8, 4), (64, 6, 8, 3), (48, 4, 1, 1)])
def test_select_sixteen_lanes_undecided(softmax, E, K, groups, keep):
    """Every third row leaves groups or experts undecided in binary32: all equal, equal pairs, groups alike, biases that bring
    choices together.  The rows between are of the ordinary kind and are to stay as they are."""
    say("select, sixteen lanes, undecided", softmax, E, K, groups, keep)
    g = gen(E)
    few = torch.randn(99, E, generator=g, device="cuda")
    e = torch.arange(E, device="cuda")
    size = E // groups
    few[0] = 0
    few[3] = (e // 2) / 64.0
    few[6] = (e % size) / 8.0                                   # groups alike
    few[9] = (e % size) / 8.0 + 2.0 ** -20 * (e // size)        # and nearly
    few[12] = torch.randint(0, 3, (E,), generator=g, device="cuda").float()
    few[15] = -1.0
    few[18] = few[17].flip(0)
    few[21] = (e % size == size - 1).float()
    score = torch.softmax(few[1].double(), 0) if softmax else torch.sigmoid(few[1].double())
    for bias in (None, torch.full((E,), 0.25, device="cuda"), (0.5 - score).float()):
        for top2 in (False, True):
            check(dims(E, K, groups, keep, softmax, top2), few, bias, 2049)
