"""The choice of experts at its edge, where candidates with the same inputs hide others that fp32 (or sums of two floats)
cannot tell from them, and the weights of experts far from the largest logit: against the oracle."""

import numpy as np
import pytest

import mxfp4_a4w4_gemm_gb300 as a4w4
from oracle import route
from test_gpu_route import Router

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def test_one_better_expert_behind_two_equal_ones():
    x = np.zeros((1, 8))
    x[0, :3] = 20.0, 20.0, 20.125                                   # 1 + exp(-x) is 1 in fp32 for all three
    for bias in (np.zeros(8), np.full(8, 0.5)):
        assert route.route(x[0], False, bias, 1, 1, 1, 1, True, 1.0)[0] == [2]
        for bf16 in (False, True):
            Router(x, False, bias, topk=1, bf16=bf16).go()
    x = np.full((1, 8), -60.0)
    x[0, 1], x[0, 3], x[0, 4], x[0, 6] = 0.0, -20.0, -20.0, -19.875  # one dominant logit, three that the bias swallows
    assert route.route(x[0], True, np.ones(8), 1, 1, 1, 2, True, 1.0)[0] == [1, 6]
    for bf16 in (False, True):
        Router(x, True, np.ones(8), topk=2, bf16=bf16).go()


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("E,topk,groups", [(8, 1, 1), (64, 5, 1), (256, 8, 8), (896, 16, 1), (300, 32, 1)])
def test_equal_experts_at_the_edge_of_the_choice(E, topk, groups, softmax):
    # topk - 1 experts that the bias lifts; then some equal ones, and a few slightly better ones anywhere among them
    rng = np.random.default_rng(E + topk)
    T = 60
    x, bias = np.full((T, E), -70.0), np.full(E, -1.0)
    order = rng.permutation(E)
    lifted, top, equal = order[: topk - 1], order[topk - 1], np.sort(order[topk: topk + 100])
    bias[lifted], bias[equal] = 1.0 + np.arange(topk - 1) / 64.0, 0.25
    bias[top] = -10.0                                               # for a softmax the dominant logit, nobody's choice
    x[:, lifted], x[:, top] = 0.0, 0.0
    for t in range(T):
        x[t, equal] = -22.0 if softmax else 21.0
        better = rng.permutation(equal)[: rng.integers(0, 3)]
        x[t, better] += 0.125 * rng.integers(1, 3, len(better))
    for bf16 in (False, True):
        Router(x, softmax, bias, groups, 2, groups, topk, bf16=bf16).go()


def test_equal_experts_before_one_that_sums_of_two_floats_cannot_tell():
    # pairs of experts whose exact score + bias lie 2^-50 to 2^-47.5 apart: the lower one is there twice, and first
    rng = np.random.default_rng(5)
    x = rng.uniform(-1.0, 3.0, 60000).astype(np.float32).astype(np.float64)
    s = 1.0 / (1.0 + np.exp(-x))
    b = (0.75 - s).astype(np.float32)
    c = s + b.astype(np.float64)
    order = np.argsort(c)
    gap = np.diff(c[order])
    at = np.nonzero((gap > 2.0 ** -50) & (gap < 2.0 ** -47.5))[0][:300]
    assert len(at) >= 100
    n = len(at)
    logits, bias = np.full((n, 3 * n), -np.inf), np.empty(3 * n, np.float32)
    for j, i in enumerate(at):
        u, v = order[i], order[i + 1]
        logits[j, 3 * j: 3 * j + 3] = x[u], x[u], x[v]
        bias[3 * j: 3 * j + 3] = b[u], b[u], b[v]
    assert all(route.route(logits[j], False, bias, 1, 1, 1, 1, True, 1.0)[0] == [3 * j + 2] for j in range(n))
    Router(logits, False, bias, topk=1).go()
    Router(logits, False, bias, topk=2).go()


@pytest.mark.parametrize("softmax,renorm", [(False, True), (True, True), (True, False), (False, False)])
def test_weights_of_experts_far_below_the_largest(softmax, renorm):
    # In 2^-24: an exponential 4 (two units in the last place) and 1 for its argument's remainder, however far the logits
    # lie apart.  Softmax: that, the same of the chosen ones' sum and its 5 additions, the quotient 4, the scale 1: 20; not
    # renormalised the row's 23 additions, its terms' 4 and rounded arguments (distances weighted by their exponentials: 4)
    # instead, 1 / sum and a product: 38.  Sigmoid below 0: 5, the denominator 3, the quotient 4, in the sum again: 34.
    rng = np.random.default_rng(7)
    x = (rng.uniform(-45.0, 40.0, (200, 48)) - (50.0 if not softmax else 0.0)).astype(np.float32)
    bias = np.full(48, -10.0, np.float32)
    bias[rng.permutation(48)[:10]] = 10.0                           # the bias chooses, so that the chosen lie far apart
    r = Router(x, softmax, bias, topk=8, renorm=renorm)
    r.run()
    assert a4w4.a4w4_get_device_status() == 0
    w = r.w.cpu().numpy().astype(np.float64)
    tol = (38 if not renorm else 20) * 2.0 ** -24 if softmax else 34 * 2.0 ** -24
    worst = 0.0
    for t in range(200):
        ids, want = route.route(r.x[t], softmax, r.bias, 1, 1, 1, 8, renorm, r.scale)
        assert r.ids[t].tolist() == ids
        assert np.all(np.abs(w[t] - want) <= tol * want + 2.0 ** -126), (t, w[t] / want - 1.0)
        worst = max(worst, np.max(np.where(want > 2.0 ** -100, np.abs(w[t] - want) / want, 0.0)))
    assert worst > 0.0
