"""Pins of the routing oracle, and the refusals of a4w4_moe_route (no GPU needed)."""

import numpy as np
import pytest

import mxfp4_a4w4_gemm_gb300 as a4w4
from oracle import route


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def test_by_hand():
    x = np.log([1.0, 2.0, 4.0, 2.0])
    ids, w = route.route(x, True, None, 1, 1, 1, 3, False, 9.0)
    assert ids == [2, 1, 3] and np.allclose(w, [4.0, 2.0, 2.0])            # of equals the lower first
    ids, w = route.route(x, True, None, 1, 1, 1, 2, True, 1.0)
    assert ids == [2, 1] and np.allclose(w, [2 / 3, 1 / 3])
    ids, w = route.route([0.0, 0.0, 0.0], False, [0.1, 0.3, 0.2], 1, 1, 1, 2, False, 1.0)
    assert ids == [1, 2] and np.allclose(w, 0.5)                           # the bias chooses, the score weighs


def test_groups():
    x = np.array([3.0, -9.0, 2.0, 2.0, 2.5, 1.0])
    assert route.route(x, False, None, 3, 1, 1, 1, True, 1.0)[0] == [0]
    assert route.route(x, False, None, 3, 2, 1, 2, True, 1.0)[0] == [2, 3]  # two of the middle outweigh one
    assert route.route(np.zeros(6), False, None, 3, 2, 2, 3, True, 1.0)[0] == [0, 1, 2]


def test_out_of_the_ordinary_logits():
    x = [np.nan, -np.inf, 1.0, np.inf]
    ids, w = route.route(x, True, None, 1, 1, 1, 4, True, 1.0)
    assert ids == [3, 2, 0, 1] and w.tolist() == [1.0, 0.0, 0.0, 0.0]
    ids, w = route.route([-np.inf] * 3, True, None, 1, 1, 1, 2, True, 1.0)
    assert ids == [0, 1] and w.tolist() == [0.0, 0.0]


def test_refusals_need_no_device():
    good = dict(logits=16, logits_type=0, stride=64, num_tokens=None, T=2, E=64, score=0, bias=None, groups=1, group_top=1,
                top_groups=1, topk=4, renormalise=1, scale=1.0, topk_ids=16, topk_weights=16)
    for change in (dict(logits=None), dict(logits=2), dict(logits=1, logits_type=1), dict(logits_type=2), dict(logits_type=-1),
                   dict(stride=63), dict(T=-1), dict(E=0), dict(E=2049, stride=4096), dict(score=2), dict(score=-1), dict(bias=2),
                   dict(num_tokens=2), dict(groups=0), dict(groups=3), dict(groups=64), dict(groups=33, E=66, stride=66),
                   dict(group_top=0), dict(group_top=3), dict(top_groups=0), dict(top_groups=2), dict(topk=0), dict(topk=33),
                   dict(topk=5, E=4), dict(groups=8, top_groups=1, topk=9), dict(renormalise=2), dict(scale=float("nan")),
                   dict(scale=float("inf")), dict(topk_ids=None), dict(topk_ids=2), dict(topk_weights=None), dict(topk_weights=2),
                   dict(T=1 << 30, topk=2)):
        with pytest.raises(a4w4.A4W4Error) as e:
            a4w4.a4w4_moe_route(*{**good, **change}.values(), stream=0)
        assert e.value.code == a4w4.A4W4_ERR_ARG, change


def test_logits_must_have_the_given_stride():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        a4w4.a4w4_moe_route(x, 0, 32, None, 4, 32, 0, None, 1, 1, 1, 2, 1, 1.0, 16, 16, stream=0)
    with pytest.raises(ValueError):
        a4w4.a4w4_moe_route(x.T, 0, 4, None, 64, 4, 0, None, 1, 1, 1, 2, 1, 1.0, 16, 16, stream=0)
