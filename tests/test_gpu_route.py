"""GPU parity of the routing to experts against the oracle, at the logits and biases where it can go wrong."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
import workloads
from oracle import mxfp4, route

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


class Router:
    def __init__(self, x, softmax=False, bias=None, groups=1, group_top=1, top_groups=1, topk=4, renorm=True, scale=2.5, bf16=False,
                 stride=None, shift=0):
        """x float32 [T, E]; rows `stride` apart, the first `shift` elements behind an aligned address."""
        x = np.asarray(x, dtype=np.float32)
        self.T, self.E = x.shape
        self.x = mxfp4.bf16_bits_to_f64(workloads.to_bf16_bits(x)).reshape(x.shape) if bf16 else x.astype(np.float64)
        self.bias = None if bias is None else np.asarray(bias, dtype=np.float32)
        self.softmax, self.groups, self.group_top, self.top_groups = softmax, groups, group_top, top_groups
        self.topk, self.renorm, self.scale, self.bf16 = topk, renorm, scale, bf16
        self.stride = stride or self.E
        flat = torch.full((self.T * self.stride + shift + 64,), float("nan"), dtype=torch.bfloat16 if bf16 else torch.float32)
        self.rows = flat.cuda()[shift:][: self.T * self.stride].view(self.T, self.stride)[:, : self.E]
        self.rows.copy_(torch.from_numpy(x).to(flat.dtype))
        self.dev_bias = None if bias is None else torch.from_numpy(self.bias).cuda()
        self.ids = torch.full((self.T, topk), -9, dtype=torch.int32, device="cuda")
        self.w = torch.full((self.T, topk), -9.0, dtype=torch.float32, device="cuda")
        self.count = None

    def run(self, stream=None):
        a4w4.a4w4_moe_route(self.rows, a4w4.A4W4_BF16 if self.bf16 else a4w4.A4W4_F32, self.stride, self.count, self.T, self.E,
                            a4w4.A4W4_MOE_SCORE_SOFTMAX if self.softmax else a4w4.A4W4_MOE_SCORE_SIGMOID, self.dev_bias, self.groups,
                            self.group_top, self.top_groups, self.topk, int(self.renorm), self.scale, self.ids, self.w, stream)

    def check(self, live=None):
        assert a4w4.a4w4_get_device_status() == 0
        ids, w = self.ids.cpu().numpy(), self.w.cpu().numpy().astype(np.float64)
        live = self.T if live is None else live
        for t in range(self.T):
            if t >= live:
                assert np.all(ids[t] == -1) and np.all(w[t] == 0.0)
                continue
            want, weights = route.route(self.x[t], self.softmax, self.bias, self.groups, self.group_top, self.top_groups, self.topk,
                                        self.renorm, self.scale)
            assert ids[t].tolist() == want, (t, ids[t].tolist(), want)
            # fp32: scores to 2^-21.7, their sum's five additions, the division and the scale; a softmax's exponents are
            # rounded to 2^-24 of themselves, twice, and the sum over a whole row has 23 additions
            x, _ = route.scores(self.x[t], self.softmax)
            far = np.where(np.isfinite(x), x, 0.0)
            reach = np.minimum(np.abs(far.max() - far[want]), 200.0) if self.softmax else np.zeros(self.topk)
            tol = 2.0 ** -20 + 2.0 ** -23 * reach.max() + (2.0 ** -18.5 if self.softmax and not self.renorm else 0.0)
            assert np.all(np.abs(w[t] - weights) <= tol * np.abs(weights) + 2.0 ** -126), (t, w[t], weights)

    def go(self, live=None):
        self.run()
        self.check(live)
        return self


def logits(T, E, seed=0, spread=1.5):
    rng = np.random.default_rng(seed + T + E)
    return rng.standard_normal((T, E)) * spread + 0.5 * rng.standard_normal(E)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E,topk", [(1, 1), (2, 2), (5, 5), (32, 8), (33, 32), (63, 1), (64, 6), (128, 8), (129, 4), (256, 8),
                                    (257, 31), (384, 6), (511, 16), (896, 16), (1000, 32), (1025, 10), (2048, 32)])
def test_plain_routing(E, topk, bf16):
    rng = np.random.default_rng(E)
    for i, (softmax, renorm) in enumerate(((True, True), (False, True), (True, False), (False, False))):
        Router(logits(9, E, i), softmax, None, topk=topk, renorm=renorm, bf16=bf16).go()
        Router(logits(9, E, i + 4), softmax, 0.05 * rng.standard_normal(E), topk=topk, renorm=renorm, bf16=bf16).go()


@pytest.mark.parametrize("E,groups,top_groups,topk", [(4, 2, 1, 2), (64, 8, 3, 8), (256, 8, 4, 8), (96, 32, 5, 15), (640, 5, 2, 32),
                                                      (896, 16, 8, 16), (2048, 32, 31, 32), (66, 3, 3, 7), (130, 13, 1, 10)])
def test_groups(E, groups, top_groups, topk):
    rng = np.random.default_rng(E)
    for softmax in (True, False):
        for group_top in (1, 2):
            for bias in (None, 0.05 * rng.standard_normal(E)):
                for bf16 in (False, True):                          # (BF16: groups of equal strength)
                    Router(logits(7, E, group_top), softmax, bias, groups, group_top, top_groups, topk, bf16=bf16).go()


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 131, 1500])
def test_tokens(T):
    Router(logits(T, 64), False, np.linspace(-0.1, 0.1, 64), topk=6).go()


@pytest.mark.parametrize("bf16", [False, True])
def test_strides_and_alignment(bf16):
    for E, stride, shift in ((64, 64, 1), (64, 65, 0), (64, 68, 0), (64, 72, 2), (62, 64, 0), (896, 1000, 4), (7, 8, 3)):
        Router(logits(6, E), True, 0.01 * np.arange(E), topk=4, bf16=bf16, stride=stride, shift=shift).go()


def test_bias_at_any_alignment():
    r = Router(logits(5, 64), False, np.linspace(0.2, -0.2, 64), topk=8)
    r.dev_bias = torch.cat([torch.zeros(3, device="cuda"), r.dev_bias])[3:]
    r.go()


def test_rows_of_padding():
    for live in (-5, 0, 1, 4, 10, 11, 1000):
        r = Router(logits(11, 100), True, topk=8)
        r.rows[max(live, 0):].fill_(float("nan"))
        r.count = torch.tensor([live], dtype=torch.int32, device="cuda")
        r.go(min(max(live, 0), 11))


def test_scores_that_tie_go_to_the_lower_index():
    rng = np.random.default_rng(1)
    x = rng.integers(-2, 3, (40, 300)).astype(np.float64)
    for softmax in (True, False):
        for bias in (None, np.zeros(300), rng.integers(0, 3, 300) / 8.0):
            Router(x, softmax, bias, topk=20).go()
    x = np.zeros((6, 896))
    x[1, 500], x[2, ::2], x[3] = 1.0, -1.0, -0.0
    x[4, 100:] = -0.0
    for softmax in (True, False):
        for bias in (None, np.zeros(896)):
            Router(x, softmax, bias, topk=16).go()


def test_scores_that_nearly_tie_are_ordered_as_the_exact_ones():
    rng = np.random.default_rng(2)
    for softmax in (False, True):
        for E in (64, 300, 896):
            x = rng.standard_normal((12, E)).astype(np.float32).astype(np.float64)
            # the bias brings every expert of row 0 to the same sum, to the last bit that fp32 has
            s = route.scores(x[0], softmax)[1]
            bias = (0.75 - s).astype(np.float32)
            x[1:4] = x[0]
            x[1, : E // 2] += 1e-6
            r = Router(x, softmax, bias, topk=8)
            c = np.sort((s + bias.astype(np.float64)))[::-1]
            assert np.median(-np.diff(c)) < 1e-9                    # nearer than fp32 can tell
            r.go()
            # the same between a few candidates and between groups
            few = np.where(np.arange(E) % 7 == 0, bias, -1.0)
            Router(x, softmax, few, topk=8).go()
            Router(x, softmax, bias, E // 20 if E % (E // 20) == 0 and E // 20 <= 32 else 4, 2, 2, 8).go()


def test_out_of_the_ordinary_logits_and_biases():
    inf, nan = np.inf, np.nan
    x = logits(12, 70, 3)
    x[0], x[1], x[2] = -inf, nan, inf
    x[3, ::3], x[4, 1::2], x[5, 7] = inf, -inf, nan
    x[6], x[7], x[8] = 1e30 * x[6], -200.0 + x[7], 60.0 + x[8]
    x[9, 3:] = -inf
    x[10] = 3.0e38
    x[11] = -120.0 + 0.1 * x[11]
    bias = 0.1 * np.random.default_rng(0).standard_normal(70)
    bias[5], bias[6], bias[7], bias[8] = nan, inf, -inf, 3e38
    for softmax in (True, False):
        for renorm in (True, False):
            Router(x, softmax, None, topk=9, renorm=renorm).go()
            Router(x, softmax, bias, topk=9, renorm=renorm).go()
            Router(x, softmax, np.full(70, 1e4), topk=9, renorm=renorm).go()       # scores that the bias swallows
    Router(x, True, None, 7, 2, 3, 9).go()
    Router(x, False, None, 7, 1, 3, 9).go()


def test_scores_far_below_the_bias_keep_their_weights():
    x = logits(4, 40) - 95.0                                        # sigmoid scores of 1e-41 and less
    bias = np.zeros(40)
    bias[[3, 30]] = 1.0
    Router(x, False, bias, topk=3).go()
    x[:, 0] = 0.0                                                   # a softmax whose others have run out of fp32
    Router(x, True, bias, topk=2).go()


def test_two_streams_and_a_captured_graph():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    r = Router(logits(300, 256), False, np.linspace(-0.1, 0.1, 256), 8, 2, 4, 8, bf16=True)
    s = Router(logits(300, 896, 1), True, None, topk=16)
    torch.cuda.synchronize()
    for _ in range(3):
        r.run(a)
        s.run(b)
    torch.cuda.synchronize()
    r.check()
    s.check()
    r.count = torch.tensor([300], dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=a):
        r.run()
    r.ids.fill_(-9)
    r.count.fill_(211)
    g.replay()
    g.replay()
    r.check(211)


def test_no_tokens():
    a4w4.a4w4_moe_route(None, 0, 8, None, 0, 8, 0, None, 1, 1, 1, 2, 1, 1.0, None, None)
    assert a4w4.a4w4_get_device_status() == 0
