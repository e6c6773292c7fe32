"""GPU parity of the norms and the rotation of query and key heads, to rows and to the cache, against the oracle."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
import workloads
from gpu_util import host_bits
from oracle import kv, mxfp4, rope

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Heads:
    """A fused projection's rows [T, Hq + 2 Hkv + 1, D] (a head of padding behind them) and what goes with them."""

    def __init__(self, T, Hq, Hkv, D, rot, inter, norm="qk", far=131072, seed=0, scale=1.0):
        rng = np.random.default_rng(seed + 7 * T + Hq + D + rot)
        self.T, self.Hq, self.Hkv, self.D, self.rot, self.inter = T, Hq, Hkv, D, rot, inter
        x = rng.standard_normal((T, Hq + 2 * Hkv + 1, D)) * (1.0 + 5.0 * (rng.random((Hq + 2 * Hkv + 1, D)) < 0.05)) * scale
        self.bits = workloads.to_bf16_bits(x.astype(np.float32)).reshape(x.shape)
        self.wq = (1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32) if "q" in norm else None
        self.wk = (1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32) if "k" in norm else None
        self.freq = (500000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))).astype(np.float32)
        self.pos = rng.integers(0, far, T).astype(np.int32)
        self.load()

    def load(self):
        c = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.x = workloads.bits_to_torch(self.bits.reshape(-1)).view(self.bits.shape).cuda()
        self.dev = dict(wq=c(self.wq), wk=c(self.wk), freq=c(self.freq) if self.rot else None, pos=c(self.pos) if self.rot else None)
        self.stride = self.bits.shape[1] * self.D

    def part(self, x, which):
        at = {"q": 0, "k": self.Hq, "v": self.Hq + self.Hkv}[which]
        return x[:, at: at + (self.Hq if which == "q" else self.Hkv)]

    def want(self, which):
        x = mxfp4.bf16_bits_to_f64(self.part(self.bits, which))
        return rope.heads(x, self.wq if which == "q" else self.wk, EPS, self.pos, self.freq, self.rot, self.inter)

    def run(self, q_out, k_out, stream=None):
        d, none = self.dev, (None, 0)
        q, k = (self.part(self.x, "q"), self.stride) if self.Hq else none, (self.part(self.x, "k"), self.stride) if self.Hkv else none
        a4w4.a4w4_qk_norm_rope(*q, *k, d["pos"], self.T, self.Hq, self.Hkv, self.D, d["wq"], d["wk"], EPS, d["freq"], self.rot,
                               self.inter, q_out if self.Hq else None, q_out.stride(0) if self.Hq else 0,
                               k_out if self.Hkv else None, k_out.stride(0) if self.Hkv else 0, stream)

    def outputs(self):
        return (torch.full((self.T, self.Hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda"),
                torch.full((self.T, self.Hkv, self.D), 7.0, dtype=torch.bfloat16, device="cuda"))

    def check(self, which, out):
        assert a4w4.a4w4_get_device_status() == 0
        want, reach = self.want(which)
        got = mxfp4.bf16_bits_to_f64(host_bits(out))
        bad = ~(np.abs(got - want) <= rope.bound(want, reach))
        assert not bad.any(), (which, bad.sum(), np.argwhere(bad)[:5])


SHAPES = [
    # T, Hq, Hkv, D, rot, interleaved, norms
    (1, 1, 1, 128, 128, 0, "qk"), (1, 32, 8, 128, 128, 0, "qk"), (2, 3, 1, 128, 128, 1, ""), (3, 5, 3, 64, 64, 0, "q"),
    (7, 16, 4, 64, 32, 1, "k"), (5, 33, 7, 128, 64, 0, "qk"), (4, 6, 2, 64, 16, 0, "qk"), (9, 2, 2, 128, 48, 0, "qk"),
    (9, 7, 1, 128, 112, 1, "qk"), (333, 8, 2, 64, 48, 0, ""), (6, 4, 2, 128, 0, 0, "qk"), (6, 4, 2, 64, 0, 1, "k"),
    (3, 0, 5, 128, 128, 0, "qk"), (3, 5, 0, 64, 64, 1, "qk"), (2, 260, 68, 128, 128, 0, "qk"), (700, 300, 2, 64, 64, 0, "qk"),
    (2000, 4, 1, 128, 128, 0, "qk"), (1300, 9, 3, 64, 64, 1, "q"),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm", SHAPES, ids=lambda v: str(v))
def test_rows_match_the_oracle(T, Hq, Hkv, D, rot, inter, norm):
    h = Heads(T, Hq, Hkv, D, rot, inter, norm)
    q, k = h.outputs()
    h.run(q, k)
    for which, out in (("q", q), ("k", k)):
        if out.numel():
            h.check(which, out)


def test_in_place_and_back_in_the_projection():
    h = Heads(50, 6, 2, 128, 128, 0)
    before = h.x.clone()
    h.run(h.part(h.x, "q"), h.part(h.x, "k"))
    h.check("q", h.part(h.x, "q"))
    h.check("k", h.part(h.x, "k"))
    assert torch.equal(h.x[:, 8:].view(torch.int16), before[:, 8:].view(torch.int16))       # values and padding are left


def test_positions_at_the_ends_of_their_range():
    h = Heads(8, 4, 2, 128, 128, 0)
    h.pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 30, 123456789, -987654321], dtype=np.int32)
    h.freq[:] = np.float32(1.0) / np.arange(1, 65, dtype=np.float32)
    h.freq[5], h.freq[6], h.freq[7], h.freq[8] = 0.0, 2.0 ** -130, -0.75, 3.5
    h.load()
    q, k = h.outputs()
    h.run(q, k)
    h.check("q", q)
    h.check("k", k)


def test_squares_beyond_fp32_and_rows_of_zeros():
    h = Heads(6, 8, 4, 128, 128, 0)
    v = mxfp4.bf16_bits_to_f64(h.bits)
    v[0] *= 2.0 ** 90
    v[1, 3] *= 2.0 ** 100                                           # one head among ordinary ones
    v[2] *= 2.0 ** -100
    v[3] = 0.0
    v[4, 2] = 0.0
    h.bits = workloads.to_bf16_bits(v.astype(np.float32)).reshape(v.shape)
    h.load()
    q, k = h.outputs()
    h.run(q, k)
    h.check("q", q)
    h.check("k", k)
    assert torch.all(q[3] == 0) and torch.all(q[4, 2] == 0)


def test_what_does_not_turn_takes_nothing_from_its_neighbours():
    h = Heads(2, 2, 1, 128, 32, 0, "")
    h.bits[0, 0, 40], h.bits[1, 1, 100] = 0x7F80, 0x7FC0            # an infinity, a NaN behind the first 32 dimensions
    h.load()
    q, k = h.outputs()
    h.run(q, k)
    got, want = mxfp4.bf16_bits_to_f64(host_bits(q)), mxfp4.bf16_bits_to_f64(h.part(h.bits, "q"))
    assert np.array_equal(got[:, :, 32:], want[:, :, 32:], equal_nan=True)       # (any NaN is a NaN)


def test_no_tokens_and_no_heads():
    h = Heads(2, 2, 1, 64, 64, 0)
    q, k = h.outputs()
    a4w4.a4w4_qk_norm_rope(None, 128, None, 64, None, 0, 2, 1, 64, None, None, EPS, None, 64, 0, None, 128, None, 64)
    a4w4.a4w4_qk_norm_rope(None, 0, None, 0, h.dev["pos"], 2, 0, 0, 64, None, None, EPS, h.dev["freq"], 64, 0, None, 0, None, 0)
    assert a4w4.a4w4_get_device_status() == 0 and torch.all(q == 7.0)


# ---------------------------------------------------------------------------
# to the cache

class Cache:
    def __init__(self, h, page, slots, pages):
        self.h, self.page, self.pages = h, page, pages
        self.slots = np.asarray(slots, dtype=np.int32)
        self.bytes = a4w4.a4w4_kv_cache_bytes(pages, page, h.Hkv, h.D)
        self.cache = torch.full((self.bytes,), 0xA5, dtype=torch.uint8, device="cuda")
        self.map = i32(self.slots)
        self.q = torch.full((h.T, h.Hq, h.D), 7.0, dtype=torch.bfloat16, device="cuda")

    def run(self, stream=None):
        h, d = self.h, self.h.dev
        q = (h.part(h.x, "q"), h.stride) if h.Hq else (None, 0)
        a4w4.a4w4_kv_append_rope(*q, h.part(h.x, "k"), h.stride, h.part(h.x, "v"), h.stride, d["pos"], self.map, h.T, h.Hq, h.Hkv,
                                 h.D, d["wq"], d["wk"], EPS, d["freq"], h.rot, h.inter, self.q if h.Hq else None, h.Hq * h.D,
                                 self.cache, self.pages, self.page, stream)

    def check(self):
        assert a4w4.a4w4_get_device_status() == 0
        h = self.h
        total = self.pages * self.page
        live = (self.slots >= 0) & (self.slots < total)
        k, _ = h.want("k")
        codes, scales = [], []
        for x in (k, mxfp4.bf16_bits_to_f64(h.part(h.bits, "v"))):
            c, s = mxfp4.quantize_blocks(x.reshape(-1, h.D))
            codes.append(c.reshape(h.T, h.Hkv, h.D))
            scales.append(s.reshape(h.T, h.Hkv, h.D // 32))
        kp, ks, vp, vs = kv.byte_places(h.D)
        want = np.full((self.pages, h.Hkv, self.page // 16, 17 * h.D), 0xA5, dtype=np.uint8)
        for t in np.nonzero(live)[0]:
            s = int(self.slots[t])
            pg, ch, r = s // self.page, s % self.page // 16, s % 16
            for places, values in ((kp, mxfp4.pack_codes(codes[0][t])), (ks, scales[0][t]), (vp, mxfp4.pack_codes(codes[1][t])),
                                   (vs, scales[1][t])):
                want[pg, :, ch, places[r]] = values.T
        got = self.cache.cpu().numpy().reshape(want.shape)
        bad = got != want
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5])
        if h.Hq:
            assert torch.all(self.q[torch.from_numpy(~live).cuda()] == 7.0)      # rows without a slot are left
            wq, reach = h.want("q")
            q = mxfp4.bf16_bits_to_f64(host_bits(self.q))
            assert np.all((np.abs(q - wq) <= rope.bound(wq, reach))[live])


def scattered(T, page, seed=0, skip=()):
    rng = np.random.default_rng(seed)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T]
    for i, v in skip:
        slots[i] = v
    return slots, pages


CACHED = [
    (1, 32, 8, 128, 128, 0, "qk", 64), (2, 1, 1, 64, 64, 0, "", 16), (5, 4, 3, 128, 64, 1, "qk", 32), (40, 0, 2, 64, 32, 1, "k", 128),
    (33, 12, 5, 64, 48, 0, "qk", 16), (17, 8, 2, 128, 0, 0, "qk", 16), (17, 8, 2, 128, 0, 0, "", 16), (50, 6, 2, 128, 96, 0, "q", 64),
    (3, 300, 40, 64, 64, 0, "qk", 16), (900, 2, 1, 64, 64, 0, "qk", 32),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm,page", CACHED, ids=lambda v: str(v))
def test_cache_bytes_match_the_oracle(T, Hq, Hkv, D, rot, inter, norm, page):
    h = Heads(T, Hq, Hkv, D, rot, inter, norm)
    c = Cache(h, page, *scattered(T, page))
    c.run()
    c.check()


def test_slots_outside_the_cache_are_skipped():
    h = Heads(30, 4, 2, 128, 128, 0)
    slots, pages = scattered(30, 16)
    for i, v in ((0, -1), (7, pages * 16), (8, 2 ** 31 - 1), (29, -2 ** 31), (3, pages * 16 - 1), (4, 0)):
        slots = np.where(slots == v, -1, slots)
        slots[i] = v
    c = Cache(h, 16, slots, pages)
    c.run()
    c.check()
    empty = Cache(h, 16, np.full(30, -1), pages)
    empty.run()
    empty.check()


def test_values_near_a_border_go_where_the_exact_ones_do():
    # 2.5 million keys: of the values some 10 lie nearer to a border of E2M1 than fp32 arithmetic can tell
    h = Heads(1250, 1, 16, 128, 128, 0, far=1 << 20)
    k, reach = h.want("k")
    unit = np.exp2(np.floor(np.log2(np.abs(k).reshape(*k.shape[:2], 4, 32).max(-1))) - 2).repeat(32, -1)
    near = np.zeros(k.shape, dtype=bool)
    for border in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        near |= np.abs(np.abs(k) - border * unit) <= 2.0 ** -20 * reach
    assert near.sum() >= 3
    c = Cache(h, 64, *scattered(h.T, 64))
    c.run()
    c.check()


@pytest.mark.parametrize("D", [64, 128])
def test_scales_near_a_power_of_two(D):
    # one pair of dimensions decides the block's largest magnitude, and comes as near to 2 as BF16 pairs can, from either side
    T, half = 96, D // 2
    h = Heads(T, 1, 1, D, D, 0, "", far=100000, seed=4)
    m = np.arange(128, 256)
    v = np.zeros((T, h.bits.shape[1], D))
    ang = h.pos.astype(np.float64) * float(h.freq[0])
    gap = np.empty(T)
    for t in range(T):
        c, s = np.cos(ang[t]), np.sin(ang[t])
        best = (np.inf, 0.0, 0.0)
        for ea in (-8, -7):
            for eb in (-9, -8, -7):
                a, b = m[:, None] * 2.0 ** ea * np.sign(c), m[None] * 2.0 ** eb * -np.sign(s)
                d = np.abs(a * c - b * s - 2.0)
                i = np.unravel_index(np.argmin(d), d.shape)
                if d[i] < best[0]:
                    best = (d[i], a[i[0], 0], b[0, i[1]])
        gap[t] = best[0]
        v[t, 1, 0], v[t, 1, half] = best[1], best[2]
        v[t, 1, 1], v[t, 2, 3] = 1.0, -3.0
    assert np.median(gap) < 1e-4 and gap.min() < 2e-6
    h.bits = workloads.to_bf16_bits(v.astype(np.float32)).reshape(v.shape)
    h.load()
    c = Cache(h, 16, *scattered(T, 16))
    c.run()
    c.check()


def test_the_same_as_norm_rope_and_append_but_for_the_rounding_between():
    # without a norm and a rotation nothing is rounded on the way
    h = Heads(70, 2, 3, 64, 0, 0, "")
    c = Cache(h, 16, *scattered(70, 16))
    c.run()
    other = torch.full_like(c.cache, 0xA5)
    a4w4.a4w4_kv_append(h.part(h.x, "k"), h.stride, h.part(h.x, "v"), h.stride, c.map, 70, 3, 64, other, c.pages, 16)
    assert torch.equal(c.cache, other)


def test_two_streams_and_a_captured_graph():
    h, g = Heads(60, 8, 2, 128, 128, 0), Heads(60, 8, 2, 128, 128, 0, seed=9)
    c, d = Cache(h, 16, *scattered(60, 16)), Cache(g, 16, *scattered(60, 16, seed=1))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        c.run(stream=a)
        d.run(stream=b)
    torch.cuda.synchronize()
    c.check()
    d.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=a):
        c.run()
    h.pos[:] = h.pos[::-1]
    h.dev["pos"].copy_(torch.from_numpy(h.pos))
    c.slots[10:] = -1                                               # a step with fewer tokens
    c.map[10:] = -1
    c.cache.fill_(0xA5)
    c.q.fill_(7.0)
    graph.replay()
    graph.replay()
    c.check()


def test_the_call_after_an_expired_wait_is_right():
    # (the heads are mostly there before they are looked for: no wait, nothing to report)
    h = Heads(2000, 32, 8, 128, 128, 0)
    q, k = h.outputs()
    torch.cuda.synchronize()
    a4w4.a4w4_set_wait_limit_ns(1)
    try:
        h.run(q, k)
        status = a4w4.a4w4_get_device_status()
    finally:
        a4w4.a4w4_set_wait_limit_ns(0)
    assert status in (0, a4w4.A4W4_ERR_TIMEOUT)
    assert a4w4.a4w4_get_device_status() == 0
    h.run(q, k)
    h.check("q", q)
    h.check("k", k)


@pytest.mark.parametrize("T,Hq,Hkv,D,cached", [(2, 4094, 1, 128, False), (1, 0, 2048, 64, False), (2, 2048, 1024, 128, True), (3, 0, 2048, 64, True)])
def test_as_many_heads_as_there_may_be(T, Hq, Hkv, D, cached):
    h = Heads(T, Hq, Hkv, D, D, 0)
    if cached:
        c = Cache(h, 16, *scattered(T, 16))
        c.run()
        c.check()
        return
    q, k = h.outputs()
    h.run(q, k)
    for which, out in (("q", q), ("k", k)):
        if out.numel():
            h.check(which, out)


def test_append_with_the_queries_in_place():
    h = Heads(40, 6, 2, 128, 128, 0)
    c = Cache(h, 16, *scattered(40, 16, skip=((5, -1),)))
    before = h.x.clone()
    c.q = h.part(h.x, "q")
    d = h.dev
    a4w4.a4w4_kv_append_rope(c.q, h.stride, h.part(h.x, "k"), h.stride, h.part(h.x, "v"), h.stride, d["pos"], c.map, 40, 6, 2, 128,
                             d["wq"], d["wk"], EPS, d["freq"], 128, 0, c.q, h.stride, c.cache, c.pages, 16)
    assert torch.equal(h.x[5], before[5]) and torch.equal(h.x[:, 6:], before[:, 6:])
    c.q = c.q.clone()
    c.q[5] = 7.0
    c.check()


def test_one_slot_given_to_two_tokens():
    h = Heads(6, 1, 2, 64, 64, 0)
    slots, pages = scattered(6, 16)
    slots[4] = slots[1]
    cells = []
    for drop in (None, 1, 4):                                       # both; the one token alone; the other
        s = slots.copy()
        if drop is not None:
            s[drop] = -1
        c = Cache(h, 16, s, pages)
        c.run()
        cells.append(c.cache)
    assert torch.all((cells[0] == cells[1]) | (cells[0] == cells[2]))


def test_infinities_and_nan_in_keys_and_values():
    # as a4w4_kv_append has them where nothing is computed on the way; with a norm and a rotation they stay in their heads
    h = Heads(40, 2, 3, 128, 0, 0, "")
    rng = np.random.default_rng(3)
    for pattern in (0x7F80, 0xFF80, 0x7FC0, 0xFFC1, 0x7F7F):
        h.bits[rng.integers(0, 40, 5), rng.integers(2, 8, 5), rng.integers(0, 128, 5)] = pattern
    h.load()
    c = Cache(h, 16, *scattered(40, 16))
    c.run()
    other = torch.full_like(c.cache, 0xA5)
    a4w4.a4w4_kv_append(h.part(h.x, "k"), h.stride, h.part(h.x, "v"), h.stride, c.map, 40, 3, 128, other, c.pages, 16)
    assert torch.equal(c.cache, other)
    h = Heads(40, 2, 3, 128, 128, 0)
    c = Cache(h, 16, *scattered(40, 16))
    c.run()
    clean = c.cache.clone().view(c.pages, 3, -1)
    c.check()
    h.bits[:, 3, 17], h.bits[::2, 3, 100] = 0x7F80, 0x7FC0          # the middle one of the heads of keys
    h.load()
    c.cache.fill_(0xA5)
    c.run()
    assert a4w4.a4w4_get_device_status() == 0
    got = c.cache.view(c.pages, 3, -1)
    assert torch.equal(got[:, 0], clean[:, 0]) and torch.equal(got[:, 2], clean[:, 2])
