"""Norms and rotation where fp32 comes to its limits (small angles, angles near quarter turns, the smallest and the largest
heads, any eps, signs of zeros): rows within bounds that are relative to each product, cells byte for byte, against the
oracle."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
import test_gpu_rope as base
import workloads
from gpu_util import host_bits
from oracle import mxfp4
from test_gpu_rope import Cache, Heads, scattered

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def set_values(h, v):
    h.bits = workloads.to_bf16_bits(v.astype(np.float32)).reshape(v.shape)
    h.load()


def firsts(h):
    """The dimensions that come first in their pairs."""
    return np.arange(0, h.rot, 2) if h.inter else np.arange(h.rot // 2)


def cached(h, page=16, seed=0):
    c = Cache(h, page, *scattered(h.T, page, seed))
    c.run()
    c.check()


def rows_are_near(h):
    """The result within BF16's rounding and 2^-19.5 of |y cos| + |y' sin|: the norm's reciprocal 2^-20.9 (nine roundings
    halved, two units in the last place), sine and cosine 2^-21.7, four roundings of 2^-24."""
    q, k = h.outputs()
    h.run(q, k)
    assert a4w4.a4w4_get_device_status() == 0
    for which, out, w in (("q", q, h.wq), ("k", k, h.wk)):
        y = mxfp4.bf16_bits_to_f64(h.part(h.bits, which))
        if w is not None:
            y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(base.EPS))) * w.astype(np.float64)
        reach = np.abs(y)
        for i in range(h.rot // 2):
            a, b = (2 * i, 2 * i + 1) if h.inter else (i, i + h.rot // 2)
            wide = np.longdouble if np.abs(h.pos).max() > 1000 else np.float64        # (slow where it has 113 bits)
            ang = np.asarray(h.pos, dtype=wide) * wide(h.freq[i])
            c, s = (np.abs(f(ang).astype(np.float64))[:, None] for f in (np.cos, np.sin))
            reach[..., a], reach[..., b] = (np.abs(y[..., a]) * c + np.abs(y[..., b]) * s,
                                            np.abs(y[..., b]) * c + np.abs(y[..., a]) * s)
        want, _ = h.want(which)
        got = mxfp4.bf16_bits_to_f64(host_bits(out))
        bad = ~(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19.5 * reach + 2.0 ** -133)
        assert not bad.any(), (which, bad.sum(), [(tuple(i), got[tuple(i)], want[tuple(i)]) for i in np.argwhere(bad)[:5]])


def small_angles(D, inter, norm, theta, low=0.0, T=100):
    h = Heads(T, 2, 3, D, D, inter, norm)
    h.freq = (theta ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
    h.pos = np.arange(1, T + 1, dtype=np.int32)
    v = mxfp4.bf16_bits_to_f64(h.bits)
    v[:, :, firsts(h)] *= low                                       # first halves nearly zero, of every other head
    v[:, 1::2] = np.where(np.isin(np.arange(D), firsts(h)), 0.0, v[:, 1::2])       # zero
    set_values(h, v)
    return h


@pytest.mark.parametrize("theta", [5e5, 1e7, 1e9])
@pytest.mark.parametrize("inter", [0, 1])
@pytest.mark.parametrize("D", [64, 128])
def test_small_angles(D, inter, theta):
    for norm, low in (("", 0.0), ("qk", 2.0 ** -20)):
        h = small_angles(D, inter, norm, theta, low)
        rows_are_near(h)
        cached(h)


@pytest.mark.parametrize("inter", [0, 1])
def test_angles_near_quarter_turns(inter):
    # sines of 355, 710, 103993, 104348, 245850922 ... are near zero, as are cosines of halves of them
    h = Heads(12, 2, 3, 128, 128, inter, "qk")
    h.pos = np.array([355, 710, 1, 2, 103993, 104348, 208341, 312689, 245850922, -355, -245850922, 3], dtype=np.int32)
    h.freq[0::4], h.freq[1::4], h.freq[2::4], h.freq[3::4] = 1.0, 0.5, np.float32(np.pi / 2), 1.5
    v = mxfp4.bf16_bits_to_f64(h.bits)
    for head in range(v.shape[1]):
        v[:, head, firsts(h)[head % 2:: 2]] = 0.0
    set_values(h, v)
    rows_are_near(h)
    cached(h)


def test_the_largest_heads():
    # A x passes fp32's range where r A x does not
    rng = np.random.default_rng(2)
    for D, inter in ((128, 0), (64, 1)):
        h = Heads(24, 3, 4, D, D, inter, "qk")
        v = np.sign(rng.standard_normal(h.bits.shape)) * rng.uniform(0.5, 0.99, h.bits.shape) * 2.0 ** 128
        v[::3] *= rng.choice([1.0, 2.0 ** -3, 2.0 ** -40], v[::3].shape)
        h.wq, h.wk = (3.0 * h.wq).astype(np.float32), (np.float32(2.0 ** 20) * h.wk).astype(np.float32)
        set_values(h, v)
        rows_are_near(h)
        cached(h)
        h = Heads(24, 0, 4, D, D, inter, "")                        # rotated keys up to sqrt(2) 2^128
        set_values(h, v[:, :9])
        cached(h)


@pytest.mark.parametrize("D,rot,inter,norm", [(128, 0, 0, ""), (64, 0, 1, "k"), (128, 64, 0, ""), (64, 32, 1, "qk"), (128, 128, 0, ""),
                                              (64, 64, 1, "qk")])
def test_zeros_keep_their_sign(D, rot, inter, norm):
    h = Heads(30, 2, 3, D, rot, inter, norm)
    rng = np.random.default_rng(3)
    h.bits[rng.random(h.bits.shape) < 0.3] = 0x8000
    h.bits[rng.random(h.bits.shape) < 0.2] = 0x0000
    h.bits[5], h.bits[6] = 0x8000, 0x0000
    h.load()
    cached(h)
    if rot == 0 and not norm:
        c = Cache(h, 16, *scattered(30, 16))
        c.run()
        other = torch.full_like(c.cache, 0xA5)
        a4w4.a4w4_kv_append(h.part(h.x, "k"), h.stride, h.part(h.x, "v"), h.stride, c.map, 30, 3, D, other, c.pages, 16)
        assert torch.equal(c.cache, other)


@pytest.mark.parametrize("scale", [-100, -120, -126, -130])
def test_the_smallest_keys(scale):
    for D, inter, rot, norm in ((128, 0, 128, ""), (64, 1, 32, ""), (128, 0, 64, "qk"), (64, 1, 64, "k")):
        h = Heads(40, 1, 4, D, rot, inter, norm)
        v = mxfp4.bf16_bits_to_f64(h.bits)
        v[::2, 1:3] = 0.0                                           # heads of zeros and of zeros but for a few dimensions
        v[::4, 1, 3], v[::4, 1, D // 2 + 3], v[::4, 2, 5] = 1.0, -1.0, -1.0
        set_values(h, np.ldexp(v, scale))
        cached(h)
        rows_are_near(h)


def test_the_smallest_weights_and_heads_of_few_large_values():
    h = Heads(40, 1, 4, 128, 128, 0, "qk")
    h.wk = np.ldexp(h.wk, np.random.default_rng(1).choice([-140, -120, -60, 0], 128)).astype(np.float32)
    h.load()
    cached(h)
    h = Heads(40, 1, 4, 128, 128, 0, "qk")
    v = mxfp4.bf16_bits_to_f64(h.bits)
    v[:, :, 32:64] *= 2.0 ** -120                                   # next to others of the head their squares are nothing
    v[:, :, 96:] *= 2.0 ** -125
    v[::2] *= 2.0 ** 90
    set_values(h, v)
    cached(h)
    rows_are_near(h)


@pytest.mark.parametrize("eps", [1e-45, 1e-42, 1e-38, 1e-30, 1e-12, 1.0])
def test_any_eps(eps, monkeypatch):
    monkeypatch.setattr(base, "EPS", eps)
    for scale in (-64, -67, -70, -75, -110, 0):
        h = Heads(24, 3, 3, 128, 128, 0, "qk")
        set_values(h, np.ldexp(mxfp4.bf16_bits_to_f64(h.bits), scale))
        rows_are_near(h)
        cached(h)
