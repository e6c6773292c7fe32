"""Pins of the oracle of norms and rotation, and the refusals of a4w4_qk_norm_rope and a4w4_kv_append_rope (no GPU needed)."""

import numpy as np
import pytest

import mxfp4_a4w4_gemm_gb300 as a4w4
from oracle import rope


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def test_rotation_keeps_lengths_and_relative_angles():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 1, 64))
    f = (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    for inter in (0, 1):
        y, _ = rope.heads(np.repeat(x[:1], 3, 0), None, 1.0, [0, 5, 9], f, 32, inter)
        z, _ = rope.heads(np.repeat(x[1:], 3, 0), None, 1.0, [2, 7, 11], f, 32, inter)
        assert np.array_equal(y[0], x[0])
        assert np.allclose((y ** 2).sum(-1), (x[0] ** 2).sum())
        assert np.allclose((y * z).sum(-1), (y[0] * z[0]).sum())       # the same distance, the same product
        assert np.array_equal(y[..., 32:], np.repeat(x[:1], 3, 0)[..., 32:])


def test_pairs_by_hand():
    x = np.zeros((1, 1, 64))
    x[0, 0, [0, 1, 16, 17]] = 1.0, 2.0, 3.0, 4.0
    f = np.zeros(16, np.float32)
    f[0] = 1.0
    c, s = np.cos(2.0), np.sin(2.0)
    half, _ = rope.heads(x, None, 1.0, [2], f, 32, 0)
    assert np.allclose(half[0, 0, [0, 16, 1, 17]], [c - 3 * s, 3 * c + s, 2.0, 4.0])
    inter, _ = rope.heads(x, None, 1.0, [2], f, 32, 1)
    assert np.allclose(inter[0, 0, [0, 1, 16, 17]], [c - 2 * s, 2 * c + s, 3.0, 4.0])


def test_norm_by_hand():
    x = np.full((1, 2, 64), 3.0)
    x[0, 1] = 0.0
    y, _ = rope.heads(x, np.full(64, 2.0), 2.0 ** -20, [0], None, 0, 0)
    assert np.allclose(y[0, 0], 2.0) and np.all(y[0, 1] == 0.0)


def refused(fn, good, change):
    with pytest.raises(a4w4.A4W4Error) as e:
        fn(*{**good, **change}.values(), stream=0)
    assert e.value.code == a4w4.A4W4_ERR_ARG, change


SHARED = [dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(Hq=4097), dict(Hq=4000, Hkv=100), dict(D=96), dict(D=256), dict(rot_dim=-16),
          dict(rot_dim=8), dict(rot_dim=144), dict(interleaved=2), dict(interleaved=-1), dict(eps=0.0), dict(eps=-1.0),
          dict(eps=float("nan")), dict(eps=float("inf")), dict(q_weight=8), dict(k_weight=4), dict(q_stride=4 * 128 - 8),
          dict(q_stride=4 * 128 + 4), dict(k_stride=4), dict(q_out_stride=8), dict(q=None), dict(q=8), dict(k=None), dict(k=2),
          dict(q_out=None), dict(q_out=4), dict(positions=None), dict(positions=2), dict(inv_freq=None), dict(inv_freq=2)]


def test_norm_rope_refusals():
    good = dict(q=16, q_stride=512, k=16, k_stride=256, positions=16, T=2, Hq=4, Hkv=2, D=128, q_weight=16, k_weight=16, eps=1e-6,
                inv_freq=16, rot_dim=128, interleaved=0, q_out=16, q_out_stride=512, k_out=16, k_out_stride=256)
    for change in SHARED + [dict(k_out=None), dict(k_out=8), dict(k_out_stride=128)]:
        refused(a4w4.a4w4_qk_norm_rope, good, change)


def test_append_rope_refusals():
    good = dict(q=16, q_stride=512, k=16, k_stride=256, v=16, v_stride=256, positions=16, slot_map=16, T=2, Hq=4, Hkv=2, D=128,
                q_weight=16, k_weight=16, eps=1e-6, inv_freq=16, rot_dim=128, interleaved=0, q_out=16, q_out_stride=512, cache=16,
                num_pages=4, page_size=16)
    for change in SHARED + [dict(Hkv=0), dict(v=None), dict(v=8), dict(v_stride=128), dict(slot_map=None), dict(slot_map=1),
                            dict(cache=None), dict(cache=8), dict(num_pages=0), dict(page_size=8), dict(num_pages=1 << 30)]:
        refused(a4w4.a4w4_kv_append_rope, good, change)


def test_rows_must_have_the_given_stride():
    torch = pytest.importorskip("torch")
    x = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        a4w4.a4w4_qk_norm_rope(x[:, :4], 64 * 4, None, 0, None, 3, 4, 0, 64, None, None, 1.0, None, 0, 0, x[:, :4], 64 * 8, None, 0, stream=0)
    with pytest.raises(ValueError):
        a4w4.a4w4_qk_norm_rope(x.transpose(0, 1), 64, None, 0, None, 3, 4, 0, 64, None, None, 1.0, None, 0, 0, x, 64 * 8, None, 0, stream=0)
