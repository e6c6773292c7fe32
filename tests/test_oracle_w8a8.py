"""Pins of the 8-bit product's oracle, and the refusals of the a4w4_*w8* calls (no GPU needed)."""

import numpy as np
import pytest

import mxfp4_a4w4_gemm_gb300 as a4w4
from oracle import w8a8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def test_e4m3_agrees_with_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * np.exp2(rng.integers(-12, 9, 4000)), w8a8.decode(np.arange(127)),
                        (w8a8.decode(np.arange(126)) + w8a8.decode(np.arange(1, 127))) / 2])       # values and midpoints
    x = x[np.abs(x) <= 448.0]
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn)
    assert np.array_equal(w8a8.e4m3(x.astype(np.float32).astype(np.float64)), want.double().numpy())
    assert np.array_equal(w8a8.encode(w8a8.e4m3(x)) & 127, want.view(torch.uint8).numpy() & 127)
    assert w8a8.e4m3(1e9) == 448.0 and w8a8.e4m3(-449.0) == -448.0


def test_activation_scales_are_the_smallest_powers_of_two():
    a = np.zeros((5, 256))
    a[0, 3], a[0, 200] = 448.0, 448.0001
    a[1, 0], a[1, 255] = -224.0, 2.0 ** -140
    a[2, 7] = np.inf
    a[3, 130] = np.nan
    q, s = w8a8.quant_activations(a)
    assert s[0].tolist() == [1.0, 2.0] and s[1].tolist() == [0.5, 2.0 ** -126]
    assert np.isnan(s[2, 0]) and s[2, 1] == 2.0 ** -126 and np.isnan(s[3, 1])
    assert q[0, 3] == 448.0 and q[0, 200] == 224.0 and q[1, 0] == -448.0 and q[1, 255] == 0.0


def test_tiles_use_every_byte_once():
    codes = np.arange(256 * 384).reshape(256, 384)
    flat = np.empty(256 * 384, dtype=np.int64)
    n, k = 129, 257
    got = w8a8.tiles((codes % 251).astype(np.uint8))
    flat[:] = got
    # row 129 is row 1 of the second tile of rows; k 257 is byte 1 of the third tile of bytes: piece 0 ^ 1 of row 1
    assert flat[(1 * 3 + 2) * 16384 + 128 + 16 + 1] == codes[n, k] % 251


def test_sizes():
    assert a4w4.a4w4_w8_weight_bytes(384, 256) == 384 * 256
    assert a4w4.a4w4_gemm_w8a8_workspace_bytes(1, 7168, 4224) == 0
    assert a4w4.a4w4_gemm_w8a8_workspace_bytes(129, 1536, 4224) == 2 * 33 * (16384 + 512)
    assert a4w4.a4w4_gemm_w8a8_workspace_bytes(0, 128, 128) == 0


def refused(code, fn, *args):
    with pytest.raises(a4w4.A4W4Error) as e:
        fn(*args, stream=0)
    assert e.value.code == code


def test_refusals_need_no_device():
    arg = a4w4.A4W4_ERR_ARG
    good = dict(A=16, M=1, K=256, W8=16, Ws=16, N=256, C=16, workspace=None, ws_bytes=0, flags=0)

    def call(**change):
        refused(arg, a4w4.a4w4_gemm_w8a8, *{**good, **change}.values())

    for change in (dict(M=0), dict(M=-1), dict(N=0), dict(N=192), dict(K=0), dict(K=192), dict(A=None), dict(A=8), dict(W8=None),
                   dict(W8=24), dict(Ws=None), dict(Ws=2), dict(C=None), dict(C=2), dict(flags=2)):
        call(**change)
    for fn in (a4w4.a4w4_prepare_w8_weight,):
        for a in ((16, 192, 128, 16, 16), (16, 128, 64, 16, 16), (16, 0, 128, 16, 16), (8, 128, 128, 16, 16), (16, 128, 128, None, 16),
                  (16, 128, 128, 16, 2), (16, 128, 128, 16, None)):
            refused(arg, fn, *a)
    for a in ((16, 192, 128, 32), (16, 128, 64, 32), (None, 128, 128, 32), (16, 128, 128, 8), (16, 128, 128, 16)):
        refused(arg, a4w4.a4w4_shuffle_w8_weight, *a)
