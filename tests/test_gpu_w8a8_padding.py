"""Weights whose sizes are no multiples of 128, padded with zeros, through the 8-bit product; NaN and infinities in either form."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
from gpu_util import host_bits
from oracle import mxfp4, w8a8
from test_gpu_w8a8 import Product, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


@pytest.mark.parametrize("M", [1, 20, 70, 1100])
def test_padding_of_zeros(M):
    # 192 rows of 200 k's: the last blocks hold 64 rows, 72 k's
    a_bits, w, ws = problem(M, 256, 256)
    a_bits[:, 200:], w[192:], w[:, 200:] = 0, 0.0, 0.0
    p = Product(a_bits, w, ws)
    p.run()
    p.check()
    assert np.all(mxfp4.bf16_bits_to_f64(host_bits(p.C))[:M, 192:] == 0.0)
    c, reach = w8a8.gemm(mxfp4.bf16_bits_to_f64(a_bits), w, ws)
    assert np.all(np.abs(mxfp4.bf16_bits_to_f64(host_bits(p.C))[:M, :192] - c[:, :192]) <= w8a8.bound(c, reach, 256)[:, :192])


@pytest.mark.parametrize("M", [3, 40, 1100])
@pytest.mark.parametrize("pattern", [0x7F80, 0xFF80, 0x7FC0, 0xFFFF, 0x7F81])
def test_infinity_or_nan_anywhere_makes_its_row_nan(M, pattern):
    a_bits, w, ws = problem(M, 256, 384)
    w[:, 130] = 0.0                                                 # even where the weights are zero
    a_bits[1, 130] = pattern
    a_bits[2, 256:] = pattern                                       # a whole block
    p = Product(a_bits, w, ws)
    p.run()
    assert a4w4.a4w4_get_device_status() == 0
    nan = torch.isnan(p.C[:M]).all(1).cpu().numpy()
    assert np.array_equal(np.nonzero(nan)[0], [1, 2]) and not torch.isnan(p.C[:M][~torch.from_numpy(nan).cuda()]).any()
