"""Sizes that the 8-bit product's entry points give (no GPU needed)."""

import pytest

import mxfp4_a4w4_gemm_gb300 as a4w4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


@pytest.mark.parametrize("M", [33, 128, 129, 1 << 20, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 1])
def test_workspace_is_a_tile_for_each_128_tokens_and_ks(M):
    for N, K in ((128, 128), (1536, 7168)):
        assert a4w4.a4w4_gemm_w8a8_workspace_bytes(M, N, K) == -(-M // 128) * (K // 128) * (128 * 128 + 128 * 4)


@pytest.mark.parametrize("M", [-1, 0, 1, 32])
def test_few_tokens_need_none(M):
    assert a4w4.a4w4_gemm_w8a8_workspace_bytes(M, 256, 256) == 0
