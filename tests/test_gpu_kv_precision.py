"""How exact attention's probabilities are where a few keys carry a row, in either kernel, and that the answers of the
kernel for many rows do not hang on the block table's width."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
import workloads
from gpu_util import dev_bits, host_bits
from oracle import kv, mxfp4
from test_gpu_kv import call_attention, i32, ok, problem

pytestmark = pytest.mark.gpu

PROMPT = 256                                   # a bound on new tokens that sends any call to the kernel for many rows


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def two_keys(B, G, D, kv_len, page, seed):
    """B requests of one new token; two of their keys carry a row, the second with p in (1/2, 1) of the first and a value of
    ones; the other keys are e^-24 of the first and have values too.  Every product is exact."""
    rng = np.random.default_rng(seed)
    pages = B * -(-kv_len // page)
    keys, vals = np.zeros((B, kv_len, 1, D)), np.zeros((B, kv_len, 1, D))
    keys[:, :, 0, 2] = -24
    order = np.argsort(rng.random((B, kv_len)), axis=1)[:, :2]
    vals[:, :, 0, :] = rng.choice([-1.0, 1.0], (B, kv_len, 1))
    b = np.arange(B)
    keys[b, order[:, 0]], vals[b, order[:, 0]] = 0, 0
    keys[b, order[:, 1]], vals[b, order[:, 1]] = 0, 1
    keys[b, order[:, 1], 0, 1] = 1
    q = np.zeros((B, G, D))
    q[..., 1] = -rng.uniform(0.001, 0.69, (B, G))
    q[..., 2] = 1
    q_bits = workloads.to_bf16_bits(q)
    table = rng.permutation(pages).astype(np.int32).reshape(B, -1)
    parts = [np.zeros((pages * page, 1, n), np.uint8) for n in (D, D // 32) * 2]
    slot = np.take_along_axis(table, np.arange(kv_len)[None] // page, 1) * page + np.arange(kv_len) % page
    for i, x in enumerate((keys, vals)):
        parts[2 * i][slot], parts[2 * i + 1][slot] = (a.reshape(B, kv_len, 1, -1) for a in mxfp4.quantize_blocks(x.reshape(-1, 1, D)))
    cache = torch.from_numpy(kv.cache_from_rows(*parts, page)).cuda()
    return q_bits, keys, vals, table, cache, pages


@pytest.mark.parametrize("kv_len", [2, 60, 128])
@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (64, 12), (128, 16)])
@pytest.mark.parametrize("max_q,p_round", [(PROMPT, kv.P_TWO_BF16), (1, kv.P_FP16)])
def test_few_keys_carry_a_row(kv_len, D, G, max_q, p_round):
    """Up to 128 keys: the output is off by its own rounding and little more, on a table of any width."""
    B, page = 400 // G, 16
    q_bits, keys, vals, table, cache, pages = two_keys(B, G, D, kv_len, page, 61)
    q, want, bound = mxfp4.bf16_bits_to_f64(q_bits), [], []
    for b in range(B):
        o, l, spread, reach = kv.attention(q[b:b + 1], keys[b], vals[b], 1.0)
        dx = (2.0 ** -17 + 2.0 ** -22) * reach
        rel = 2 * np.expm1(dx) + p_round + 2.0 ** -18 + kv_len * 2.0 ** -23
        want.append(o)
        bound.append(rel[..., None] * spread)
    want, bound = np.concatenate(want), np.concatenate(bound)
    bound = bound + 2.0 ** (np.floor(np.log2(np.abs(want) + bound)) - 8)        # half a unit in the output's last place
    for width in (table.shape[1], 4096):
        wide = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = i32(table)
        out, _ = call_attention(dev_bits(q_bits), i32(np.arange(B + 1)), i32([kv_len] * B), wide, cache, pages, page, G, 1, D, 1.0, max_q)
        ok()
        err = np.abs(mxfp4.bf16_bits_to_f64(host_bits(out)) - want)
        assert np.all(err <= bound), (width, float(np.max(err / bound)))


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page", [
    ([128], [128], 1, 1, 128, 16), ([70, 1, 200], [570, 300, 200], 4, 2, 128, 16), ([300], [300], 3, 1, 64, 64),
    ([600, 5], [600, 470], 2, 2, 64, 32), ([40, 33, 90], [39, 3, 300], 8, 1, 64, 16)])
def test_the_width_of_the_table_changes_nothing(q_lens, kv_lens, Hq, Hkv, D, page):
    """The kernel for many rows: the same bits on a table as wide as the longest request and on wider ones."""
    q_bits, _, _, _, _, _, _, table, cache, pages, _, scale = problem(q_lens, kv_lens, Hq, Hkv, D, page, 62)
    cu, lens, got = i32(np.concatenate([[0], np.cumsum(q_lens)])), i32(kv_lens), []
    for width in (table.shape[1], 640 // page, 131072 // page):
        wide = torch.zeros(len(q_lens), width, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = i32(table)
        got.append(call_attention(dev_bits(q_bits), cu, lens, wide, cache, pages, page, Hq, Hkv, D, scale, max(PROMPT, max(q_lens))))
        ok()
    for out, lse in got[1:]:
        assert torch.equal(out.view(torch.int16), got[0][0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), got[0][1].view(torch.int32))
