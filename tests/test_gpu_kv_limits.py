"""The cache's calls at the largest arguments that they accept, and just beyond what they once took."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
from gpu_util import dev_bits, host_bits
from oracle import kv, mxfp4
from test_gpu_kv import call_attention, i32, ok, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def ones_cache(pages, page, Hkv, D):
    """Keys of zeros and values of ones in every cell."""
    z = np.zeros((page, Hkv, D), np.uint8)
    e = np.full((page, Hkv, D // 32), 127, np.uint8)
    return torch.from_numpy(kv.cache_from_rows(z, e, z + 2, e, page)).repeat(pages).cuda()


@pytest.mark.parametrize("max_q", [1, 256])                    # the kernel for few rows, and the one for many
@pytest.mark.parametrize("page,short", [(128, 0), (128, 700), (16, 0), (16, 345)])
def test_contexts_that_end_just_below_2_to_31(page, short, max_q):
    """Positions near the end of a table of 2^31 - 256 tokens (its pages repeat): lookups of whole runs of steps stay
    in the request's row of the table."""
    D, pages = 64, 1024
    width = (2 ** 31 - 256) // page
    lens = [width * page - short, 5]
    g = torch.Generator(device="cuda").manual_seed(1)
    table = torch.randint(0, pages, (2, width), generator=g, device="cuda", dtype=torch.int32)
    q = torch.randn(2, 1, D, generator=g, device="cuda").bfloat16()
    out, lse = call_attention(q, i32([0, 1, 2]), i32(lens), table, ones_cache(pages, page, 1, D), pages, page, 1, 1, D, 0.125, max_q)
    ok()
    assert (out == 1).all()
    assert np.allclose(lse.cpu().numpy()[:, 0], np.log(np.array(lens, np.float64)), rtol=2.0 ** -18, atol=0)


def test_a_plan_for_2_to_31_tokens():
    """max_tokens at its largest: the loop over the tokens ends, and every entry beyond the tokens is padding."""
    most, page = 2 ** 31 - 1, 16
    past, new = [30, 0, 7], [20, 1, -1]
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    ring = np.arange(20, 36, dtype=np.int32)
    want = kv.plan(past, new, page, table, ring, 3, 9, 64)
    t, r, state = i32(table), i32(ring), i32([3, 9])
    so, lens, cu, refused = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 3, 4, 1))
    slots, positions = (torch.full((most,), 7, dtype=torch.int32, device="cuda") for _ in range(2))
    a4w4.a4w4_kv_plan(i32(past), i32(new), 3, page, t, 4, r, 16, state, so, lens, cu, slots, positions, most, refused)
    ok()
    for k, x in (("block_table", t), ("free_ring", r), ("ring_state", so), ("kv_lens", lens), ("cu_new", cu), ("refused", refused),
                 ("slot_map", slots[:64]), ("positions", positions[:64])):
        assert np.array_equal(x.cpu().numpy(), want[k]), k
    assert int((slots[64:] != -1).sum()) == 0 and int((positions[64:] != 0).sum()) == 0


@pytest.mark.parametrize("past", [[65, 64, 4], [1000, 3, 70], [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]])
def test_a_plan_gives_back_no_more_than_a_row_of_the_table(past):
    """Finished requests longer than their rows (4 pages of 16), and one that is refused for its length."""
    page, new = 16, [-1, 2, -1]
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    ring = np.full(40, -3, np.int32)
    ring[:5] = np.arange(20, 25)
    want = kv.plan(past, new, page, table, ring, 0, 5, 8)
    buf = torch.full((36,), -9, dtype=torch.int32, device="cuda")      # the table with nothing of its own around it
    t = buf[12:24]
    t.copy_(i32(table.reshape(-1)))
    r, state = i32(ring), i32([0, 5])
    so, lens, cu, refused, slots, positions = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 3, 4, 1, 8, 8))
    a4w4.a4w4_kv_plan(i32(past), i32(new), 3, page, t, 4, r, 40, state, so, lens, cu, slots, positions, 8, refused)
    ok()
    for k, x in (("block_table", t.view(3, 4)), ("free_ring", r), ("ring_state", so), ("kv_lens", lens), ("cu_new", cu),
                 ("refused", refused), ("slot_map", slots), ("positions", positions)):
        assert np.array_equal(x.cpu().numpy(), want[k]), k
    assert (buf[:12] == -9).all() and (buf[24:] == -9).all()


# ---------------------------------------------------------------------------
# calls whose arguments allow for more work than there is

def widened(prob, width):
    """The same request lists over a table of `width` pages a row, made on the GPU."""
    table = torch.zeros(len(prob[1]), width, dtype=torch.int32, device="cuda")
    table[:, :prob[7].shape[1]] = i32(prob[7])
    return table


def check_widened(prob, width, max_q, rows=None):
    q_bits, q_lens, kv_lens, Hq, Hkv, D, page, _, cache, pages, vals, scale = prob
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    out, lse = call_attention(dev_bits(q_bits), i32(cu), i32(kv_lens), widened(prob, width), cache, pages, page, Hq, Hkv, D, scale, max_q)
    ok()
    got, gl, q = mxfp4.bf16_bits_to_f64(host_bits(out)), lse.cpu().numpy().astype(np.float64), mxfp4.bf16_bits_to_f64(q_bits)
    for b, n in enumerate(q_lens):
        for i in range(n) if rows is None else [i for i in rows if i < n]:
            seen = max(0, kv_lens[b] - n + i + 1)
            r = cu[b] + i
            if seen == 0:
                assert (got[r] == 0).all() and np.isneginf(gl[r]).all()
                continue
            o, l, spread, reach = kv.attention(q[r:r + 1], vals[b][0][:seen], vals[b][1][:seen], float(np.float32(scale)))
            bo, bl = kv.attention_bounds(o, l, spread, reach)
            assert np.all(np.abs(got[r:r + 1] - o) <= bo + 2.0 ** -9 * spread), (b, i)       # one BF16 term: 2^-8
            assert np.all(np.abs(gl[r:r + 1] - l) <= bl), (b, i)


def test_few_tokens_in_a_large_batch_on_a_wide_table():
    # 2000 places of a batch, 64 of them taken, rows of the table for 8 million tokens: 2^32 steps if all were full
    lens = [0] * 2000
    for b in range(0, 2000, 31):
        lens[b] = 1 + b % 77
    q_lens = [int(n > 0) for n in lens]
    check_widened(problem(q_lens, lens, 8, 8, 64, 128, 51), 65536, 2)


def test_one_chunk_in_a_large_batch_on_a_wide_table():
    rng = np.random.default_rng(52)
    lens, q_lens = rng.integers(1, 30, 2000).tolist(), [1] * 2000
    lens[1234], q_lens[1234] = 700, 600
    check_widened(problem(q_lens, lens, 8, 8, 64, 128, 53), 65536, 600, rows=(0, 1, 127, 128, 300, 599))


def test_a_chunk_of_which_b_times_its_length_passes_2_to_31():
    # 4000 requests, one of 70000 tokens: 2.2e9 rows of query heads if all were as long
    lens, q_lens = [7] * 4000, [1] * 4000
    lens[77], q_lens[77] = 300, 70000
    check_widened(problem(q_lens, lens, 8, 1, 64, 16, 54), 20, 70000, rows=(0, 69700, 69701, 69800, 69999))


@pytest.mark.parametrize("max_q,total", [(4, 64), (20000, 20000)])
def test_overlapping_rows_of_more_work_than_is_counted(max_q, total):
    """cu_q that goes up and down: every other request claims the same rows.  Nothing is computed, and the next call works."""
    B, Hq, Hkv, D, page, width = 4096, 64, 8, 64, 128, 32768
    cu = np.zeros(B + 1, np.int32)
    cu[1::2] = max_q
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    q = torch.zeros(total, Hq, D, dtype=torch.bfloat16, device="cuda")
    cache = ones_cache(1, page, Hkv, D)
    most = max(a4w4.a4w4_kv_attention_workspace_bytes(1, n, Hq, Hkv, D) for n in (max_q, 1))
    ws = torch.zeros(most, dtype=torch.uint8, device="cuda")
    out, _ = call_attention(q, i32(cu), i32([width * page] * B), table, cache, 1, page, Hq, Hkv, D, 1.0, max_q, ws=ws)
    ok()
    assert torch.isnan(out).all()
    out, _ = call_attention(q[:1], i32([0, 1]), i32([40]), table[:1], cache, 1, page, Hq, Hkv, D, 1.0, max_q, ws=ws)
    ok()
    assert (out == 1).all()
