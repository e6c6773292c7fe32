"""The cache's calls at the largest arguments that they accept, and just beyond what they once took."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
from oracle import kv
from test_gpu_kv import call_attention, i32, ok

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
