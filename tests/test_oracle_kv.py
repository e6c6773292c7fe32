"""Pins of the key/value cache oracle, and the refusals of the a4w4_kv_* calls (no GPU needed)."""

import numpy as np
import pytest

import mxfp4_a4w4_gemm_gb300 as a4w4
from oracle import kv, mxfp4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def test_plan_worked_example():
    # pages of 16: request 0 grows into a second page, 1 is finished (two pages), 2 starts, 3 finds no page left
    table = np.array([[5, -1, -1], [7, 9, -1], [-1, -1, -1], [4, -1, -1]], dtype=np.int32)
    ring = np.array([30, 31, 32, 33, 20, 21], dtype=np.int32)
    got = kv.plan([16, 20, 0, 10], [1, -1, 17, 20], 16, table, ring, 4, 3, 64)
    assert got["block_table"].tolist() == [[5, 20, -1], [7, 9, -1], [21, 30, -1], [4, -1, -1]]
    assert got["free_ring"].tolist() == [30, 7, 9, 33, 20, 21]
    assert got["ring_state"].tolist() == [1, 2]
    assert got["kv_lens"].tolist() == [17, 0, 17, 10]
    assert got["cu_new"].tolist() == [0, 1, 1, 18, 18]
    assert got["slot_map"][:18].tolist() == [20 * 16] + [21 * 16 + i for i in range(16)] + [30 * 16]
    assert got["slot_map"][18:].tolist() == [-1] * 46
    assert got["positions"][:3].tolist() == [16, 0, 1]
    assert got["refused"].tolist() == [1]


@pytest.mark.parametrize("D", [64, 128])
def test_chunk_layout_uses_every_byte_once(D):
    places = np.concatenate([p.reshape(-1) for p in kv.byte_places(D)])
    assert np.array_equal(np.sort(places), np.arange(17 * D))


def test_attention_of_one_key_is_its_value_and_of_equal_keys_their_mean():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((1, 4, 64)), rng.standard_normal((1, 2, 64)), rng.standard_normal((1, 2, 64))
    out, lse, spread, reach = kv.attention(q, k, v, 0.125)
    assert np.array_equal(out[0], v[0][[0, 0, 1, 1]])
    assert np.allclose(lse[0, 3], 0.125 * q[0, 3] @ k[0, 1])
    out, lse, _, _ = kv.attention(q, np.repeat(k, 5, 0), np.arange(5)[:, None, None] * np.ones((5, 2, 64)), 0.125)
    assert np.allclose(out, 2.0)
    assert np.allclose(lse[0, 0], 0.125 * q[0, 0] @ k[0, 0] + np.log(5))


def test_attention_is_causal_and_empty_rows_are_zero():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((4, 1, 64)), rng.standard_normal((2, 1, 64)), rng.standard_normal((2, 1, 64))
    out, lse, _, _ = kv.attention(q, k, v, 1.0)
    assert np.all(out[:2] == 0) and np.all(np.isneginf(lse[:2]))
    assert np.array_equal(out[2, 0], v[0, 0])
    assert np.all(np.isfinite(lse[2:]))


def test_cache_rows_are_where_the_chunk_says():
    rng = np.random.default_rng(2)
    c = rng.integers(0, 16, (2, 64, 3, 128)).astype(np.uint8)
    s = rng.integers(0, 255, (2, 64, 3, 4)).astype(np.uint8)
    cache = kv.cache_from_rows(c[0], s[0], c[1], s[1], 32).reshape(2, 3, 2, 17 * 128)
    want = kv.chunk_bytes(c[0, 48:, 1], s[0, 48:, 1], c[1, 48:, 1], s[1, 48:, 1])
    assert np.array_equal(cache[1, 1, 1], want)
    assert mxfp4.unpack_codes(cache[1, 1, 1][0:1])[0] == c[0, 48, 1, 0]


# ---------------------------------------------------------------------------
# refusals: arguments are looked at before any device is

def refused(fn, *args, code=a4w4.A4W4_ERR_ARG, **kw):
    with pytest.raises(a4w4.A4W4Error) as e:
        fn(*args, stream=0, **kw)
    assert e.value.code == code


PLAN = dict(past_lens=16, new_lens=32, B=2, page_size=16, block_table=48, max_pages=4, free_ring=64, ring_size=8,
            ring_state=80, ring_state_out=96, kv_lens=112, cu_new=128, slot_map=144, positions=160, max_tokens=4, refused=176)


@pytest.mark.parametrize("change", [
    dict(B=0), dict(B=4097), dict(page_size=24), dict(page_size=256), dict(max_pages=0), dict(ring_size=0), dict(max_tokens=-1),
    dict(max_pages=1 << 27), dict(past_lens=None), dict(new_lens=18), dict(block_table=0), dict(slot_map=None),
    dict(positions=2), dict(ring_state_out=80), dict(kv_lens=16), dict(kv_lens=32), dict(refused=None)])
def test_plan_refuses(change):
    refused(a4w4.a4w4_kv_plan, **{**PLAN, **change})


APPEND = dict(k=16, k_stride=256, v=32, v_stride=256, slot_map=48, T=3, Hkv=2, D=128, cache=64, num_pages=4, page_size=16)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(Hkv=0), dict(D=96), dict(D=256), dict(num_pages=0), dict(page_size=8), dict(k=8), dict(v=None),
    dict(cache=8), dict(slot_map=50), dict(k_stride=255), dict(v_stride=248), dict(num_pages=1 << 27)])
def test_append_refuses(change):
    refused(a4w4.a4w4_kv_append, **{**APPEND, **change})


READ = dict(cache=16, num_pages=4, page_size=16, slot_map=32, T=3, Hkv=2, D=64, k_out=48, v_out=64)


@pytest.mark.parametrize("change", [dict(T=-1), dict(D=32), dict(k_out=8), dict(v_out=None), dict(cache=None), dict(page_size=0)])
def test_read_refuses(change):
    refused(a4w4.a4w4_kv_read, **{**READ, **change})


ATTENTION = dict(q=16, q_stride=1024, cu_q=32, B=2, total_q=3, max_q=2, kv_lens=48, block_table=64, max_pages=4, cache=80,
                 num_pages=8, page_size=16, Hq=8, Hkv=2, D=128, sm_scale=0.1, out=96, lse=112, ws=128, ws_bytes=1 << 40)


@pytest.mark.parametrize("change", [
    dict(B=0), dict(total_q=-1), dict(max_q=0), dict(max_pages=0), dict(num_pages=0), dict(page_size=48), dict(Hq=7), dict(Hq=0),
    dict(Hkv=0), dict(D=192), dict(q_stride=1016), dict(q_stride=1028), dict(sm_scale=0.0), dict(sm_scale=-1.0),
    dict(sm_scale=float("nan")), dict(sm_scale=float("inf")), dict(q=24), dict(out=100), dict(lse=113), dict(cache=None),
    dict(cu_q=None), dict(kv_lens=1), dict(block_table=None), dict(max_pages=1 << 27), dict(B=1 << 16, max_q=1 << 14)])
def test_attention_refuses(change):
    refused(a4w4.a4w4_kv_attention, **{**ATTENTION, **change})


def test_attention_refuses_a_small_workspace():
    need = a4w4.a4w4_kv_attention_workspace_bytes(2, 2, 8, 2, 128)
    assert need > 0
    refused(a4w4.a4w4_kv_attention, **{**ATTENTION, "ws_bytes": need - 1}, code=a4w4.A4W4_ERR_WORKSPACE)
    refused(a4w4.a4w4_kv_attention, **{**ATTENTION, "ws": None}, code=a4w4.A4W4_ERR_WORKSPACE)
    refused(a4w4.a4w4_kv_attention, **{**ATTENTION, "ws": 8}, code=a4w4.A4W4_ERR_WORKSPACE)


def test_sizes():
    assert a4w4.a4w4_kv_cache_bytes(10, 64, 8, 128) == 10 * 64 * 8 * 136
    assert a4w4.a4w4_kv_cache_bytes(3, 16, 1, 64) == 3 * 16 * 68
    assert a4w4.a4w4_kv_cache_bytes(0, 16, 1, 64) == 0
    assert a4w4.a4w4_kv_cache_bytes(3, 16, 1, 80) == 0
    assert a4w4.a4w4_kv_attention_workspace_bytes(2, 2, 8, 3, 128) == 0
