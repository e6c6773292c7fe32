"""GPU parity of the paged MXFP4 key/value cache: plan, append, read and
attention against the oracle, at the sizes and masks where they can go wrong."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
import workloads
from gpu_util import dev_bits, host_bits
from oracle import kv, mxfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def ok():
    assert a4w4.a4w4_get_device_status() == 0


# ---------------------------------------------------------------------------
# plan

def run_plan(past, new, page, table, ring, head, count, max_tokens, times=1):
    B, width = table.shape
    t, r, st = i32(table), i32(ring), i32([head, count])
    out = {k: torch.full((n,), -7, dtype=torch.int32, device="cuda") for k, n in
           (("ring_state", 2), ("kv_lens", B), ("cu_new", B + 1), ("slot_map", max_tokens), ("positions", max_tokens), ("refused", 1))}
    p, n = i32(past), i32(new)
    for _ in range(times):
        a4w4.a4w4_kv_plan(p, n, B, page, t, width, r, len(ring), st, out["ring_state"], out["kv_lens"], out["cu_new"],
                          out["slot_map"], out["positions"], max_tokens, out["refused"])
    ok()
    out.update(block_table=t, free_ring=r)
    return {k: v.cpu().numpy() for k, v in out.items()}


def random_plan(B, page, seed, tight, longest=300, new_most=40):
    rng = np.random.default_rng(seed)
    past = rng.integers(0, longest, B)
    new = rng.choice([0, 1, 1, 1, -1, 2, page, new_most], B)
    width = -(-(longest + new_most) // page) - (1 if tight else 0)      # tight: some rows of the table are too short
    pages = B * width + 9
    ids = rng.permutation(pages)
    table = ids[:B * width].reshape(B, width).astype(np.int32)
    need = sum(-(-(p + n) // page) - -(-p // page) for p, n in zip(past, new) if n > 0)
    count = need // 2 if tight else need + 3
    ring = np.full(pages, -1, np.int32)
    head = pages - max(1, count // 2)
    ring[(head + np.arange(count)) % pages] = rng.permutation(pages)[:count]
    tokens = int(new[new > 0].sum()) + 5
    return past, new, page, table, ring, head, count, tokens


@pytest.mark.parametrize("B,page,tight", [(1, 16, False), (2, 128, True), (31, 32, False), (33, 16, True), (512, 64, False),
                                          (513, 16, True), (1025, 32, False), (4096, 16, True)])
def test_plan_matches_the_oracle(B, page, tight):
    args = random_plan(B, page, B + page, tight)
    want = kv.plan(*args)
    for times in (1, 2):                       # the same call again gives the same
        got = run_plan(*args, times=times)
        for k in want:
            assert np.array_equal(got[k], want[k]), k


def test_plan_runs_out_of_tokens_and_serves_in_order():
    args = list(random_plan(40, 16, 3, False))
    args[-1] = args[-1] // 3
    want, got = kv.plan(*args), run_plan(*args)
    assert 0 < want["refused"][0] < 40
    for k in want:
        assert np.array_equal(got[k], want[k]), k


def test_plan_without_tokens_or_pages():
    table = np.full((3, 2), -1, np.int32)
    got = run_plan([0, 5, 0], [4, 0, 1], 16, table, np.arange(4, dtype=np.int32), 2, 0, 0)
    assert got["refused"][0] == 2 and got["cu_new"].tolist() == [0, 0, 0, 0] and got["kv_lens"].tolist() == [0, 5, 0]
    assert got["ring_state"].tolist() == [2, 0]


def test_plan_of_long_requests():
    # positions beyond 2^24, a table row of its full width
    page, width = 128, 1 << 18
    table = np.arange(width, dtype=np.int32)[None].copy()
    past, new = width * page - 200, 200
    got = run_plan([past], [new], page, table, np.array([width], np.int32), 0, 1, 256)
    want = kv.plan([past], [new], page, table, np.array([width], np.int32), 0, 1, 256)
    for k in want:
        assert np.array_equal(got[k], want[k]), k
    got = run_plan([past], [new + 1], page, table, np.array([width], np.int32), 0, 1, 256)
    assert got["refused"][0] == 1 and got["kv_lens"][0] == past


# ---------------------------------------------------------------------------
# append and read

def row_bits(T, H, D, seed):
    """BF16 rows with outliers, ties, subnormals and zero blocks."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, D)) * rng.choice([1e-3, 1.0, 30.0], (T, H, 1))
    bits = workloads.to_bf16_bits(x)
    flat = bits.reshape(-1, 32)
    flat[::7] = 0
    flat[3::11] = rng.integers(0, 0x7F80, flat[3::11].shape) | (rng.integers(0, 2, flat[3::11].shape) << 15)   # any finite value
    flat[5::13, 0] = 0x40C0                                                                                    # 6: blocks full of ties
    flat[5::13, 1:9] = workloads.to_bf16_bits(np.array([0.25, -0.75, 1.25, -1.75, 2.5, -3.5, 5.0, -0.0], np.float32))
    return bits


def slots_for(T, pages, page, seed):
    s = np.random.default_rng(seed).permutation(pages * page)[:T].astype(np.int32)
    if T > 4:
        s[1], s[T // 2] = -1, pages * page                # both outside: skipped, read as zeros
    return s


def quantised(bits):
    c, e = mxfp4.quantize_blocks(mxfp4.bf16_bits_to_f64(bits))
    return c, e


@pytest.mark.parametrize("T,Hkv,D,page,fused", [(1, 1, 64, 16, False), (1, 8, 128, 64, True), (5, 3, 128, 16, True), (16, 2, 64, 32, False),
                                                (100, 5, 64, 128, True), (257, 8, 128, 32, False), (1000, 1, 128, 128, True)])
def test_append_then_read(T, Hkv, D, page, fused):
    pages = T // page + 3
    kb, vb = row_bits(T, Hkv, D, 1), row_bits(T, Hkv, D, 2)
    if fused:                                             # slices of one projection, another head before and after
        x = torch.cat([torch.zeros(T, 1, D).bfloat16(), workloads.bits_to_torch(kb), workloads.bits_to_torch(vb),
                       torch.zeros(T, 1, D).bfloat16()], 1).cuda()
        k, v = x[:, 1:1 + Hkv], x[:, 1 + Hkv:1 + 2 * Hkv]
    else:
        k, v = dev_bits(kb), dev_bits(vb)
    slots = slots_for(T, pages, page, 3)
    n = a4w4.a4w4_kv_cache_bytes(pages, page, Hkv, D)
    before = np.random.default_rng(4).integers(0, 256, n).astype(np.uint8)
    cache = torch.from_numpy(before).cuda()
    sm = i32(slots)
    a4w4.a4w4_kv_append(k, k.stride(0), v, v.stride(0), sm, T, Hkv, D, cache, pages, page)
    ok()
    # every byte: the rows at their places, everything else untouched
    live = (slots >= 0) & (slots < pages * page)
    rows = []
    for bits in (kb, vb):
        c, e = quantised(bits)
        cc, ee = np.zeros((pages * page, Hkv, D), np.uint8), np.zeros((pages * page, Hkv, D // 32), np.uint8)
        cc[slots[live]], ee[slots[live]] = c[live], e[live]
        rows += [cc, ee]
    hit = np.zeros(pages * page, np.uint8)
    hit[slots[live]] = 255
    mask = kv.cache_from_rows(*[np.broadcast_to(hit[:, None, None], r.shape) & (0xFF if i % 2 else 0x0F) for i, r in enumerate(rows)], page)
    want = np.where(mask == 255, kv.cache_from_rows(*rows, page), before)
    assert np.array_equal(cache.cpu().numpy(), want)
    ko = torch.full((T, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vo = torch.full_like(ko, float("nan"))
    a4w4.a4w4_kv_read(cache, pages, page, sm, T, Hkv, D, ko, vo)
    ok()
    for got, bits in ((ko, kb), (vo, vb)):
        c, e = quantised(bits)
        val = mxfp4.decode(c, e) * live[:, None, None]
        assert np.array_equal(mxfp4.bf16_bits_to_f64(host_bits(got)), val)
        # the sign of zero is kept
        assert np.array_equal(host_bits(got)[live] >> 15, (c[live] >> 3).astype(np.uint16))


def test_append_and_read_of_nothing():
    cache = torch.zeros(a4w4.a4w4_kv_cache_bytes(1, 16, 1, 64), dtype=torch.uint8, device="cuda")
    a4w4.a4w4_kv_append(None, 64, None, 64, None, 0, 1, 64, cache, 1, 16)
    a4w4.a4w4_kv_read(cache, 1, 16, None, 0, 1, 64, None, None)
    ok()
    assert not cache.any()


def test_cache_offsets_beyond_32_bits():
    # 4.6 GB of cache: the last pages lie past 2^32 bytes
    page, Hkv, D = 128, 8, 128
    pages = 33000
    n = a4w4.a4w4_kv_cache_bytes(pages, page, Hkv, D)
    assert n > 1 << 32
    cache = torch.zeros(n, dtype=torch.uint8, device="cuda")
    T = 200
    kb, vb = row_bits(T, Hkv, D, 5), row_bits(T, Hkv, D, 6)
    kb.reshape(-1, 32)[:, :] = np.where((kb.reshape(-1, 32) & 0x7F80) > 0x4200, 0x3F80, kb.reshape(-1, 32))
    vb.reshape(-1, 32)[:, :] = np.where((vb.reshape(-1, 32) & 0x7F80) > 0x4200, 0x3F80, vb.reshape(-1, 32))
    slots = (pages * page - T + np.arange(T)).astype(np.int32)
    k, v = dev_bits(kb), dev_bits(vb)
    a4w4.a4w4_kv_append(k, Hkv * D, v, Hkv * D, i32(slots), T, Hkv, D, cache, pages, page)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    a4w4.a4w4_kv_read(cache, pages, page, i32(slots), T, Hkv, D, ko, vo)
    ok()
    kc, vc = (mxfp4.decode(*quantised(b)) for b in (kb, vb))
    assert np.array_equal(mxfp4.bf16_bits_to_f64(host_bits(ko)), kc)
    assert np.array_equal(mxfp4.bf16_bits_to_f64(host_bits(vo)), vc)
    # attention over the tokens of those pages: the first of them starts inside a page
    table = np.array([[pages - 2, pages - 1]], np.int32)
    first = 2 * page - T
    q = np.random.default_rng(7).standard_normal((1, 16, D))
    keys, vals = np.zeros((2 * page, Hkv, D)), np.zeros((2 * page, Hkv, D))
    keys[first:], vals[first:] = kc, vc
    check_attention(workloads.to_bf16_bits(q), [1], [2 * page], 16, Hkv, D, page, table, cache, pages, [(keys, vals)], 0.05)


# ---------------------------------------------------------------------------
# attention

def call_attention(q, cu, lens, table, cache, pages, page, Hq, Hkv, D, scale, max_q, ws=None, out=None, lse=True, stream=None):
    B = len(lens)
    total = q.shape[0]
    out = torch.full((total, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    l = torch.full((total, Hq), float("nan"), dtype=torch.float32, device="cuda") if lse else None
    if ws is None:
        n = a4w4.a4w4_kv_attention_workspace_bytes(B, max_q, Hq, Hkv, D)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        a4w4.a4w4_workspace_init(ws, n)
    a4w4.a4w4_kv_attention(q, q.stride(0), cu, B, total, max_q, lens, table, table.shape[1], cache, pages, page, Hq, Hkv, D,
                           scale, out, l, ws, ws.numel(), stream=stream)
    return out, l


def check_attention(q_bits, q_lens, kv_lens, Hq, Hkv, D, page, table, cache, pages, rows, scale, max_q=None, p_extra=0.0):
    """One call against the oracle; rows[b] = (keys, values) float64 [len, Hkv, D] of request b; p_extra: what a
    probability's rounding may be off by beyond the bound's 2^-9, relatively."""
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    out, lse = call_attention(dev_bits(q_bits), i32(cu), i32(kv_lens), i32(table), cache, pages, page, Hq, Hkv, D, scale,
                              max_q or max(1, max(q_lens)))
    ok()
    got, gl = mxfp4.bf16_bits_to_f64(host_bits(out)), lse.cpu().numpy().astype(np.float64)
    q = mxfp4.bf16_bits_to_f64(q_bits)
    for b, n in enumerate(q_lens):
        if n == 0:
            continue
        sl = slice(cu[b], cu[b + 1])
        o, l, spread, reach = kv.attention(q[sl], rows[b][0], rows[b][1], float(np.float32(scale)))
        bo, bl = kv.attention_bounds(o, l, spread, reach)
        bo = bo + p_extra * spread
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(gl[sl]), empty), b
        assert np.all(got[sl][empty] == 0)
        bad = np.argwhere(~(np.abs(got[sl] - o) <= bo))
        assert bad.size == 0, (b, len(bad), bad[:4].tolist(), float(np.nanmax(np.abs(got[sl] - o) / np.maximum(bo, 1e-300))))
        e = np.abs(np.where(empty, 0, gl[sl]) - np.where(empty, 0, l))
        assert np.all(e <= bl), (b, float(np.max(e / bl)))
    return out, lse


def problem(q_lens, kv_lens, Hq, Hkv, D, page, seed, q_gain=1.0, k_gain=None, v_gain=None):
    """Random ragged problem; every cell of the cache that no request holds, the tails of last pages among them, is
    a NaN scale with full codes."""
    rng = np.random.default_rng(seed)
    held = [-(-n // page) for n in kv_lens]
    pages, width = sum(held) + 2, max(1, max(held))
    ids = rng.permutation(pages)
    table = np.zeros((len(kv_lens), width), np.int32)
    codes = [np.full((pages * page, Hkv, D), 15, np.uint8) for _ in range(2)]
    scales = [np.full((pages * page, Hkv, D // 32), 255, np.uint8) for _ in range(2)]
    rows, at = [], 0
    for b, n in enumerate(kv_lens):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
        tok = np.arange(n)
        slot = table[b, tok // page] * page + tok % page if n else tok
        vals = []
        for which, gain in ((0, k_gain), (1, v_gain)):
            x = rng.standard_normal((n, Hkv, D))
            if gain is not None:
                x = x * gain(rng, (n, Hkv, D))
            c, e = mxfp4.quantize_blocks(mxfp4.bf16_bits_to_f64(workloads.to_bf16_bits(x))) if n else (codes[0][:0], scales[0][:0])
            codes[which][slot], scales[which][slot] = c, e
            vals.append(mxfp4.decode(c, e) if n else np.zeros((0, Hkv, D)))
        rows.append(tuple(vals))
    cache = torch.from_numpy(kv.cache_from_rows(codes[0], scales[0], codes[1], scales[1], page)).cuda()
    q_bits = workloads.to_bf16_bits(rng.standard_normal((sum(q_lens), Hq, D)) * q_gain)
    return (q_bits, q_lens, kv_lens, Hq, Hkv, D, page, table, cache, pages, rows, 1.0 / np.sqrt(D))


EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1025]


@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 4, 128, 16), (8, 1, 64, 32), (6, 2, 128, 64), (14, 2, 64, 128), (16, 1, 128, 16), (36, 3, 64, 16)])
def test_single_tokens_over_lengths(Hq, Hkv, D, page):
    check_attention(*problem([1] * len(EDGES), EDGES, Hq, Hkv, D, page, 11))


@pytest.mark.parametrize("B,kv_len,Hq,Hkv,D,page", [(1, 3000, 8, 1, 128, 64), (2, 5001, 32, 2, 64, 16), (1, 12000, 5, 1, 128, 32)])
def test_long_contexts_are_split_and_joined(B, kv_len, Hq, Hkv, D, page):
    check_attention(*problem([1] * B, [kv_len - 7 * b for b in range(B)], Hq, Hkv, D, page, 12))


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (24, 1, 64), (32, 1, 128)])
def test_empty_requests_idle_rows_and_more_queries_than_keys(Hq, Hkv, D):
    q_lens, kv_lens = [1, 0, 3, 4, 1, 0, 2], [0, 50, 2, 0, 17, 0, 2]
    check_attention(*problem(q_lens, kv_lens, Hq, Hkv, D, 16, 13))


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 8, 128, 16), (8, 2, 64, 64), (16, 2, 128, 32), (40, 1, 64, 16)])
def test_several_new_tokens_per_request(Hq, Hkv, D, page):
    check_attention(*problem([2, 5, 1, 8, 3], [130, 5, 64, 301, 16], Hq, Hkv, D, page, 14))


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page", [
    ([128], [128], 1, 1, 128, 16), ([129], [129], 2, 1, 64, 32), ([300], [300], 3, 1, 128, 64), ([70, 1, 200], [570, 300, 200], 4, 2, 128, 16),
    ([257, 31], [900, 31], 2, 2, 64, 128), ([65], [1400], 16, 1, 128, 64), ([40, 33, 90], [39, 3, 300], 8, 1, 64, 16)])
def test_prompt_chunks(q_lens, kv_lens, Hq, Hkv, D, page):
    check_attention(*problem(q_lens, kv_lens, Hq, Hkv, D, page, 15))


@pytest.mark.parametrize("q_len,Hq,Hkv,D", [(1, 48, 1, 128), (6, 8, 1, 64), (7, 7, 1, 128), (1, 49, 1, 64), (2, 64, 2, 128), (1, 100, 1, 128),
                                            (3, 100, 1, 64), (1, 256, 1, 64), (2, 255, 1, 128), (17, 3, 1, 128), (16, 3, 1, 64)])
def test_row_counts_around_the_kernels_limits(q_len, Hq, Hkv, D):
    check_attention(*problem([q_len, q_len], [333, q_len - 1], Hq, Hkv, D, 32, 24))


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page", [
    ([128], [128], 1, 1, 128, 16), ([49], [700], 1, 1, 64, 32), ([60, 7, 0, 33], [200, 0, 90, 1100], 8, 2, 128, 64),
    ([7, 7], [333, 6], 7, 1, 128, 32), ([1, 1], [333, 0], 100, 1, 128, 32), ([30, 17, 80], [29, 1000, 80], 12, 4, 64, 128),
    ([240], [1025], 1, 1, 64, 64)])
def test_little_work_on_wide_tables(q_lens, kv_lens, Hq, Hkv, D, page):
    # the table allows for more work than there is, so the kernel for larger calls takes it; its probabilities have
    # BF16's 8 bits there, rounded by up to 2^-8
    prob = list(problem(q_lens, kv_lens, Hq, Hkv, D, page, 34))
    check_attention(*prob)
    table = np.zeros((len(q_lens), 131072 // page), np.int32)
    table[:, :prob[7].shape[1]] = prob[7]
    prob[7] = table
    check_attention(*prob, p_extra=2.0 ** -9)


def test_many_short_requests():
    # more requests than a CTA has threads: several to a thread, in both kernels
    rng = np.random.default_rng(25)
    kv_lens = rng.integers(0, 40, 1500).tolist()
    check_attention(*problem([int(n > 0 or b % 3) for b, n in enumerate(kv_lens)], kv_lens, 2, 1, 64, 16, 26))
    kv_lens = rng.integers(0, 20, 700).tolist()
    check_attention(*problem(rng.integers(0, 4, 700).tolist(), kv_lens, 30, 1, 64, 16, 27))


@pytest.mark.parametrize("B,longest,q_len,Hq,Hkv,D,page", [
    (1, 700, 1, 8, 8, 128, 64), (1, 960, 1, 8, 8, 128, 64), (7, 1030, 1, 32, 8, 64, 32), (32, 500, 1, 8, 4, 128, 16),
    (33, 500, 1, 8, 4, 128, 16), (64, 900, 2, 16, 4, 64, 64), (100, 1990, 1, 16, 4, 64, 128), (20, 300, 5, 8, 2, 128, 16)])
def test_short_units_among_many(B, longest, q_len, Hq, Hkv, D, page):
    # units that are not cut, several to a thread block or one, and lengths around the limit from which they are
    kv_lens = np.random.default_rng(32).integers(0, longest + 1, B)
    kv_lens[-1], kv_lens[0] = longest, longest // 2 if B > 1 else longest
    check_attention(*problem([q_len] * B, kv_lens.tolist(), Hq, Hkv, D, page, 33))


def test_cut_units_of_long_chunks():
    check_attention(*problem([300], [5000], 4, 2, 128, 64, 28))
    check_attention(*problem([64, 1, 20], [3000, 4000, 30], 16, 2, 64, 16, 29))


def test_a_larger_bound_on_new_tokens_changes_the_kernel_only():
    prob = problem([1, 2, 0, 1], [500, 40, 9, 1200], 8, 2, 128, 32, 30)
    for max_q in (2, 12, 13, 300):
        check_attention(*prob, max_q=max_q)


def spread_gain(lo, hi):
    return lambda rng, shape: 2.0 ** rng.uniform(lo, hi, shape[:2] + (1,))


@pytest.mark.parametrize("q_lens,Hq", [([1, 1], 8), ([40, 3], 8)])
@pytest.mark.parametrize("q_gain,k_gain,v_gain,D", [
    (1e-3, spread_gain(-20, 8), spread_gain(-12, 12), 128),      # scales far apart from token to token
    (1e-30, spread_gain(90, 95), None, 64),                      # key blocks beyond every half-precision range
    (1e6, spread_gain(-25, -20), spread_gain(60, 62), 128),
    (3.0, None, spread_gain(-100, -99), 64),
    (40.0, None, None, 128),                                     # one key takes it all
])
def test_ranges(q_lens, Hq, q_gain, k_gain, v_gain, D):
    check_attention(*problem(q_lens, [300, 77], Hq, 2, D, 32, 16, q_gain, k_gain, v_gain))


def test_strided_queries_no_lse_own_stream_and_determinism():
    Hq, Hkv, D, page = 8, 2, 128, 32
    prob = problem([1, 3, 60], [700, 40, 333], Hq, Hkv, D, page, 17)
    q_bits, q_lens, kv_lens, _, _, _, _, table, cache, pages, _, scale = prob
    want, wl = check_attention(*prob)
    cu, lens, tab = i32(np.concatenate([[0], np.cumsum(q_lens)])), i32(kv_lens), i32(table)
    q = dev_bits(q_bits)
    wide = torch.full((q.shape[0], Hq + 4, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + Hq] = q
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = a4w4.a4w4_kv_attention_workspace_bytes(3, 60, Hq, Hkv, D)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(3):                                    # the same workspace, again and again
        out, _ = call_attention(wide[:, 2:2 + Hq], cu, lens, tab, cache, pages, page, Hq, Hkv, D, scale, 60, ws=ws, lse=False,
                                stream=s)
        assert a4w4.a4w4_get_device_status(s) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("q_lens,D", [([300, 9], 128), ([300, 9], 64), ([2, 1], 128)])
def test_output_on_16_bytes(q_lens, D):
    # rows that begin in the middle of a 32-byte sector
    Hq, Hkv, page = 4, 2, 32
    prob = problem(q_lens, [411, 200], Hq, Hkv, D, page, 35)
    q_bits, _, kv_lens, _, _, _, _, table, cache, pages, _, scale = prob
    want, _ = check_attention(*prob)
    buf = torch.full((want.numel() + 16,), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = buf[8:8 + want.numel()].view(want.shape)
    assert out.data_ptr() % 32 == 16
    cu = i32(np.concatenate([[0], np.cumsum(q_lens)]))
    call_attention(dev_bits(q_bits), cu, i32(kv_lens), i32(table), cache, pages, page, Hq, Hkv, D, scale, max(q_lens), out=out)
    ok()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert torch.isnan(buf[:8]).all() and torch.isnan(buf[8 + want.numel():]).all()


def test_one_workspace_serves_calls_of_other_sizes():
    probs = [problem([1] * 9, [2000 - 100 * b for b in range(9)], 16, 2, 128, 64, 18), problem([30], [900], 8, 1, 64, 16, 19),
             problem([1], [5000], 4, 1, 64, 16, 20)]
    sizes = [a4w4.a4w4_kv_attention_workspace_bytes(len(p[1]), max(p[1]), p[3], p[4], p[5]) for p in probs]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    alone = [check_attention(*p)[0] for p in probs]
    for _ in range(2):
        for p, want in zip(probs, alone):
            cu = i32(np.concatenate([[0], np.cumsum(p[1])]))
            out, _ = call_attention(dev_bits(p[0]), cu, i32(p[2]), i32(p[7]), p[8], p[9], p[6], p[3], p[4], p[5], p[11], max(p[1]), ws=ws)
            ok()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_rows_beyond_total_q_and_max_q_are_not_written():
    Hq, Hkv, D, page = 4, 2, 64, 16
    q_bits, q_lens, kv_lens, _, _, _, _, table, cache, pages, rows, scale = problem([3, 2], [40, 50], Hq, Hkv, D, page, 21)
    cu = i32([0, 3, 5])
    q = dev_bits(q_bits)
    out, lse = call_attention(q[:4], cu, i32(kv_lens), i32(table), cache, pages, page, Hq, Hkv, D, scale, 3)
    ok()
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()
    guard = torch.full((5, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    a4w4.a4w4_kv_attention(q, q.stride(0), cu, 2, 4, 3, i32(kv_lens), i32(table), table.shape[1], cache, pages, page, Hq, Hkv, D,
                           scale, guard, None, *workspace(2, 3, Hq, Hkv, D))
    ok()
    assert not torch.isnan(guard[:4]).any() and torch.isnan(guard[4]).all()


def workspace(B, max_q, Hq, Hkv, D):
    n = a4w4.a4w4_kv_attention_workspace_bytes(B, max_q, Hq, Hkv, D)
    return torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda"), max(n, 16)


def test_wild_lengths_and_pages_stay_inside_the_cache():
    # lengths beyond the table and page numbers outside the cache are clamped: the call ends and answers something finite
    Hq, Hkv, D, page = 8, 2, 128, 16
    q_bits, _, _, _, _, _, _, _, cache, pages, _, scale = problem([1, 1, 1], [16 * 9, 30, 5], Hq, Hkv, D, page, 22)
    cache = torch.zeros_like(cache)
    table = np.array([[0, -5, 1 << 30, 2], [1, 1, 1, 1], [7, 7, 7, 7]], np.int32)
    out, lse = call_attention(dev_bits(q_bits), i32([0, 1, 2, 3]), i32([1 << 30, -4, 3]), i32(table), cache, pages, page, Hq, Hkv, D,
                              scale, 1)
    ok()
    assert (out == 0).all()
    l = lse.cpu().numpy()
    assert np.allclose(l[0], np.log(64)) and np.isneginf(l[1]).all() and np.allclose(l[2], np.log(3))


def test_a_step_in_a_graph():
    """Plan, append and attention of one captured step, replayed with other lengths, equal the calls one by one."""
    B, Hq, Hkv, D, page, width = 3, 8, 2, 128, 16, 20
    pages = B * width
    rng = np.random.default_rng(23)
    qkv = torch.from_numpy(rng.standard_normal((B, Hq + 2 * Hkv, D)).astype(np.float32)).bfloat16().cuda()
    n = a4w4.a4w4_kv_cache_bytes(pages, page, Hkv, D)
    start = torch.from_numpy(rng.integers(0, 120, n).astype(np.uint8)).cuda()
    new = i32([1] * B)

    def buffers():
        e = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
        w, wn = workspace(B, 1, Hq, Hkv, D)
        return dict(past=e(B), table=i32(np.arange(pages).reshape(B, width)), ring=i32(np.arange(pages)), st=i32([0, pages]), so=e(2),
                    kv=e(B), cu=e(B + 1), sl=e(B), po=e(B), rf=e(1), cache=start.clone(), ws=w, wn=wn,
                    out=torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda"))

    def step(x):
        a4w4.a4w4_kv_plan(x["past"], new, B, page, x["table"], width, x["ring"], pages, x["st"], x["so"], x["kv"], x["cu"], x["sl"],
                          x["po"], B, x["rf"])
        k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        a4w4.a4w4_kv_append(k, k.stride(0), v, v.stride(0), x["sl"], B, Hkv, D, x["cache"], pages, page)
        a4w4.a4w4_kv_attention(qkv[:, :Hq], qkv.stride(0), x["cu"], B, B, 1, x["kv"], x["table"], width, x["cache"], pages, page, Hq,
                               Hkv, D, 0.1, x["out"], None, x["ws"], x["wn"])

    a, b = buffers(), buffers()
    step(a)
    ok()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    for past in ([0, 0, 0], [100, 15, 16], [318, 1, 200]):
        for x in (a, b):
            x["past"].copy_(i32(past))
            x["cache"].copy_(start)
        step(a)
        g.replay()
        ok()
        assert torch.equal(a["out"].view(torch.int16), b["out"].view(torch.int16))
        assert torch.equal(a["cache"], b["cache"])
