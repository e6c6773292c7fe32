"""Attention's two kernels, each made to run whatever the rules between them say: a bound on new tokens of 256 sends any
call to the kernel for many rows (`PROMPT`), short drafts on their own run in the kernel for few."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
from gpu_util import dev_bits, host_bits
from oracle import kv, mxfp4
from test_gpu_kv import call_attention, check_attention, i32, ok, problem, spread_gain

pytestmark = pytest.mark.gpu

PROMPT = 256


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


# ---------------------------------------------------------------------------
# the kernel for many rows, at what is out of the ordinary

@pytest.mark.parametrize("q_lens", [[1, 1], [40, 3]])
@pytest.mark.parametrize("q_gain,k_gain,v_gain,D", [
    (1e-3, spread_gain(-20, 8), spread_gain(-12, 12), 128),      # scales far apart from token to token
    (1e-30, spread_gain(90, 95), None, 64),                      # key blocks beyond every half-precision range
    (1e6, spread_gain(-25, -20), spread_gain(60, 62), 128),      # value scales above 127
    (3.0, None, spread_gain(-100, -99), 64),
    (40.0, None, None, 128),                                     # one key takes it all
    (1.0, None, lambda rng, s: 2.0 ** rng.choice([-20.0, 0.0, 20.0], s[:2] + (1,)), 128),     # on both sides of 127 in one step
    (1.0, None, lambda rng, s: np.where(np.arange(s[2]) // 32 % 2, 0.0, 2.0 ** 9), 64),       # scale byte 0 beside scales above 127
    (1.0, None, lambda rng, s: np.where(np.arange(s[2]) // 32 % 2, 0.0, 2.0 ** 9), 128),
])
def test_prompt_kernel_ranges(q_lens, q_gain, k_gain, v_gain, D):
    check_attention(*problem(q_lens, [300, 77], 8, 2, D, 32, 36, q_gain, k_gain, v_gain), max_q=PROMPT)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (24, 1, 64), (32, 1, 128), (255, 1, 64)])
def test_prompt_kernel_empty_requests_idle_rows_and_more_queries_than_keys(Hq, Hkv, D):
    check_attention(*problem([1, 0, 3, 4, 1, 0, 2], [0, 50, 2, 0, 17, 0, 2], Hq, Hkv, D, 16, 37), max_q=PROMPT)
    check_attention(*problem([0, 0, 1], [0, 0, 1], Hq, Hkv, D, 16, 38), max_q=PROMPT)


@pytest.mark.parametrize("B,longest,most,Hq,Hkv,D", [(33, 300, 5, 8, 2, 128), (700, 20, 4, 30, 1, 64), (1500, 40, 2, 2, 1, 64)])
def test_prompt_kernel_many_requests(B, longest, most, Hq, Hkv, D):
    # more than a warp has lanes; more than the kernel has threads
    rng = np.random.default_rng(39)
    kv_lens = rng.integers(0, longest, B).tolist()
    check_attention(*problem(rng.integers(0, most, B).tolist(), kv_lens, Hq, Hkv, D, 16, 40), max_q=PROMPT)


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_kernel_strided_queries_and_own_stream(D):
    Hq, Hkv, page = 8, 2, 32
    prob = problem([1, 3, 60], [700, 40, 333], Hq, Hkv, D, page, 41)
    q_bits, q_lens, kv_lens, _, _, _, _, table, cache, pages, _, scale = prob
    want, _ = check_attention(*prob, max_q=PROMPT)
    cu, lens, tab = i32(np.concatenate([[0], np.cumsum(q_lens)])), i32(kv_lens), i32(table)
    q = dev_bits(q_bits)
    wide = torch.full((q.shape[0], Hq + 4, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + Hq] = q
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.zeros(a4w4.a4w4_kv_attention_workspace_bytes(3, PROMPT, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out, _ = call_attention(wide[:, 2:2 + Hq], cu, lens, tab, cache, pages, page, Hq, Hkv, D, scale, PROMPT, ws=ws, lse=False,
                                stream=s)
        assert a4w4.a4w4_get_device_status(s) == 0
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_both_kernels_share_a_workspace_in_turn():
    few = [problem([1] * 9, [2000 - 100 * b for b in range(9)], 16, 2, 128, 64, 42), problem([1], [5000], 4, 1, 64, 16, 43)]
    many = [problem([30], [900], 8, 1, 64, 16, 44), problem([300, 1], [2500, 4000], 4, 2, 128, 64, 45)]
    calls = [(few[0], 1), (many[0], PROMPT), (few[1], 1), (many[1], 300)]
    n = max(a4w4.a4w4_kv_attention_workspace_bytes(len(p[1]), most, p[3], p[4], p[5]) for p, most in calls)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    alone = [check_attention(*p, max_q=most)[0] for p, most in calls]
    for _ in range(2):
        for (p, most), want in zip(calls, alone):
            cu = i32(np.concatenate([[0], np.cumsum(p[1])]))
            out, _ = call_attention(dev_bits(p[0]), cu, i32(p[2]), i32(p[7]), p[8], p[9], p[6], p[3], p[4], p[5], p[11], most, ws=ws)
            ok()
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))


# ---------------------------------------------------------------------------
# lengths that the floors are given for

def rows_problem(kv_len, Hkv, D, page, seed):
    """A request of one long context with any codes and moderate scales; returns the cache, its table and the values."""
    rng = np.random.default_rng(seed)
    pages = -(-kv_len // page)
    n = pages * page
    codes = [rng.integers(0, 16, (n, Hkv, D), dtype=np.uint8) for _ in range(2)]
    scales = [rng.integers(122, 127, (n, Hkv, D // 32), dtype=np.uint8) for _ in range(2)]
    cache = torch.from_numpy(kv.cache_from_rows(codes[0], scales[0], codes[1], scales[1], page))
    table = rng.permutation(pages).astype(np.int32)[None]
    slot = table[0, np.arange(kv_len) // page] * page + np.arange(kv_len) % page
    keys, vals = (mxfp4.decode(c[slot], e[slot]) for c, e in zip(codes, scales))
    return cache.cuda(), pages, table, keys, vals


@pytest.mark.parametrize("q_len,kv_len,Hq,Hkv,D,page,rows", [
    (1, 131000, 16, 1, 128, 128, [0]), (3, 70001, 8, 2, 64, 16, [0, 2]), (4096, 16384, 4, 1, 128, 64, [0, 1, 255, 256, 2049, 4095]),
    (1000, 30011, 4, 2, 64, 32, [0, 511, 999])])
def test_long_contexts_row_by_row(q_len, kv_len, Hq, Hkv, D, page, rows):
    """A few rows of a call of full length against the oracle.  P's rounding is one BF16 term's at most, the sums over the
    keys are off by 2^-24 each."""
    cache, pages, table, keys, vals = rows_problem(kv_len, Hkv, D, page, 46)
    g = torch.Generator(device="cuda").manual_seed(47)
    q = torch.randn(q_len, Hq, D, generator=g, device="cuda").bfloat16()
    scale = float(np.float32(D ** -0.5))
    out, lse = call_attention(q, i32([0, q_len]), i32([kv_len]), i32(table), cache, pages, page, Hq, Hkv, D, scale, q_len)
    ok()
    got, gl, qf = mxfp4.bf16_bits_to_f64(host_bits(out)), lse.cpu().numpy().astype(np.float64), q.float().cpu().numpy().astype(np.float64)
    for i in rows:
        seen = kv_len - q_len + i + 1
        o, l, spread, reach = kv.attention(qf[i:i + 1], keys[:seen], vals[:seen], scale)
        bo, bl = kv.attention_bounds(o, l, spread, reach, p_round=kv.P_ONE_BF16)
        assert np.all(np.abs(got[i:i + 1] - o) <= bo + seen * 2.0 ** -24 * spread), i
        assert np.all(np.abs(gl[i:i + 1] - l) <= bl + seen * 2.0 ** -24), i


# ---------------------------------------------------------------------------
# the same tokens by other ways

@pytest.mark.parametrize("Hq,Hkv,D,page,max_q", [(4, 2, 64, 16, 70), (4, 2, 64, 16, PROMPT), (8, 1, 128, 32, PROMPT), (3, 3, 128, 16, 70)])
def test_attention_of_a_prompt_at_once_and_token_by_token(Hq, Hkv, D, page, max_q):
    """One cache: 70 rows in one call, and row after row with the length that the row sees.  Outputs and log-sums agree to
    within the two calls' bounds."""
    n = 70
    q_bits, _, _, _, _, _, _, table, cache, pages, vals, scale = problem([n], [n], Hq, Hkv, D, page, 48)
    q, tab = dev_bits(q_bits), i32(table)
    out, lse = call_attention(q, i32([0, n]), i32([n]), tab, cache, pages, page, Hq, Hkv, D, scale, max_q)
    one = [call_attention(q[t:t + 1], i32([0, 1]), i32([t + 1]), tab, cache, pages, page, Hq, Hkv, D, scale, 1) for t in range(n)]
    ok()
    o, l, spread, reach = kv.attention(mxfp4.bf16_bits_to_f64(q_bits), vals[0][0], vals[0][1], float(np.float32(scale)))
    few, many = (kv.attention_bounds(o, l, spread, reach, p_round=r) for r in (kv.P_FP16, kv.P_ONE_BF16))
    got, gl = mxfp4.bf16_bits_to_f64(host_bits(out)), lse.cpu().numpy().astype(np.float64)
    steps = np.concatenate([mxfp4.bf16_bits_to_f64(host_bits(x)) for x, _ in one])
    sl = np.concatenate([x.cpu().numpy().astype(np.float64) for _, x in one])
    assert np.all(np.abs(got - steps) <= few[0] + many[0]) and np.all(np.abs(gl - sl) <= few[1] + many[1])
    # a row that saw another number of keys would differ by more than that in most of its elements
    shifted = np.abs(got[1:] - steps[:-1]) > (few[0] + many[0])[1:]
    assert shifted.mean() > 0.5


def test_the_example_answers_what_its_cells_say(monkeypatch):
    """Every attention call of the serving example against the oracle, over the cells read back by way of the table."""
    from test_gpu_kv_serving import example
    calls = []
    run = a4w4.a4w4_kv_attention

    def checked(q, q_stride, cu_q, B, total_q, max_q, kv_lens, table, width, cache, pages, page, Hq, Hkv, D, scale, out, lse, ws, n):
        run(q, q_stride, cu_q, B, total_q, max_q, kv_lens, table, width, cache, pages, page, Hq, Hkv, D, scale, out, lse, ws, n)
        ok()
        got, qf = mxfp4.bf16_bits_to_f64(host_bits(out)), mxfp4.bf16_bits_to_f64(host_bits(q))
        cu, lens = cu_q.tolist(), kv_lens.tolist()
        assert cu[-1] == total_q
        for b in range(B):
            if cu[b] == cu[b + 1]:
                continue
            tok = torch.arange(lens[b], device="cuda")
            slots = (table[b][(tok // page).long()] * page + tok % page).int()
            k = torch.empty(lens[b], Hkv, D, dtype=torch.bfloat16, device="cuda")
            v = torch.empty_like(k)
            a4w4.a4w4_kv_read(cache, pages, page, slots, lens[b], Hkv, D, k, v)
            ok()
            rows = slice(cu[b], cu[b + 1])
            o, l, spread, reach = kv.attention(qf[rows], *(mxfp4.bf16_bits_to_f64(host_bits(x)) for x in (k, v)), float(np.float32(scale)))
            bo, _ = kv.attention_bounds(o, l, spread, reach, p_round=kv.P_ONE_BF16)
            assert np.all(np.abs(got[rows] - o) <= bo), b
            calls.append(cu[b + 1] - cu[b])

    monkeypatch.setattr(a4w4, "a4w4_kv_attention", checked)
    example().main()
    assert sorted(set(calls)) == [1, 33, 64, 130, 300]
