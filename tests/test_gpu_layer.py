"""One decoder layer from the hidden state to the experts' sum, every call of the library that it takes, captured
once for a step's largest number of tokens and replayed for steps of any: each stage against the oracle, fed with what
the stage before it gave."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
import workloads
from gpu_util import dev_bits, host_bits
from oracle import gemm, kv, moe, mxfp4, rope, route, w8a8

pytestmark = pytest.mark.gpu

HID, HQ, HKV, D, PAGE, B, WIDTH, MOST = 512, 6, 2, 64, 16, 3, 8, 48
E, TOPK, I, GROUPS, TOP_GROUPS = 16, 4, 256, 4, 2
EPS = 1e-6
QKV = (HQ + 2 * HKV) * D


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def i32(*shape):
    return zeros(*shape, dtype=torch.int32)


class W8:
    def __init__(self, rng, n, k):
        self.n, self.k = n, k
        bits = workloads.to_bf16_bits((rng.standard_normal((n, k)) * 0.05).astype(np.float32))
        self.values, self.scales = w8a8.quant_weights(mxfp4.bf16_bits_to_f64(bits))
        self.W8, self.Ws = zeros(n * k, dtype=torch.uint8), zeros(n // 128, k // 128, dtype=torch.float32)
        a4w4.a4w4_prepare_w8_weight(dev_bits(bits), n, k, self.W8, self.Ws)
        self.ws_bytes = a4w4.a4w4_gemm_w8a8_workspace_bytes(MOST, n, k)
        self.ws = zeros(max(self.ws_bytes, 16), dtype=torch.uint8)

    def __call__(self, x, out):
        a4w4.a4w4_gemm_w8a8(x, MOST, self.k, self.W8, self.Ws, self.n, out, self.ws, self.ws_bytes)

    def check(self, x, out, n):
        c, reach = w8a8.gemm(mxfp4.bf16_bits_to_f64(host_bits(x[:n])), self.values, self.scales)
        assert np.all(np.abs(mxfp4.bf16_bits_to_f64(host_bits(out[:n])) - c) <= w8a8.bound(c, reach, self.k))


class Layer:
    def __init__(self):
        rng = np.random.default_rng(11)
        self.qkv_proj, self.o_proj = W8(rng, QKV, HID), W8(rng, HID, 384)
        self.wq, self.wk = ((1.0 + 0.1 * rng.standard_normal(D)).astype(np.float32) for _ in range(2))
        self.freq = (10000.0 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)
        self.bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
        self.gate = torch.from_numpy((0.2 * rng.standard_normal((E, HID))).astype(np.float32)).cuda()
        self.W1 = np.stack([workloads.moe_expert_weight_bits(e, 2 * I, HID) for e in range(E)])
        self.W2 = np.stack([workloads.moe_expert_weight_bits(e + 50, HID, I) for e in range(E)])
        u8 = lambda n: zeros(n, dtype=torch.uint8)  # noqa: E731
        self.W1q, self.W1s = u8(a4w4.a4w4_moe_w1_codes_bytes(E, 2 * I, HID)), u8(a4w4.a4w4_moe_w1_scales_bytes(E, 2 * I, HID))
        a4w4.a4w4_moe_prepare_w1(dev_bits(self.W1), E, 2 * I, HID, self.W1q, self.W1s)
        self.W2q, self.W2s = u8(a4w4.a4w4_weight_codes_bytes(E * HID, I)), u8(a4w4.a4w4_weight_scales_bytes(E * HID, I))
        a4w4.a4w4_prepare_gemm_weight(dev_bits(self.W2.reshape(E * HID, I)), E * HID, I, self.W2q, self.W2s)
        self.d = {k: torch.from_numpy(getattr(self, k)).cuda() for k in ("wq", "wk", "freq", "bias")}
        # a step's buffers
        pages = B * WIDTH
        self.past, self.new, self.table, self.ring = i32(B), i32(B), i32(B, WIDTH), torch.arange(pages, dtype=torch.int32, device="cuda")
        self.state, self.state_out = torch.tensor([0, pages], dtype=torch.int32, device="cuda"), i32(2)
        self.lens, self.cu, self.slots, self.pos, self.refused = i32(B), i32(B + 1), i32(MOST), i32(MOST), i32(1)
        self.cache = u8(a4w4.a4w4_kv_cache_bytes(pages, PAGE, HKV, D))
        self.hidden, self.qkv, self.q = zeros(MOST, HID), zeros(MOST, HQ + 2 * HKV, D), zeros(MOST, HQ, D)
        self.att, self.att_ws = zeros(MOST, HQ, D), u8(a4w4.a4w4_kv_attention_workspace_bytes(B, MOST, HQ, HKV, D))
        self.o, self.logits = zeros(MOST, HID), zeros(MOST, E, dtype=torch.float32)
        self.ids, self.w = i32(MOST, TOPK), zeros(MOST, TOPK, dtype=torch.float32)
        blocks = a4w4.a4w4_moe_max_blocks(MOST, TOPK, E, 128)
        self.rows, self.bexp, self.nb, self.tok, self.row_slot = i32(blocks * 128), i32(blocks), i32(1), i32(blocks * 128), i32(MOST * TOPK)
        self.sort_bytes = a4w4.a4w4_moe_sort_aux_workspace_bytes(MOST, TOPK, E)
        self.sort_ws = u8(self.sort_bytes)
        self.hq, self.hs = u8(a4w4.a4w4_moe_tiles_codes_bytes(MOST, TOPK, E, I)), u8(a4w4.a4w4_moe_tiles_scales_bytes(MOST, TOPK, E, I))
        self.g2_bytes = a4w4.a4w4_moe_gemm2_workspace_bytes(MOST, TOPK, HID)
        self.g2_ws, self.y = u8(self.g2_bytes), zeros(MOST, HID)

    def run(self):
        s, d = self, self.d
        a4w4.a4w4_kv_plan(s.past, s.new, B, PAGE, s.table, WIDTH, s.ring, B * WIDTH, s.state, s.state_out, s.lens, s.cu, s.slots,
                          s.pos, MOST, s.refused)
        s.qkv_proj(s.hidden, s.qkv)
        row = QKV
        a4w4.a4w4_kv_append_rope(s.qkv[:, :HQ], row, s.qkv[:, HQ: HQ + HKV], row, s.qkv[:, HQ + HKV:], row, s.pos, s.slots, MOST, HQ,
                                 HKV, D, d["wq"], d["wk"], EPS, d["freq"], D, 0, s.q, HQ * D, s.cache, B * WIDTH, PAGE)
        a4w4.a4w4_kv_attention(s.q, HQ * D, s.cu, B, MOST, MOST, s.lens, s.table, WIDTH, s.cache, B * WIDTH, PAGE, HQ, HKV, D,
                               D ** -0.5, s.att, None, s.att_ws, s.att_ws.numel())
        s.o_proj(s.att, s.o)
        torch.matmul(s.o.float(), s.gate.T, out=s.logits)           # (a program's own router)
        a4w4.a4w4_moe_route(s.logits, a4w4.A4W4_F32, E, s.cu[B:], MOST, E, a4w4.A4W4_MOE_SCORE_SIGMOID, d["bias"], GROUPS, 2, TOP_GROUPS,
                            TOPK, 1, 2.0, s.ids, s.w)
        a4w4.a4w4_moe_sort_aux(s.ids, MOST, TOPK, E, 128, s.rows, s.bexp, s.nb, s.tok, s.row_slot, s.sort_ws, s.sort_bytes)
        a4w4.a4w4_moe_gemm1_ex(s.o, MOST, HID, s.rows, s.bexp, s.nb, TOPK, s.W1q, s.W1s, E, I, a4w4.A4W4_MOE_ACT_SWIGLU,
                               a4w4.A4W4_MOE_OUT_TILES, s.hq, s.hs)
        a4w4.a4w4_moe_gemm2(s.hq, s.hs, MOST, I, s.rows, s.bexp, s.nb, TOPK, s.w, s.W2q, s.W2s, E, HID, s.y, s.g2_ws, s.g2_bytes)

    def check(self, keys, values):
        """keys, values: per request the oracle's cached rows so far [len, HKV, D]; they grow by this step's."""
        assert a4w4.a4w4_get_device_status() == 0
        cu, pos = self.cu.cpu().numpy(), self.pos.cpu().numpy()
        n = int(cu[-1])
        assert n == int(self.new.sum()) and int(self.refused) == 0
        f64 = lambda x: mxfp4.bf16_bits_to_f64(host_bits(x))  # noqa: E731
        self.qkv_proj.check(self.hidden, self.qkv.view(MOST, QKV), n)
        x = f64(self.qkv)[:n]
        q, reach = rope.heads(x[:, :HQ], self.wq, EPS, pos[:n], self.freq, D, 0)
        got = f64(self.q)
        assert np.all(np.abs(got[:n] - q) <= rope.bound(q, reach)) and np.all(got[n:] == 7.0)
        k, _ = rope.heads(x[:, HQ: HQ + HKV], self.wk, EPS, pos[:n], self.freq, D, 0)
        cells = [mxfp4.quant_dequant(y.reshape(-1, D)).reshape(n, HKV, D) for y in (k, x[:, HQ + HKV:])]
        att = f64(self.att)
        for b in range(B):
            keys[b] = np.concatenate([keys[b], cells[0][cu[b]: cu[b + 1]]])
            values[b] = np.concatenate([values[b], cells[1][cu[b]: cu[b + 1]]])
            if cu[b + 1] > cu[b]:
                out, lse, spread, reach = kv.attention(got[cu[b]: cu[b + 1]], keys[b], values[b], D ** -0.5)
                bound, _ = kv.attention_bounds(out, lse, spread, reach, kv.P_ONE_BF16)
                assert np.all(np.abs(att[cu[b]: cu[b + 1]] - out) <= bound)
        self.o_proj.check(self.att.view(MOST, HQ * D), self.o, n)
        logits, ids, w = self.logits.cpu().numpy(), self.ids.cpu().numpy(), self.w.cpu().numpy()
        for t in range(n):
            want, weights = route.route(logits[t], False, self.bias, GROUPS, 2, TOP_GROUPS, TOPK, True, 2.0)
            assert ids[t].tolist() == want and np.all(np.abs(w[t] - weights) <= 2.0 ** -20 * weights)
        assert np.all(ids[n:] == -1) and np.all(w[n:] == 0.0)
        rows, _, blocks = moe.sort_routed_rows(ids[:n], E, 128)
        assert int(self.nb) == blocks
        listed = self.rows.cpu().numpy()[: blocks * 128]
        assert np.array_equal(np.where(listed < n * TOPK, listed, n * TOPK), rows)
        # the experts, from the oracle's own first stage: the product's tolerance and, in relative terms, a few codes of the
        # requantisation that lie at their borders
        o = host_bits(self.o)[:n]
        first = moe.gemm1_rows(o, ids[:n], lambda e: self.W1[e], np.arange(n * TOPK), I)
        y, spread = moe.gemm2_tokens(first["codes"], first["scales"], ids[:n], w[:n].astype(np.float64), lambda e: self.W2[e], np.arange(n))[:2]
        off = f64(self.y)[:n] - y
        assert np.linalg.norm(off) <= 0.01 * np.linalg.norm(y)


def test_steps_of_any_size_through_one_graph():
    s = Layer()
    stream = torch.cuda.Stream()
    rng = np.random.default_rng(3)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):                                 # library and router warm up outside the capture
        s.run()
    torch.cuda.synchronize()
    assert a4w4.a4w4_get_device_status() == 0
    s.ring.copy_(torch.arange(B * WIDTH))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    keys, values = ([np.zeros((0, HKV, D)) for _ in range(B)] for _ in range(2))
    past = np.zeros(B, np.int32)
    # prompts, a step of single tokens, drafts, an idle request, a lone token
    for new in ([20, 3, 17], [1, 1, 1], [5, 0, 4], [0, 1, 0], [16, 16, 16]):
        n = sum(new)
        s.hidden.copy_(workloads.bits_to_torch(workloads.to_bf16_bits(rng.standard_normal((MOST, HID)).astype(np.float32))))
        s.past.copy_(torch.from_numpy(past))
        s.new.copy_(torch.tensor(new, dtype=torch.int32))
        s.q.fill_(7.0)
        graph.replay()
        s.check(keys, values)
        past = past + np.array(new, np.int32)
        s.state.copy_(s.state_out)
        assert n == int(s.cu[-1])
