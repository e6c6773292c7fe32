"""One attention layer served with continuous batching, all of it in MXFP4.

Requests arrive with prompts of different lengths, decode token by token, finish
and give their pages back; every step is

    hidden -> fused QKV projection (a4w4_gemm_noalloc)
           -> a4w4_kv_plan       block tables, slots, positions; pages from a ring
           -> a4w4_kv_append     the new keys and values into the 4-bit cache
           -> a4w4_kv_attention  the new tokens' attention over what is cached
           -> output projection  (a4w4_gemm_noalloc)

Random weights and hidden states; no positional rotation.  Run it on a GB300:

    python examples/serve_attention.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_a4w4_gemm_gb300 as a4w4  # noqa: E402


def _ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


class AttentionLayer:
    """Prepared MXFP4 weights of the fused QKV and the output projection."""

    def __init__(self, hidden, Hq, Hkv, D, seed=0):
        self.hidden, self.Hq, self.Hkv, self.D = hidden, Hq, Hkv, D
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.qkv = self._prepare((Hq + 2 * Hkv) * D, hidden, g)
        self.out = self._prepare(hidden, Hq * D, g)

    @staticmethod
    def _prepare(N, K, g):
        w = (torch.randn(N, K, generator=g, device="cuda") * K ** -0.5).bfloat16()
        q = torch.empty(a4w4.a4w4_weight_codes_bytes(N, K), dtype=torch.uint8, device="cuda")
        s = torch.empty(a4w4.a4w4_weight_scales_bytes(N, K), dtype=torch.uint8, device="cuda")
        a4w4.a4w4_prepare_gemm_weight(w, N, K, q, s)
        return N, K, q, s

    @staticmethod
    def project(weight, x):
        N, K, q, s = weight
        y = torch.empty(x.shape[0], N, dtype=torch.bfloat16, device="cuda")
        a4w4.a4w4_gemm_noalloc(x, x.shape[0], K, q, s, N, y)
        return y


class Server:
    """The cache, its tables and the workspace of up to `batch` requests of up to `longest` tokens."""

    def __init__(self, layer, batch, longest, page=32, step_tokens=512):
        self.layer, self.batch, self.page, self.width = layer, batch, page, -(-longest // page)
        self.pages, self.step_tokens = batch * self.width, step_tokens
        n = a4w4.a4w4_kv_cache_bytes(self.pages, page, layer.Hkv, layer.D)
        self.cache = torch.zeros(n, dtype=torch.uint8, device="cuda")
        empty = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.ring = empty((batch, self.width)), torch.arange(self.pages, dtype=torch.int32, device="cuda")
        self.lens, self.next_lens = empty(batch), empty(batch)
        self.state, self.next_state = _ints([0, self.pages]), empty(2)
        self.cu, self.slots, self.positions, self.refused = empty(batch + 1), empty(step_tokens), empty(step_tokens), empty(1)
        n = max(a4w4.a4w4_kv_attention_workspace_bytes(batch, q, layer.Hq, layer.Hkv, layer.D) for q in (1, step_tokens))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        a4w4.a4w4_workspace_init(self.ws, n)

    def step(self, x, new):
        """x: the new tokens' hidden states, requests in order; new[b]: how many of request b (-1: finished).  Returns
        the layer's output for them."""
        L, T, most = self.layer, x.shape[0], max(1, max(new))
        a4w4.a4w4_kv_plan(self.lens, _ints(new), self.batch, self.page, self.table, self.width, self.ring, self.pages,
                          self.state, self.next_state, self.next_lens, self.cu, self.slots, self.positions,
                          self.step_tokens, self.refused)
        qkv = L.project(L.qkv, x).view(T, L.Hq + 2 * L.Hkv, L.D)
        q, k, v = qkv[:, :L.Hq], qkv[:, L.Hq:L.Hq + L.Hkv], qkv[:, L.Hq + L.Hkv:]
        a4w4.a4w4_kv_append(k, k.stride(0), v, v.stride(0), self.slots, T, L.Hkv, L.D, self.cache, self.pages, self.page)
        o = torch.zeros(T, L.Hq, L.D, dtype=torch.bfloat16, device="cuda")
        a4w4.a4w4_kv_attention(q, q.stride(0), self.cu, self.batch, T, most, self.next_lens, self.table, self.width,
                               self.cache, self.pages, self.page, L.Hq, L.Hkv, L.D, L.D ** -0.5, o, None, self.ws,
                               self.ws.numel())
        self.lens, self.next_lens = self.next_lens, self.lens
        self.state, self.next_state = self.next_state, self.state
        return L.project(L.out, o.view(T, L.Hq * L.D))


def main(hidden=1024, Hq=16, Hkv=4, D=128, steps=24, seed=1):
    layer = AttentionLayer(hidden, Hq, Hkv, D)
    server = Server(layer, batch=4, longest=400)
    g = torch.Generator(device="cuda").manual_seed(seed)
    arrivals = {0: [(0, 130)], 3: [(1, 33), (2, 1)], 10: [(3, 300)], 14: [(1, 64)]}
    leaves = {12: [1], 20: [0]}
    live = set()
    for t in range(steps):
        new = [1 if b in live else 0 for b in range(4)]
        for b in leaves.get(t, []):
            live.discard(b)
            new[b] = -1
        for b, prompt in arrivals.get(t, []):
            live.add(b)
            new[b] = prompt
        tokens = sum(n for n in new if n > 0)
        y = server.step(torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16(), new)
        if a4w4.a4w4_get_device_status() != 0 or int(server.refused) != 0 or not torch.isfinite(y).all():
            raise RuntimeError(f"step {t} failed")
        print(f"step {t:2d}: new {new}, cached {server.lens.tolist()}, free pages {int(server.state[1])}")
    return server


if __name__ == "__main__":
    main()
