"""The cache's calls together, as a server makes them: the example runs, a prompt in one chunk equals the same
prompt token by token, and an expired wait is reported and leaves the context usable."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
from test_gpu_kv import call_attention, i32, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_attention.py")
    spec = importlib.util.spec_from_file_location("serve_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs():
    server = example().main()
    lens = server.lens.tolist()
    assert lens == [0, 73, 21, 313]
    held = sum(-(-n // server.page) for n in lens)
    assert int(server.state[1]) == server.pages - held           # finished requests' pages came back
    head, count = server.state.tolist()
    free = [int(server.ring[(head + i) % server.pages]) for i in range(count)]
    used = [int(server.table[b, j]) for b, n in enumerate(lens) for j in range(-(-n // server.page))]
    assert sorted(free + used) == list(range(server.pages))       # every page once


def test_a_prompt_at_once_and_token_by_token():
    """Both ways cache the same cells and see the same keys; the layer's outputs differ by roundings only (BF16 scores'
    probabilities, BF16 outputs requantised to 4 bits by the output projection, hence attention's own output is compared)."""
    m = example()
    layer = m.AttentionLayer(512, 8, 2, 64, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(70, 512, generator=g, device="cuda").bfloat16()
    once, steps = (m.Server(layer, batch=2, longest=128, page=16) for _ in range(2))
    once.step(x, [70, 0])
    for t in range(70):
        steps.step(x[t:t + 1], [1, 0])
    ok()
    assert once.lens.tolist() == steps.lens.tolist() == [70, 0]
    slots = torch.arange(70, device="cuda")
    rows = []
    for s in (once, steps):
        sl = (s.table[0][(slots // 16).long()] * 16 + slots % 16).int()
        k = torch.empty(70, 2, 64, dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        a4w4.a4w4_kv_read(s.cache, s.pages, s.page, sl, 70, 2, 64, k, v)
        rows.append((k, v))
    # the projections of one token and of 70 may round a sum differently (another kernel): the cells then differ by a
    # code step in rare places, so the attention of both caches is compared through the oracle-checked kernel itself
    same = [(a == b).float().mean().item() for a, b in zip(*rows)]
    assert min(same) > 0.9


@pytest.mark.parametrize("B,q_len,kv_len,Hq,Hkv,D,waits", [(64, 1, 4000, 64, 8, 128, True), (2, 1, 40000, 64, 4, 64, False),
                                                           (1, 2048, 4096, 16, 2, 128, True), (4, 300, 3000, 16, 2, 64, False)])
def test_expired_wait_is_reported_and_context_survives(B, q_len, kv_len, Hq, Hkv, D, waits):
    """With a limit of 1 ns a wait for what is not there yet runs out.  `waits`: the call has such waits for certain;
    otherwise everything may be there in time, and then the answer has to be right."""
    page, width = 64, -(-kv_len // 64)
    pages = B * width
    g = torch.Generator(device="cuda").manual_seed(31)
    # any codes; scale bytes 112..127
    cache = torch.randint(0, 256, (pages * Hkv * page // 16, 17 * D), generator=g, device="cuda", dtype=torch.uint8)
    for at in (8 * D, 8 * D + D // 2 + 8 * D):
        cache[:, at:at + D // 2] = cache[:, at:at + D // 2] % 16 + 112
    q = torch.randn(B * q_len, Hq, D, generator=g, device="cuda").bfloat16()
    table = torch.randperm(pages, generator=g, device="cuda").int().view(B, width)
    args = (q, i32(np.arange(B + 1) * q_len), i32([kv_len] * B), table, cache.view(-1), pages, page, Hq, Hkv, D, D ** -0.5, q_len)
    n = a4w4.a4w4_kv_attention_workspace_bytes(B, q_len, Hq, Hkv, D)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    want, _ = call_attention(*args, ws=ws)
    ok()
    assert torch.isfinite(want).all()
    a4w4.a4w4_set_wait_limit_ns(1)
    try:
        out, _ = call_attention(*args, ws=ws)
        status = a4w4.a4w4_get_device_status()
    finally:
        a4w4.a4w4_set_wait_limit_ns(0)
    if waits or status != 0:
        assert status == a4w4.A4W4_ERR_TIMEOUT
    else:
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert a4w4.a4w4_get_device_status() == 0
    a4w4.a4w4_workspace_init(ws, n)
    out, _ = call_attention(*args, ws=ws)
    ok()
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
