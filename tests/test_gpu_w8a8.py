"""GPU parity of the 8-bit product (a4w4_gemm_w8a8) and its weights' preparation against the oracle."""

import numpy as np
import pytest
import torch

import mxfp4_a4w4_gemm_gb300 as a4w4
import workloads
from gpu_util import dev_bits, host_bits
from oracle import mxfp4, w8a8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mxfp4_a4w4_gemm_gb300 import build
    build.build()
    a4w4.lib()


def problem(M, N, K, seed=0):
    rng = np.random.default_rng(seed + M + N + K)
    a = rng.standard_normal((M, K)).astype(np.float32)
    a[:, rng.integers(0, K, max(1, K // 100))] *= 20.0
    w = w8a8.e4m3(rng.standard_normal((N, K)) * np.exp2(rng.integers(-3, 7, (N, K))))
    ws = np.exp2(rng.uniform(-12, -4, (N // 128, K // 128))).astype(np.float32)
    return workloads.to_bf16_bits(a), w, ws


class Product:
    def __init__(self, a_bits, w, ws):
        self.a_bits, self.w, self.ws = a_bits, w, ws
        (self.M, self.K), self.N = a_bits.shape, w.shape[0]
        self.A = dev_bits(a_bits)
        codes = torch.from_numpy(w8a8.encode(w)).cuda()
        self.W8 = torch.empty(a4w4.a4w4_w8_weight_bytes(self.N, self.K), dtype=torch.uint8, device="cuda")
        a4w4.a4w4_shuffle_w8_weight(codes, self.N, self.K, self.W8)
        self.Ws = torch.from_numpy(ws).cuda()
        self.bytes = a4w4.a4w4_gemm_w8a8_workspace_bytes(self.M, self.N, self.K)
        self.work = torch.full((self.bytes + 64,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN wherever it is not written
        self.C = torch.full((self.M + 3, self.N), 7.0, dtype=torch.bfloat16, device="cuda")

    def run(self, flags=0, stream=None, C=None):
        a4w4.a4w4_gemm_w8a8(self.A, self.M, self.K, self.W8, self.Ws, self.N, self.C if C is None else C, self.work, self.bytes,
                            flags, stream)

    def check(self):
        assert a4w4.a4w4_get_device_status() == 0
        a = mxfp4.bf16_bits_to_f64(self.a_bits)
        c, reach = w8a8.gemm(a, self.w, self.ws)
        got = mxfp4.bf16_bits_to_f64(host_bits(self.C))
        assert np.all(got[self.M:] == 7.0)                          # rows behind the last are left
        bad = ~(np.abs(got[:self.M] - c) <= w8a8.bound(c, reach, self.K))
        assert not bad.any(), (bad.sum(), np.argwhere(bad)[:5])


# every plan: one and two tiles of few tokens, K whole and cut into up to 16 parts, narrow, odd and wide tiles of many
SIZES = [(1, 128, 128), (1, 256, 2176), (3, 384, 640), (16, 128, 4224), (17, 256, 1152), (32, 1536, 896), (31, 640, 7168),
         (33, 128, 128), (33, 128, 1024), (100, 384, 640), (127, 256, 128), (128, 640, 1152), (129, 1536, 256), (257, 128, 4224),
         (513, 1536, 512), (300, 8448, 384), (1100, 2304, 256),
         (33, 384, 4224), (64, 1536, 2176), (97, 256, 4224), (500, 128, 7168), (1024, 128, 9088),    # tiles of 32 tokens, ragged
         (1100, 384, 2304), (1025, 640, 4224), (650, 1536, 4224), (160, 19456, 1152)]               # tiles of 128, long sums


@pytest.mark.parametrize("M,N,K", SIZES, ids=lambda v: str(v))
def test_matches_the_oracle(M, N, K):
    p = Product(*problem(M, N, K))
    p.run()
    p.check()


def test_several_waves_of_tiles():
    p = Product(*problem(2500, 2432, 128))                          # 20 x 9 wide tiles, the last wave's as halves, and narrow ones
    p.run()
    p.check()


@pytest.mark.parametrize("M", [5, 70])
def test_runs_again_bit_for_bit_and_with_weights_ahead(M):
    p = Product(*problem(M, 512, 2304))
    p.run()
    first = p.C.clone()
    for flags in (0, a4w4.A4W4_GEMM_WEIGHT_PREFETCH):
        p.C.fill_(7.0)
        p.work.fill_(0xFF)
        p.run(flags)
        assert torch.equal(p.C.view(torch.int16), first.view(torch.int16))
    p.check()


@pytest.mark.parametrize("M", [4, 90])
def test_blocks_of_zeros_tiny_and_huge_values(M):
    a_bits, w, ws = problem(M, 256, 768)
    a = mxfp4.bf16_bits_to_f64(a_bits)
    a[0] = 0.0
    a[1, :128] = 0.0
    a[1, 128:256] *= 2.0 ** -120
    a[2, 256:384] *= 2.0 ** 60
    a[3, ::128] = 448.0                                             # a scale's border: 448 takes 2^0, a step more 2^1
    a[3, 1::128] = 450.0 if M > 4 else 447.0
    w[:128, 128:256] = 0.0
    p = Product(workloads.to_bf16_bits(a.astype(np.float32)), w, ws)
    p.run()
    p.check()


@pytest.mark.parametrize("M", [6, 40])
def test_infinities_and_nan_stay_in_their_rows(M):
    a_bits, w, ws = problem(M, 384, 512)
    clean = Product(a_bits, w, ws)
    clean.run()
    a_bits = a_bits.copy()
    a_bits[2, 7], a_bits[4, 500] = 0x7F80, 0x7FC1                   # +infinity, NaN
    p = Product(a_bits, w, ws)
    p.run()
    assert a4w4.a4w4_get_device_status() == 0
    for m in range(M):
        if m in (2, 4):
            assert torch.isnan(p.C[m]).all()
        else:
            assert torch.equal(p.C[m].view(torch.int16), clean.C[m].view(torch.int16))


@pytest.mark.parametrize("N,K", [(128, 128), (384, 640)])
def test_prepared_weights(N, K):
    rng = np.random.default_rng(N)
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    w[:, 5] *= 30.0
    if N > 128:
        w[128:256, 128:256] = 0.0
    bits = workloads.to_bf16_bits(w)
    values, scales = w8a8.quant_weights(mxfp4.bf16_bits_to_f64(bits))
    W8 = torch.empty(N * K, dtype=torch.uint8, device="cuda")
    Ws = torch.empty(N // 128, K // 128, dtype=torch.float32, device="cuda")
    a4w4.a4w4_prepare_w8_weight(dev_bits(bits), N, K, W8, Ws)
    assert np.array_equal(Ws.cpu().numpy(), scales)
    got = w8a8.decode(W8.cpu().numpy())
    assert np.array_equal(got, w8a8.decode(w8a8.tiles(w8a8.encode(values))))


def test_shuffled_weights_are_the_checkpoints_bytes():
    codes = np.random.default_rng(3).integers(0, 256, (384, 256)).astype(np.uint8)
    W8 = torch.empty(384 * 256, dtype=torch.uint8, device="cuda")
    a4w4.a4w4_shuffle_w8_weight(torch.from_numpy(codes).cuda(), 384, 256, W8)
    assert np.array_equal(W8.cpu().numpy(), w8a8.tiles(codes))


@pytest.mark.parametrize("M", [8, 200])
def test_two_streams_and_a_captured_graph(M):
    p, q = Product(*problem(M, 256, 1152)), Product(*problem(M, 256, 1152, seed=5))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        p.run(stream=a)
        q.run(stream=b)
    torch.cuda.synchronize()
    p.check()
    q.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=a):
        p.run()
        q.run()
    p.C.fill_(7.0)
    q.C.fill_(7.0)
    p.A.copy_(q.A)
    p.a_bits = q.a_bits
    g.replay()
    g.replay()
    p.check()
    q.check()


def test_workspace_is_asked_for():
    p = Product(*problem(200, 128, 256))
    for work, size in ((None, 0), (p.work, p.bytes - 1), (p.work.data_ptr() + 8, p.bytes)):
        with pytest.raises(a4w4.A4W4Error) as e:
            a4w4.a4w4_gemm_w8a8(p.A, p.M, p.K, p.W8, p.Ws, p.N, p.C, work, size)
        assert e.value.code == a4w4.A4W4_ERR_WORKSPACE


@pytest.mark.parametrize("M,N,K", [(8, 1536, 7168), (20, 256, 2304), (300, 640, 4224), (700, 5120, 1152)])
def test_expired_wait_is_reported_and_the_next_call_is_right(M, N, K):
    p = Product(*problem(M, N, K))
    torch.cuda.synchronize()
    a4w4.a4w4_set_wait_limit_ns(1)
    try:
        p.run()
        status = a4w4.a4w4_get_device_status()
    finally:
        a4w4.a4w4_set_wait_limit_ns(0)
    assert status == a4w4.A4W4_ERR_TIMEOUT
    assert a4w4.a4w4_get_device_status() == 0
    p.C.fill_(7.0)
    p.run()
    p.check()


@pytest.mark.parametrize("M", [2, 40])
def test_weights_beyond_31_bits_of_bytes(M):
    N, K = 131072, 16512
    free, _ = torch.cuda.mem_get_info()
    if free < 6 * N * K:
        pytest.skip("not enough memory")
    g = torch.Generator(device="cuda").manual_seed(M)
    codes = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda", generator=g)     # up to 240
    codes[:, 1::2] += 128
    a_bits, _, _ = problem(M, 128, K)
    ws = np.exp2(np.random.default_rng(M).uniform(-12, -4, (N // 128, K // 128))).astype(np.float32)
    W8 = torch.empty(N * K, dtype=torch.uint8, device="cuda")
    a4w4.a4w4_shuffle_w8_weight(codes, N, K, W8)
    Ws, A = torch.from_numpy(ws).cuda(), dev_bits(a_bits)
    work = torch.empty(a4w4.a4w4_gemm_w8a8_workspace_bytes(M, N, K) + 16, dtype=torch.uint8, device="cuda")
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    a4w4.a4w4_gemm_w8a8(A, M, K, W8, Ws, N, C, work, work.numel())
    assert a4w4.a4w4_get_device_status() == 0
    a = mxfp4.bf16_bits_to_f64(a_bits)
    for n0 in (0, 1015 * 128, 1016 * 128, N - 128):                    # byte 2^31 lies in row tile 1016 of 1024
        rows = slice(n0, n0 + 128)
        c, reach = w8a8.gemm(a, w8a8.decode(codes[rows].cpu().numpy()), ws[n0 // 128:n0 // 128 + 1])
        got = mxfp4.bf16_bits_to_f64(host_bits(C[:, rows].contiguous()))
        assert np.all(np.abs(got - c) <= w8a8.bound(c, reach, K))
