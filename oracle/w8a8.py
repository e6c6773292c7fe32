"""Oracle of the 8-bit product with a scale for each block of 128 (a4w4_gemm_w8a8 of
include/a4w4.h, restated from that header's text): E4M3 rounding, both quantisers,
the weight tiles' bytes, the product in float64.
"""

import numpy as np


def e4m3(y):
    """float64 -> the nearest E4M3 value, ties to even, saturating at 448.  E4M3: three bits behind the leading one,
    exponents from -6; below 2^-6 steps of 2^-9."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    step = np.exp2(np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6.0) - 3.0)
    return np.copysign(np.minimum(np.round(a / step) * step, 448.0), y)      # np.round takes ties to even


def decode(codes):
    """E4M3 code bytes -> float64 (S.1111.111 is NaN; there are no infinities)."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    return np.where((c & 127) == 127, np.nan, np.where(c >> 7, -v, v))


def encode(values):
    """E4M3 values (as e4m3 gives them) -> code bytes."""
    table = decode(np.arange(127))
    i = np.searchsorted(table, np.abs(values))
    assert np.array_equal(table[i], np.abs(values))
    return (i + 128 * np.signbit(values)).astype(np.uint8)


def quant_activations(a):
    """float64 [M, K] -> (E4M3 values [M, K], scales [M, K/128]): 2^e with the smallest e >= -126 such that the block's
    largest magnitude is at most 448 * 2^e; NaN where the block holds an infinity or NaN."""
    M, K = a.shape
    b = a.reshape(M, K // 128, 128)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(top)
    e = np.full(top.shape, -126)
    t = np.where(bad, 0.0, top)
    while np.any(t > 448.0 * np.exp2(e)):
        e = np.where(t > 448.0 * np.exp2(e), e + 1, e)
    unit = np.exp2(e.astype(np.float64))
    with np.errstate(invalid="ignore"):
        q = e4m3(np.where(bad[..., None], 0.0, b / unit[..., None]))
    return q.reshape(M, K), np.where(bad, np.nan, unit)


def quant_weights(w):
    """float32 [N, K] -> (E4M3 values, float32 scales [N/128, K/128]): largest magnitude / 448, w / scale, both rounded to
    fp32 and the latter then to E4M3."""
    N, K = w.shape
    b = np.asarray(w, dtype=np.float32).reshape(N // 128, 128, K // 128, 128)
    s = (np.abs(b).max((1, 3)) / np.float32(448.0)).astype(np.float32)
    d = np.where(s > 0, s, np.float32(1.0))[:, None, :, None]
    return e4m3((b / d).astype(np.float32).astype(np.float64)).reshape(N, K), s


def tiles(codes):
    """Code bytes [N, K] -> the library's tiles, flat."""
    N, K = codes.shape
    out = np.empty(N * K, dtype=np.uint8)
    n, k = np.arange(N)[:, None], np.arange(K)[None]
    r, b = n % 128, k % 128
    at = ((n // 128) * (K // 128) + k // 128) * 16384 + r // 8 * 1024 + r % 8 * 128 + ((b // 16) ^ (r % 8)) * 16 + b % 16
    out[at] = codes
    return out


def gemm(a, w, ws):
    """float64 activations [M, K] (before quantisation), E4M3 values [N, K], scales [N/128, K/128] -> (C, sum of the
    products' magnitudes), float64."""
    q, s = quant_activations(a)
    a = q * np.repeat(s, 128, 1)
    w = w * np.repeat(np.repeat(ws.astype(np.float64), 128, 0), 128, 1)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def bound(c, reach, K):
    """What a kernel with exact products, fp32 sums and a BF16 result may be off by: each of a block's 128 additions, the
    K / 128 blocks', up to 16 parts' and two scalings round by 2^-24 of a partial sum, which is at most `reach`."""
    return 2.0 ** -8 * np.abs(c) + (128 + K // 128 + 16 + 2) * 2.0 ** -24 * reach
