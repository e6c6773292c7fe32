"""Paged MXFP4 key/value cache oracle: step plan, cache bytes, attention.

Plain restatement of the calls a4w4_kv_* of include/a4w4.h, from that header's
text: requests one after another for the plan, the byte formulas for the cache,
float64 for the attention.
"""

import functools

import numpy as np

from . import mxfp4


def plan(past, new, page_size, table, ring, head, count, max_tokens):
    """One step's plan, request after request.  table [B, W] and ring are not
    changed; returns a dict of the call's outputs."""
    B, width = table.shape
    table, ring = table.copy(), ring.copy()
    size = len(ring)
    kv, cu, slots, pos, gone = [], [0], [], [], []
    left, tokens, refused, closed, taken = count, max_tokens, 0, False, 0
    for b in range(B):
        p, n = int(past[b]), int(new[b])
        held = -(-p // page_size)
        if n < 0:
            gone += list(table[b, :held])
            kv.append(0)
            cu.append(cu[-1])
            continue
        if n > 0 and p + n > width * page_size:
            refused += 1
            kv.append(p)
            cu.append(cu[-1])
            continue
        need = -(-(p + n) // page_size) - held
        if n > 0 and (closed or need > left or n > tokens):
            closed = True
            refused += 1
            kv.append(p)
            cu.append(cu[-1])
            continue
        for j in range(need):
            table[b, held + j] = ring[(head + taken) % size]
            taken += 1
        left -= need
        tokens -= n
        for t in range(p, p + n):
            slots.append(int(table[b, t // page_size]) * page_size + t % page_size)
            pos.append(t)
        kv.append(p + n)
        cu.append(cu[-1] + n)
    for i, pg in enumerate(gone):
        ring[(head + count + i) % size] = pg
    pad = max_tokens - len(slots)
    i32 = lambda x: np.asarray(x, dtype=np.int32)  # noqa: E731
    return {"block_table": table, "free_ring": ring, "ring_state": i32([(head + taken) % size, count - taken + len(gone)]),
            "kv_lens": i32(kv), "cu_new": i32(cu), "slot_map": i32(slots + [-1] * pad), "positions": i32(pos + [0] * pad),
            "refused": i32([refused])}


def chunk_bytes(codes_k, scales_k, codes_v, scales_v):
    """One chunk: unpacked codes [16, D] and scales [16, D/32] -> uint8 [17 * D]."""
    D = codes_k.shape[1]
    J = D // 32
    out = np.zeros(17 * D, dtype=np.uint8)
    for r in range(16):
        for n in range(0, D, 2):
            j, t, b = n // 32, n % 32 // 8, n % 8 // 2
            out[r * (D // 2) + (t * J + j) * 4 + b] = codes_k[r, n] | codes_k[r, n + 1] << 4
            i, g = n // 16, n % 16 // 2
            at = (r // 8) * 4 * D + (g * 4 + r % 8 // 2) * (D // 8) + (r % 2) * (D // 16) + i
            out[8 * D + D // 2 + at] = codes_v[r, n] | codes_v[r, n + 1] << 4
        for j in range(J):
            out[8 * D + r * J + j] = scales_k[r, j]
            out[8 * D + D // 2 + 8 * D + r * J + j] = scales_v[r, j]
    return out


@functools.lru_cache(maxsize=None)
def byte_places(D):
    """Offsets in a chunk of (key codes [16, D/2], key scales [16, D/32], value codes, value scales), found
    from chunk_bytes one byte at a time."""
    J = D // 32
    parts = [np.zeros((16, D), np.uint8), np.zeros((16, J), np.uint8), np.zeros((16, D), np.uint8), np.zeros((16, J), np.uint8)]
    places = []
    for part in range(4):
        cols = J if part % 2 else D // 2
        place = np.empty((16, cols), dtype=np.int64)
        for r in range(16):
            for c in range(cols):
                a = [x.copy() for x in parts]
                a[part][r, c if part % 2 else 2 * c] = 1
                hit = np.nonzero(chunk_bytes(*a))[0]
                assert hit.size == 1
                place[r, c] = hit[0]
        places.append(place)
    return tuple(places)


def cache_from_rows(k_codes, k_scales, v_codes, v_scales, page_size):
    """Rows in slot order (codes [slots, H, D], scales [slots, H, D/32]) -> cache bytes, flat."""
    S, H, D = k_codes.shape
    places = byte_places(D)
    out = np.zeros((S // page_size, H, page_size // 16, 17 * D), dtype=np.uint8)
    for part, x in enumerate((mxfp4.pack_codes(k_codes), k_scales, mxfp4.pack_codes(v_codes), v_scales)):
        x = x.reshape(S // page_size, page_size // 16, 16, H, -1).transpose(0, 3, 1, 2, 4)
        out[..., places[part]] = x
    return out.reshape(-1)


def attention(q, keys, values, sm_scale):
    """q [n, Hq, D], keys/values [len, Hkv, D], all float64 -> (out [n, Hq, D], lse [n, Hq], spread [n, Hq, D] =
    sum p |v|, reach [n, Hq] = the largest sm_scale * sum |q k| among the keys seen)."""
    n, Hq, D = q.shape
    L, Hkv = keys.shape[:2]
    out, spread = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, reach = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        seen = max(0, L - n + i + 1)
        if seen == 0:
            continue
        for h in range(Hq):
            k, v = keys[:seen, h // (Hq // Hkv)], values[:seen, h // (Hq // Hkv)]
            x = sm_scale * (k @ q[i, h])
            top = x.max()
            e = np.exp(x - top)
            p = e / e.sum()
            out[i, h], spread[i, h] = p @ v, p @ np.abs(v)
            lse[i, h] = top + np.log(e.sum())
            reach[i, h] = sm_scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, lse, spread, reach


# What rounding may put a probability off by, relatively: half a unit in the last place of a type of n significant bits
# is up to 2^-n of the value (a value just above a power of two).
P_ONE_BF16 = 2.0 ** -8       # one BF16 term
P_TWO_BF16 = 2.0 ** -16      # two: the second holds what the first leaves, to 2^-8 of it
# FP16, 2^-11; its product with a value's power of two may fall to FP16's last exponent but one, where 10 bits are left
P_FP16 = 2.0 ** -11 + 2.0 ** -10


def attention_bounds(out, lse, spread, reach, p_round=2.0 ** -9):
    """Error bounds of a kernel that holds exact products and fp32 sums, rounds each probability by at most p_round
    of it (the default covers FP16 and two BF16 terms; one BF16 term takes P_ONE_BF16) and the output to BF16.

    A score is a sum of at most 128 exact products in fp32: its error is at most 128 * 2^-24 * reach, plus a few
    roundings of the score itself (2^-22 |x| <= 2^-22 reach).  A probability is then off by that much relatively,
    in the numerator and in the sum (twice), by p_round in the numerator, whose rounding follows the sum's, and by
    the exponential's and the sums' few 2^-22 (2^-18 in all).  The output's own rounding is 2^-8 of it; the sum over
    keys adds n * 2^-24 at most, 2^-10 up to 16384 keys.  The log-sum-exp takes the score's error once."""
    dx = (2.0 ** -17 + 2.0 ** -22) * reach
    rel = 2 * np.expm1(dx) + p_round + 2.0 ** -10 + 2.0 ** -18
    return 2.0 ** -8 * np.abs(out) + rel[..., None] * spread, dx + 2.0 ** -18 * (1 + np.where(np.isfinite(lse), np.abs(lse), 0))
