"""Oracle of the norms and the rotation of query and key heads (a4w4_qk_norm_rope and
a4w4_kv_append_rope of include/a4w4.h, restated from that header's text), in float64.
"""

import numpy as np


def heads(x, weight, eps, positions, inv_freq, rot, interleaved):
    """x [T, H, D] float64; weight [D] or None; positions [T]; inv_freq [rot/2] float32 -> (result, reach), float64.
    reach: r (|w x| + |w' x'|) with x' the pair's other half (|w x| alone where nothing turns): what roundings are
    relative to."""
    T, H, D = x.shape
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + float(np.float32(eps))) * weight.astype(np.float64)
    out, reach = y.copy(), np.abs(y)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        # positions and frequencies are exact in long double; their product is to 2^-64 of it
        ang = np.asarray(positions, dtype=np.longdouble) * np.longdouble(inv_freq[i])
        c, s = (f(ang).astype(np.float64)[:, None] for f in (np.cos, np.sin))
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        reach[..., a] = reach[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, reach


def bound(want, reach):
    """fp32 within 2^-20.1 of reach (the norm's reciprocal 2^-20.9, sine and cosine 2^-22.7, four roundings), then BF16."""
    return 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * reach + 2.0 ** -133
