"""Oracle of the routing to experts (a4w4_moe_route of include/a4w4.h, restated from that
header's text), one token after another in float64.
"""

import numpy as np

FLT_MAX = float(np.finfo(np.float32).max)


def scores(x, softmax):
    """Logits of one token, as they count (NaN as -infinity, +infinity as the largest float) -> (those, scores)."""
    x = np.asarray(x, dtype=np.float64)
    x = np.minimum(np.where(np.isnan(x), -np.inf, x), FLT_MAX)
    if softmax:
        top = x.max()
        if np.isneginf(top):
            return x, np.zeros_like(x)
        e = np.exp(x - top)
        return x, e / e.sum()
    with np.errstate(over="ignore"):
        return x, np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def best(c, k):
    """Indices of the k largest, largest first, of equals the lower first."""
    return sorted(range(len(c)), key=lambda i: (-c[i], i))[:k]


def route(x, softmax, bias, groups, group_top, top_groups, topk, renormalise, scale):
    """One token -> (ids [topk], weights [topk])."""
    x, s = scores(x, softmax)
    c = s if bias is None else s + np.where(np.isnan(bias), -np.inf, np.asarray(bias, dtype=np.float64))
    allowed = list(range(len(x)))
    # scores of logits that differ may round to the same number: without a bias the logits order them
    order = c if bias is not None else x
    if groups > 1:
        per = len(x) // groups
        by = order if group_top == 1 else c
        strength = [sum(sorted(by[g * per: (g + 1) * per])[-group_top:]) for g in range(groups)]
        kept = best(strength, top_groups)
        allowed = [i for i in allowed if i // per in kept]
    ids = [allowed[i] for i in best([order[j] for j in allowed], topk)]
    w = s[ids]
    if renormalise:
        if softmax:                                     # (scores may be too small even for float64)
            m = x[ids].max()
            w = np.zeros(topk) if np.isneginf(m) else np.exp(x[ids] - m)
        w = w / w.sum() if w.sum() > 0 else np.zeros(topk)
    return ids, w * scale
