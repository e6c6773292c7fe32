"""The operators between the projections, the cache, attention and the experts of a decoder layer, as cases to be measured.

  gemm    BF16 activations, quantised to E4M3 with a scale for each row and 128 columns, times E4M3 weights with a scale
          for each block of 128 x 128
  rope    norms of query and key heads and the rotation by position, one pass
  append  the same, with the keys and the values quantised into the paged MXFP4 cache
  route   a router's logits -> the experts of each token and their weights

`run` computes them from elementary torch operations, or, where `own` is set, through the library's entry points.
Layouts are those of include/a4w4.h: weights in swizzled tiles of 128 rows x 128 bytes, the cache in chunks of 16 tokens.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 2.0 ** -20
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one token of one user through a projection: the weights' bytes are everything
        dict(name="gemm_m1_n7168_k4224", op="gemm", m=1, n=7168, k=4224),
        # a decode step of 32 users, few output columns and a long sum
        dict(name="gemm_m32_n1536_k7168", op="gemm", m=32, n=1536, k=7168),
        # a ragged prompt chunk, few output columns
        dict(name="gemm_m513_n1536_k4224", op="gemm", m=513, n=1536, k=4224),
        # a long prompt chunk
        dict(name="gemm_m2048_n8448_k7168", op="gemm", m=2048, n=8448, k=7168),
        # one token: latency; rotation and norms of 32 + 8 heads
        dict(name="rope_t1", op="rope", t=1, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, far=131072),
        # a long prompt chunk, in place of the projection's heads
        dict(name="rope_t8191", op="rope", t=8191, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, far=131072),
        # one decode step of eight users: queries rotated, keys and values to the cache
        dict(name="append_t8", op="append", t=8, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, far=131072, page=64),
        # small heads, half of each rotated in neighbouring pairs, no norm, padding rows behind the last token
        dict(name="append_t333_d64", op="append", t=333, hq=16, hkv=4, d=64, rot=32, inter=True, norm=False, far=9000, page=16),
        # a long prompt chunk, keys and values as slices of one fused projection
        dict(name="append_t8191", op="append", t=8191, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, far=131072, page=32),
        # one token over many experts: latency
        dict(name="route_t1_e896", op="route", t=1, live=1, e=896, topk=16, score="softmax", bias=False, groups=1, group_top=1,
             top_groups=1, renorm=True, bf16=False),
        # experts in groups, BF16 logits, rows of padding behind the step's tokens
        dict(name="route_t1000_e256_g8", op="route", t=1000, live=977, e=256, topk=8, score="sigmoid", bias=True, groups=8,
             group_top=2, top_groups=4, renorm=True, bf16=True),
        # a prompt chunk over many experts, balanced by a bias
        dict(name="route_t4096_e896", op="route", t=4096, live=4096, e=896, topk=16, score="sigmoid", bias=True, groups=1,
             group_top=1, top_groups=1, renorm=True, bf16=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gemm", "gemm", "rope", "append", "append", "route", "route"))
    if op == "gemm":
        return dict(op=op, m=_log(rng, 1, 2048), n=128 * _log(rng, 1, 66), k=128 * _log(rng, 1, 56))
    if op == "route":
        e, g = _log(rng, 8, 1024), 1
        if rng.random() < 0.4:
            g = rng.choice((2, 4, 8, 16))
            e = g * _log(rng, 2, 64)
        top_groups = rng.randint(1, g)
        t = _log(rng, 1, 4096)
        return dict(op=op, t=t, live=t - rng.randint(0, t // 8), e=e, topk=rng.randint(1, min(32, e // g * top_groups)),
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.6, groups=g, group_top=rng.randint(1, 2),
                    top_groups=top_groups, renorm=rng.random() < 0.7, bf16=rng.random() < 0.4)
    d = rng.choice((64, 128))
    case = dict(op=op, t=_log(rng, 1, 8191), hq=rng.choice((4, 8, 12, 16, 32)), hkv=rng.choice((1, 2, 4, 8)), d=d,
                rot=16 * rng.randint(1, d // 16) if rng.random() < 0.4 else d, inter=rng.random() < 0.4, norm=rng.random() < 0.6,
                far=_log(rng, 100, 1 << 20))
    return dict(case, page=rng.choice((16, 32, 64, 128))) if op == "append" else case


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _weights(n, k, g):
    """A checkpoint's matrix: E4M3 codes and a float scale for each block of 128 x 128."""
    w = torch.randn(n, k, generator=g, device=DEV) * 0.02
    w *= 1.0 + 19.0 * (torch.rand(n, k, generator=g, device=DEV) < 0.001)
    b = w.view(n // 128, 128, k // 128, 128)
    scale = b.abs().amax((1, 3)) / 448.0
    return (b / scale[:, None, :, None]).to(torch.float8_e4m3fn).reshape(n, k), scale


def _tiles(w):
    """[N, K] bytes -> tiles of 128 x 128, row r's 16-byte piece c at place c ^ r % 8 of its 128 bytes."""
    n, k = w.shape
    t = w.view(n // 128, 16, 8, k // 128, 8, 16).permute(0, 3, 1, 2, 4, 5)  # [n/128, k/128, r/8, r%8, piece, byte]
    r, c = torch.arange(8, device=DEV)[:, None], torch.arange(8, device=DEV)[None]
    return t[:, :, :, r, c ^ r].contiguous().view(-1)


def _gemm_inputs(case, seed):
    g = _gen(seed)
    w, scale = _weights(case["n"], case["k"], g)
    a = torch.randn(case["m"], case["k"], generator=g, device=DEV)
    a *= 1.0 + 19.0 * (torch.rand(case["k"], generator=g, device=DEV) < 0.01)  # a few strong channels
    return a.bfloat16(), w, scale


def _heads_inputs(case, seed):
    """One fused projection's rows, norm weights, frequencies, positions."""
    g, t, hq, hkv, d, rot = _gen(seed), case["t"], case["hq"], case["hkv"], case["d"], case["rot"]
    x = torch.randn(t, hq + 2 * hkv, d, generator=g, device=DEV)
    x *= 1.0 + 5.0 * (torch.rand(hq + 2 * hkv, d, generator=g, device=DEV) < 0.03)
    wq, wk = (1.0 + 0.2 * torch.randn(d, generator=g, device=DEV) for _ in range(2))
    freq = (500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)).float()
    first = torch.randint(0, max(1, case["far"] - t), (1,), generator=g, device=DEV)
    pos = first + torch.arange(t, device=DEV)
    if t <= 64:  # tokens of different requests
        pos = torch.randint(0, case["far"], (t,), generator=g, device=DEV)
    return x.bfloat16(), wq, wk, freq, pos.int(), g


def _slots(case, g):
    t, page = case["t"], case["page"]
    pages = (t + page - 1) // page + 3
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(t, device=DEV) + page // 2 + 1
    slots = (order[at // page] * page + at % page).int()
    if t > 40:  # rows of padding at the end of a captured step
        slots[-3:] = -1
    return pages, slots


def _route_inputs(case, seed):
    g, t, e = _gen(seed), case["t"], case["e"]
    x = torch.randn(t, e, generator=g, device=DEV) * 1.5 + 0.5 * torch.randn(e, generator=g, device=DEV)
    bias = 0.05 * torch.randn(e, generator=g, device=DEV) if case["bias"] else None
    return x.bfloat16() if case["bf16"] else x, bias


def prepare(case, seed):
    s = dict(case)
    if case["op"] == "gemm":
        a, w, scale = _gemm_inputs(case, seed)
        m, n, k = case["m"], case["n"], case["k"]
        s.update(a=a, w=w, scale=scale, w8=_tiles(w.view(torch.uint8)), out=torch.empty(m, n, dtype=torch.bfloat16, device=DEV),
                 ws=torch.zeros(((m + 127) // 128) * 128 * (k + k // 32) + 4096, dtype=torch.uint8, device=DEV))
        return s
    if case["op"] == "route":
        x, bias = _route_inputs(case, seed)
        t, topk = case["t"], case["topk"]
        s.update(x=x, bias=bias, count=torch.tensor([case["live"]], dtype=torch.int32, device=DEV), scale=2.5,
                 ids=torch.empty(t, topk, dtype=torch.int32, device=DEV), weights=torch.empty(t, topk, dtype=torch.float32, device=DEV))
        return s
    x, wq, wk, freq, pos, g = _heads_inputs(case, seed)
    t, hq, hkv, d = case["t"], case["hq"], case["hkv"], case["d"]
    s.update(q=x[:, :hq], k=x[:, hq: hq + hkv], v=x[:, hq + hkv:], wq=wq if case["norm"] else None,
             wk=wk if case["norm"] else None, freq=freq, pos=pos,
             q_out=torch.zeros(t, hq, d, dtype=torch.bfloat16, device=DEV),
             k_out=torch.zeros(t, hkv, d, dtype=torch.bfloat16, device=DEV))
    if case["op"] == "append":
        pages, slots = _slots(case, g)
        s.update(pages=pages, slots=slots, v_out=torch.zeros_like(s["k_out"]),
                 cache=torch.zeros(pages, hkv, case["page"] // 16, 17 * d, dtype=torch.uint8, device=DEV))
    return s


# ---------------------------------------------------------------------------
# the library's operators

def _own(s):
    import mxfp4_a4w4_gemm_gb300 as lib

    if s["op"] == "gemm":
        lib.a4w4_gemm_w8a8(s["a"], s["m"], s["k"], s["w8"], s["scale"], s["n"], s["out"], s["ws"], s["ws"].numel())
        return s["out"]
    if s["op"] == "route":
        lib.a4w4_moe_route(s["x"], lib.A4W4_BF16 if s["bf16"] else lib.A4W4_F32, s["e"], s["count"], s["t"], s["e"],
                           lib.A4W4_MOE_SCORE_SOFTMAX if s["score"] == "softmax" else lib.A4W4_MOE_SCORE_SIGMOID, s["bias"],
                           s["groups"], s["group_top"], s["top_groups"], s["topk"], int(s["renorm"]), s["scale"], s["ids"],
                           s["weights"])
        return {"ids": s["ids"], "weights": s["weights"]}
    q, k, v = s["q"], s["k"], s["v"]
    if s["op"] == "rope":
        lib.a4w4_qk_norm_rope(q, q.stride(0), k, k.stride(0), s["pos"], s["t"], s["hq"], s["hkv"], s["d"], s["wq"], s["wk"], EPS,
                              s["freq"], s["rot"], int(s["inter"]), s["q_out"], s["hq"] * s["d"], s["k_out"], s["hkv"] * s["d"])
        return {"q": s["q_out"], "k": s["k_out"]}
    lib.a4w4_kv_append_rope(q, q.stride(0), k, k.stride(0), v, v.stride(0), s["pos"], s["slots"], s["t"], s["hq"], s["hkv"], s["d"],
                            s["wq"], s["wk"], EPS, s["freq"], s["rot"], int(s["inter"]), s["q_out"], s["hq"] * s["d"], s["cache"],
                            s["pages"], s["page"])
    lib.a4w4_kv_read(s["cache"], s["pages"], s["page"], s["slots"], s["t"], s["hkv"], s["d"], s["k_out"], s["v_out"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


# ---------------------------------------------------------------------------
# the plain form

def _plain_gemm(s):
    m, n, k = s["m"], s["n"], s["k"]
    a = s["a"].float().view(m, k // 128, 128)
    frac, exp = torch.frexp(a.abs().amax(-1, keepdim=True))  # amax = frac 2^exp, frac in [1/2, 1); 448 = 7/8 2^9
    exp = torch.where(frac <= 0.875, exp - 9, exp - 8).clamp(min=-126)
    codes = torch.ldexp(a, -exp).to(torch.float8_e4m3fn).float()
    a = torch.ldexp(codes, exp).view(m, k)
    w = (s["w"].float().view(n // 128, 128, k // 128, 128) * s["scale"][:, None, :, None]).view(n, k)
    return (a @ w.T).bfloat16()


def _rotated(s, x, w, wide):
    """Norm and rotation of heads [t, h, d]; in 64 bits where `wide` is set."""
    x = x.to(torch.float64 if wide else torch.float32)
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)
    ang = s["pos"].double()[:, None, None] * s["freq"].double()  # far positions: 32 bits would lose the angle
    c, z = torch.cos(ang).to(x.dtype), torch.sin(ang).to(x.dtype)
    r = s["rot"]
    if s["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * z, b * c + a * z], -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y = torch.cat([a * c - b * z, b * c + a * z], -1)
    return torch.cat([y, x[..., r:]], -1)


def _cells(x):
    """Rows -> (signed codes 0..15, E8M0 scale bytes) of their MXFP4 form, blocks of 32."""
    b = x.unflatten(-1, (-1, 32))
    e = (torch.frexp(b.abs().amax(-1, keepdim=True)).exponent - 3).clamp(min=-127)
    y = torch.ldexp(b.abs(), -e)
    # round to the nearest of E2M1's magnitudes, ties to the even code: a midpoint goes up where the code above is even
    c = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    e = torch.where(b.abs().amax(-1, keepdim=True) > 0, e, torch.full_like(e, -127))
    return (c + torch.signbit(b) * 8).flatten(-2).to(torch.uint8), (e + 127).squeeze(-1).to(torch.uint8)


def _places(d):
    """Byte offsets in a chunk: code pairs [16, d/2] and scales [16, d/32], for keys and for values."""
    tok = torch.arange(16, device=DEV)[:, None]
    p = 2 * torch.arange(d // 2, device=DEV)[None]
    j, t, b = p // 32, p % 32 // 8, p % 8 // 2
    kc = tok * (d // 2) + (t * (d // 32) + j) * 4 + b
    ks = 8 * d + tok * (d // 32) + torch.arange(d // 32, device=DEV)[None]
    i, g = p // 16, p % 16 // 2
    vc = 17 * d // 2 + tok // 8 * 4 * d + (g * 4 + tok % 8 // 2) * (d // 8) + tok % 2 * (d // 16) + i
    return kc, ks, vc, ks + 17 * d // 2


def _values(codes, scales):
    """Packed code bytes [..., n/2] and scale bytes [..., n/32] -> float32 [..., n]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return lut[nib.int()] * torch.exp2(scales.float() - 127.0).repeat_interleave(32, -1)


def _plain_append(s):
    page, cache, ok = s["page"], s["cache"], s["slots"] >= 0
    kc, ks, vc, vs = _places(s["d"])
    live = ok.nonzero()[:, 0]
    heads = torch.arange(s["hkv"], device=DEV)[None, :, None]

    def at(where, slot):
        return (slot // page)[:, None, None], heads, (slot % page // 16)[:, None, None], where[slot % 16][:, None, :]

    slot = s["slots"][live].long()
    for x, where_codes, where_scales in ((_rotated(s, s["k"], s["wk"], True), kc, ks),  # a code hangs on which side of a border the value lies
                                         (s["v"].float(), vc, vs)):
        c, e = _cells(x[live])
        cache[at(where_codes, slot)] = c[..., 0::2] | c[..., 1::2] << 4
        cache[at(where_scales, slot)] = e
    slot, gone = s["slots"].clamp(min=0).long(), ~ok[:, None, None]
    k = _values(cache[at(kc, slot)], cache[at(ks, slot)]).masked_fill(gone, 0.0).bfloat16()
    v = _values(cache[at(vc, slot)], cache[at(vs, slot)]).masked_fill(gone, 0.0).bfloat16()
    q = torch.where(gone, s["q_out"], _rotated(s, s["q"], s["wq"], False).bfloat16())  # rows behind the last token stay
    return {"q": q, "k": k, "v": v}


def _plain_route(s):
    x = s["x"].double()  # scores that nearly tie: 32 bits would order them otherwise
    score = torch.softmax(x, -1) if s["score"] == "softmax" else torch.sigmoid(x)
    c = score if s["bias"] is None else score + s["bias"].double()
    if s["groups"] > 1:
        members = c.unflatten(-1, (s["groups"], -1))
        strength = members.sort(-1, descending=True).values[..., : s["group_top"]].sum(-1)
        best = strength.sort(dim=-1, descending=True, stable=True).indices[:, : s["top_groups"]]
        kept = torch.zeros_like(strength, dtype=torch.bool).scatter_(1, best, True)
        c = members.masked_fill(~kept[..., None], -torch.inf).flatten(1)
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, : s["topk"]]
    w = score.gather(1, ids)
    w = w / w.sum(-1, keepdim=True) if s["renorm"] else w
    dead = torch.arange(s["t"], device=DEV)[:, None] >= s["count"]
    return {"ids": ids.masked_fill(dead, -1).int(), "weights": (w * s["scale"]).masked_fill(dead, 0.0).float()}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "gemm":
        return _plain_gemm(s)
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "append":
        return _plain_append(s)
    return {"q": _rotated(s, s["q"], s["wq"], False).bfloat16(), "k": _rotated(s, s["k"], s["wk"], False).bfloat16()}


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits

def work(case):
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k + 4 * (n // 128) * (k // 128) + 2 * m * n, "flops": 2 * m * n * k}
    if case["op"] == "route":
        t, e = case["live"], case["e"]
        return {"bytes": t * e * (2 if case["bf16"] else 4) + 4 * e + 8 * case["t"] * case["topk"], "flops": 8 * t * e}
    t, hq, hkv, d = case["t"], case["hq"], case["hkv"], case["d"]
    flops = 10 * t * (hq + hkv) * d
    if case["op"] == "rope":
        return {"bytes": 4 * t * (hq + hkv) * d + 4 * t, "flops": flops}
    cell = 2 * (d // 2 + d // 32)  # a key row and a value row of one head
    # the cells are written and read back, and their values written
    return {"bytes": 4 * t * hq * d + t * hkv * (4 * d + 2 * cell + 4 * d) + 12 * t, "flops": flops}


def _near(x, step):
    return torch.round(x / step) * step  # torch.round takes ties to even, as the codes do


def _exact_heads(case, x, w, freq, pos):
    x = x.double()
    if case["norm"]:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + EPS) * w.double()
    r = case["rot"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[:, None] * freq.double()[None])[:, None]
    if case["inter"]:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., r:]], -1)
    z = torch.complex(x[..., : r // 2].contiguous(), x[..., r // 2: r].contiguous()) * turn
    return torch.cat([z.real, z.imag, x[..., r:]], -1)


def _exact_cells(x):
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    exp = torch.frexp(top).exponent - 3  # top = m 2^exponent with m in [1/2, 1): floor(log2 top) - 2
    unit = torch.ldexp(torch.ones_like(top), exp.clamp(min=-127))
    y = (b.abs() / unit).clamp(max=6.0)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
    return (_near(y, step).clamp(max=6.0) * unit * torch.sign(b)).flatten(-2)


def exact(case, seed):
    if case["op"] == "gemm":
        a, w, scale = _gemm_inputs(case, seed)
        m, n, k = case["m"], case["n"], case["k"]
        a = a.double().view(m, -1, 128)
        top = a.abs().amax(-1, keepdim=True)
        unit = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
        unit = torch.where(top > 448.0 * unit, 2 * unit, torch.where(top <= 224.0 * unit, unit / 2, unit))
        unit = torch.where(top > 0, unit, torch.ones_like(unit))
        y = a / unit
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)  # three bits behind the leading one
        a = (_near(y, step) * unit).view(m, k)
        return a @ (w.double() * scale.double().repeat_interleave(128, 0).repeat_interleave(128, 1)).T
    if case["op"] == "route":
        x, bias = _route_inputs(case, seed)
        x, e = x.double(), case["e"]
        s = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) if case["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-x))
        c = s.clone() if bias is None else s + bias.double()
        if case["groups"] > 1:
            per = e // case["groups"]
            strength = torch.stack([c[:, i * per: (i + 1) * per].topk(case["group_top"]).values.sum(-1) for i in range(case["groups"])], 1)
            other, mine = strength[:, None, :], strength[:, :, None]
            before = torch.ones(case["groups"], case["groups"], dtype=torch.bool, device=DEV).tril(-1)  # of equals the lower comes first
            rank = ((other > mine) | (other == mine) & before).sum(-1)
            c[(rank >= case["top_groups"]).repeat_interleave(per, 1)] = -torch.inf
        got = []
        for _ in range(case["topk"]):
            best = torch.argmax(c, -1, keepdim=True)
            got.append(s.gather(1, best))
            c.scatter_(1, best, -torch.inf)
        w = torch.cat(got, 1)
        w = (w / w.sum(-1, keepdim=True) if case["renorm"] else w) * 2.5
        w[case["live"]:] = 0.0
        return {"ids": None, "weights": w}
    x, wq, wk, freq, pos, g = _heads_inputs(case, seed)
    hq, hkv = case["hq"], case["hkv"]
    q = _exact_heads(case, x[:, :hq], wq, freq, pos)
    k = _exact_heads(case, x[:, hq: hq + hkv], wk, freq, pos)
    if case["op"] == "rope":
        return {"q": q, "k": k}
    _, slots = _slots(case, g)
    ok = (slots >= 0).view(-1, 1, 1)
    return {"q": q * ok, "k": _exact_cells(k) * ok, "v": _exact_cells(x[:, hq + hkv:].double()) * ok}
