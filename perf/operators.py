"""The operators of the 4-bit paged key/value cache, as cases to be measured.

Four operators that a serving step runs one after the other:

  plan       block tables, slot map and positions from the requests' lengths
  append     new BF16 keys and values -> MXFP4 rows of the paged cache
  read       cache rows -> the BF16 values they stand for
  attention  softmax(Q K^T) V over the cached keys and values, ragged batches

`run` computes them from elementary torch operations, or, where `own` is set,
through the library's entry points.  Cache layout (include/a4w4.h): pages of
`page_size` tokens, per page and key/value head page_size / 16 chunks of 16
tokens, each 17 * D bytes: key codes, key scales, value codes, value scales.
"""

import math

import torch

own = False

DEV = "cuda"
WORKSPACE = 64 << 20  # bytes that a server sets aside, zeroed once, for all its attention calls
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # one decode step of a small server: eight requests, one token each
        dict(name="plan_step_b8", op="plan", b=8, new=1, past=4096, page=64, tight=False),
        # continuous batching at its largest: chunks, single tokens, finished requests, pages running out
        dict(name="plan_mixed_b2000", op="plan", b=2000, new=64, past=9000, page=16, tight=True),
        # the cache write of that decode step, one layer
        dict(name="append_step_t8", op="append", t=8, hkv=8, d=128, page=64),
        # the cache write of a long prompt chunk, keys and values as slices of a fused projection
        dict(name="append_prompt_t8191", op="append", t=8191, hkv=8, d=128, page=32),
        # a short prefix handed to another program, small heads
        dict(name="read_prefix_t333", op="read", t=333, hkv=2, d=64, page=16),
        # a long context read back whole
        dict(name="read_context_t40000", op="read", t=40000, hkv=8, d=128, page=64),
        # one user, short context: latency
        dict(name="decode_b1_kv1000", op="attention", b=1, q=1, kv=1000, hq=32, hkv=8, d=128, page=64, ragged=False),
        # a full server decoding: ragged contexts, groups of eight
        dict(name="decode_b64_kv8192", op="attention", b=64, q=1, kv=8192, hq=64, hkv=8, d=128, page=64, ragged=True),
        # two very long contexts, groups of sixteen: the key axis is all the parallelism there is
        dict(name="decode_b2_kv131000", op="attention", b=2, q=1, kv=131000, hq=64, hkv=4, d=128, page=128, ragged=False),
        # five draft tokens verified per request, small heads, some contexts empty
        dict(name="verify_b24_q5_kv3001", op="attention", b=24, q=5, kv=3001, hq=32, hkv=8, d=64, page=16, ragged=True),
        # prompts of many lengths in one batch, small heads, rows with nothing to see among them
        dict(name="prompts_b12_q700_kv1500", op="attention", b=12, q=700, kv=1500, hq=16, hkv=4, d=64, page=32, ragged=True),
        # one chunk of a long prompt against what is cached of it
        dict(name="chunk_q4096_kv16384", op="attention", b=1, q=4096, kv=16384, hq=32, hkv=8, d=128, page=64, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    page = rng.choice((16, 32, 64, 128))
    d = rng.choice((64, 128))
    op = rng.choice(("plan", "append", "read", "attention", "attention", "attention"))
    if op == "plan":
        return dict(op=op, b=_log(rng, 1, 2000), new=_log(rng, 1, 64), past=_log(rng, 1, 9000), page=page,
                    tight=rng.random() < 0.5)
    if op in ("append", "read"):
        return dict(op=op, t=_log(rng, 1, 8191 if op == "append" else 40000), hkv=rng.choice((1, 2, 4, 8)), d=d, page=page)
    hkv = rng.choice((1, 2, 4, 8))
    hq = hkv * rng.choice((1, 2, 3, 4, 6, 8, 16))
    kind = rng.random()
    if kind < 0.5:
        q, kv, b = 1, _log(rng, 1, 131000), _log(rng, 1, 64)
    elif kind < 0.7:
        q, kv, b = rng.randint(2, 8), _log(rng, 8, 16384), _log(rng, 1, 32)
    else:
        q, kv, b = _log(rng, 9, 4096), _log(rng, 64, 16384), _log(rng, 1, 16)
        q = min(q, kv)
    # no more keys, and no more scores, than the largest listed cases hold
    while b > 1 and (b * kv * hkv * d > 64 * 8192 * 8 * 128 or b * q * kv * hq > 1 << 30):
        b = (b + 1) // 2
    while b * q * kv * hq > 1 << 30 and q > 1:
        q = (q + 1) // 2
    while b * kv * hkv * d > 64 * 8192 * 8 * 128 and kv > 1:
        kv = (kv + 1) // 2
    q = min(q, kv)
    return dict(op=op, b=b, q=q, kv=kv, hq=hq, hkv=hkv, d=d, page=page, ragged=rng.random() < 0.6)


# ---------------------------------------------------------------------------
# inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _ints(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _key_values(rows, hkv, d, g):
    """Keys and values as a projection gives them: keys with a few strong channels, BF16."""
    k = torch.randn(rows, hkv, d, generator=g, device=DEV)
    k *= 1.0 + 5.0 * (torch.rand(hkv, d, generator=g, device=DEV) < 0.03)
    v = torch.randn(rows, hkv, d, generator=g, device=DEV) * 0.5
    return k.bfloat16(), v.bfloat16()


def _cells(x):
    """BF16 rows -> (codes 0..15, E8M0 scale bytes) of their MXFP4 form, blocks of 32."""
    bits = x.view(torch.int16).to(torch.int32) & 0x7FFF
    e = (bits.unflatten(-1, (-1, 32)).amax(-1) >> 7).sub(2).clamp(min=0)
    y = x.float().abs() * (254 - e << 23).view(torch.float32).repeat_interleave(32, -1)  # times 2^(127 - e)
    # round to the nearest of E2M1's magnitudes, ties to the even code: a midpoint goes up where the code above is even
    c = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    return (c + torch.signbit(x) * 8).to(torch.uint8), e.to(torch.uint8)


def _places(d):
    """Byte offsets in a chunk: code pairs [16, d/2] and scales [16, d/32], for keys and for values."""
    tok = torch.arange(16, device=DEV)[:, None]
    p = 2 * torch.arange(d // 2, device=DEV)[None, :]
    blk = torch.arange(d // 32, device=DEV)[None, :]
    w = min(d, 128)
    grp, dd = p // w, p % w
    j, t, b = dd // 32, dd % 32 // 8, dd % 8 // 2
    kc = grp * 8 * w + tok * (w // 2) + (t * (w // 32) + j) * 4 + b
    ks = 8 * d + tok * (d // 32) + blk
    i, g = dd // 16, dd % 16 // 2
    vc = 17 * d // 2 + grp * 8 * w + tok // 8 * 4 * w + (g * 4 + tok % 8 // 2) * (w // 8) + tok % 2 * (w // 16) + i
    return kc, ks, vc, ks + 17 * d // 2


def _contents(case, g, pages, live):
    """What the pages hold, in token order: codes and scales of keys and values; places that are not `live` hold anything."""
    n, hkv, d = pages * case["page"], case["hkv"], case["d"]
    out = []
    for x in _key_values(n, hkv, d, g):
        c, e = _cells(x)
        out += [c, torch.where(live.view(n, 1, 1), e, torch.full_like(e, 255))]
    return out


def _pack(case, pages, kc, ks, vc, vs):
    page, hkv, d = case["page"], case["hkv"], case["d"]
    cache = torch.empty(pages, hkv, page // 16, 17 * d, dtype=torch.uint8, device=DEV)
    at = _places(d)
    for codes, scales, ca, sa in ((kc, ks, at[0], at[1]), (vc, vs, at[2], at[3])):
        byte = codes[..., 0::2] | codes[..., 1::2] << 4
        for part, where in ((byte, ca), (scales, sa)):
            cache[..., where.reshape(-1)] = part.view(pages, page // 16, 16, hkv, -1).permute(0, 3, 1, 2, 4).flatten(3)
    return cache


def _plan_inputs(case, seed):
    g, b, page = _gen(seed), case["b"], case["page"]
    past = _ints(0, case["past"] + 1, (b,), g)
    kind = torch.rand(b, generator=g, device=DEV)
    new = torch.where(kind < 0.6, torch.ones_like(past), _ints(1, case["new"] + 1, (b,), g))
    if b > 8:  # some requests pause, some are finished and give their pages back
        new = torch.where(kind < 0.05, torch.zeros_like(new), torch.where(kind > 0.95, torch.full_like(new, -1), new))
    width = (case["past"] + case["new"] + page - 1) // page
    held = (past + page - 1) // page
    pages = b * width + 64
    ids = torch.randperm(pages, generator=g, device=DEV).int()
    table = ids[: b * width].view(b, width).clone()
    ring = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    grown = torch.where(new > 0, (past + new + page - 1) // page - held, torch.zeros_like(held)).sum().item()
    count = max(1, grown * 4 // 5) if case["tight"] else min(pages, grown + 40)
    head = pages - max(1, count // 2)  # the free pages lie across the ring's end
    ring[(head + torch.arange(count, device=DEV)) % pages] = torch.randperm(pages, generator=g, device=DEV).int()[:count]
    tokens = b * case["new"] + 8
    state = torch.tensor([head, count], dtype=torch.int32, device=DEV)
    return dict(past=past, new=new, table=table, ring=ring, state=state, width=width, pages=pages, tokens=tokens)


def _rows_inputs(case, seed):
    """Slots on scattered pages, and the rows that go there."""
    g, t, page = _gen(seed), case["t"], case["page"]
    pages = (t + page - 1) // page + 3
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(t, device=DEV) + page // 2 + 1
    slots = (order[at // page] * page + at % page).int()
    if t > 40:  # rows of padding at the end of a captured step
        slots[-3:] = -1
    return g, pages, slots


def _lengths(case, g):
    b, q, kv = case["b"], case["q"], case["kv"]
    lens, new = torch.full((b,), kv, dtype=torch.int32, device=DEV), torch.full((b,), q, dtype=torch.int32, device=DEV)
    if case["ragged"]:
        lens = _ints(1, kv + 1, (b,), g)
        new = _ints(1, q + 1, (b,), _gen(b))  # the batch's shape is the case's own: as many rows whatever the seed
        lens[0], new[-1] = kv, q
        if b > 4:  # an idle row, an empty context, and more queries than keys
            new[1] = 0
            lens[2] = 0
            lens[3] = torch.minimum(lens[3], new[3] // 2)
    return lens, new


def _attention_inputs(case, seed):
    g, b, page = _gen(seed), case["b"], case["page"]
    lens, new = _lengths(case, g)
    cu = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(new, 0)
    held = (lens + page - 1) // page
    pages, width = int(held.sum()) + 1, (case["kv"] + page - 1) // page
    order = torch.randperm(pages, generator=g, device=DEV).int()
    first = torch.cumsum(held, 0) - held
    col = torch.arange(width, device=DEV, dtype=torch.int32)[None]
    table = torch.where(col < held[:, None], order[torch.minimum(first[:, None] + col, torch.tensor(pages - 1, device=DEV)).long()], 0)
    used = (lens[:, None] - col * page).clamp(0, page)  # live tokens of each table entry
    count = torch.zeros(pages, dtype=torch.int32, device=DEV)
    count[table[used > 0].long()] = used[used > 0].int()
    live = torch.arange(page, device=DEV)[None] < count[:, None]
    total = int(cu[-1])
    x = torch.randn(total, case["hq"] + 2 * case["hkv"], case["d"], generator=g, device=DEV).bfloat16()
    return dict(lens=lens, new=new, cu=cu, pages=pages, width=width, table=table.int().contiguous(), live=live, total=total,
                qkv=x, g=g)


def prepare(case, seed):
    s = dict(case)
    if case["op"] == "plan":
        s.update(_plan_inputs(case, seed))
        b, n = case["b"], s["tokens"]
        empty = lambda k: torch.empty(k, dtype=torch.int32, device=DEV)  # noqa: E731
        s.update(state_out=empty(2), kv_lens=empty(b), cu=empty(b + 1), slots=empty(n), positions=empty(n), refused=empty(1))
        return s
    if case["op"] in ("append", "read"):
        g, pages, slots = _rows_inputs(case, seed)
        t, hkv, d, page = case["t"], case["hkv"], case["d"], case["page"]
        s.update(pages=pages, slots=slots, k_out=torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV),
                 v_out=torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV))
        if case["op"] == "append":
            k, v = _key_values(t, hkv, d, g)
            fused = torch.cat([torch.zeros_like(k), k, v], 1)  # queries, keys and values of one projection
            s.update(k=fused[:, hkv: 2 * hkv], v=fused[:, 2 * hkv:],
                     cache=torch.zeros(pages, hkv, page // 16, 17 * d, dtype=torch.uint8, device=DEV))
        else:
            live = torch.ones(pages * page, dtype=torch.bool, device=DEV)
            s.update(cache=_pack(case, pages, *_contents(case, g, pages, live)))
        return s
    a = _attention_inputs(case, seed)
    cache = _pack(case, a["pages"], *_contents(case, a["g"], a["pages"], a["live"].reshape(-1)))
    hq, d = case["hq"], case["d"]
    s.update(cache=cache, q=a["qkv"][:, :hq], q_max=case["q"], cu=a["cu"], lens=a["lens"], table=a["table"], pages=a["pages"], width=a["width"],
             total=a["total"], scale=1.0 / math.sqrt(d), out=torch.empty(a["total"], hq, d, dtype=torch.bfloat16, device=DEV),
             lse=torch.empty(a["total"], hq, dtype=torch.float32, device=DEV),
             ws=torch.zeros(WORKSPACE, dtype=torch.uint8, device=DEV))
    return s


# ---------------------------------------------------------------------------
# the library's operators

def _own(s):
    import mxfp4_a4w4_gemm_gb300 as lib

    if s["op"] == "plan":
        lib.a4w4_kv_plan(s["past"], s["new"], s["b"], s["page"], s["table"], s["width"], s["ring"], s["pages"], s["state"],
                         s["state_out"], s["kv_lens"], s["cu"], s["slots"], s["positions"], s["tokens"], s["refused"])
        return {k: s[k] for k in ("table", "ring", "state_out", "kv_lens", "cu", "slots", "positions", "refused")}
    if s["op"] in ("append", "read"):
        if s["op"] == "append":
            lib.a4w4_kv_append(s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["slots"], s["t"], s["hkv"], s["d"],
                               s["cache"], s["pages"], s["page"])
        lib.a4w4_kv_read(s["cache"], s["pages"], s["page"], s["slots"], s["t"], s["hkv"], s["d"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    lib.a4w4_kv_attention(s["q"], s["q"].stride(0), s["cu"], s["b"], s["total"], s["q_max"], s["lens"], s["table"], s["width"],
                          s["cache"], s["pages"], s["page"], s["hq"], s["hkv"], s["d"], s["scale"], s["out"], s["lse"],
                          s["ws"], s["ws"].numel())
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------------------
# the plain form

def _plain_plan(s):
    page, width, size, n = s["page"], s["width"], s["pages"], s["tokens"]
    past, new = s["past"].long(), s["new"].long()
    head, count = s["state"][0].long(), s["state"][1].long()
    held = (past + page - 1) // page
    want = new.clamp(min=0) * (past + new <= width * page)  # a request longer than its table row is refused by itself
    need = (past + want + page - 1) // page - held
    fits = (torch.cumsum(need, 0) <= count) & (torch.cumsum(want, 0) <= n)  # the first that does not fit, and all after it, wait
    take, need = want * fits, need * fits
    cu = torch.cat([torch.zeros_like(take[:1]), torch.cumsum(take, 0)])
    first = torch.cumsum(need, 0) - need  # place among the popped pages
    gone = torch.where(new < 0, held, torch.zeros_like(held))
    given = torch.cumsum(gone, 0) - gone
    col = torch.arange(width, device=DEV)[None]
    grown = (col >= held[:, None]) & (col < (held + need)[:, None])
    popped = s["ring"][((head + first[:, None] + col - held[:, None]) % size).clamp(min=0)]
    ring = s["ring"].clone()
    back = (col < gone[:, None])
    ring[((head + count + given[:, None] + col) % size)[back]] = s["table"][back]
    table = torch.where(grown, popped, s["table"])
    tok = torch.arange(n, device=DEV)
    req = torch.searchsorted(cu, tok, right=True).sub(1).clamp(max=past.numel() - 1)
    pos = past[req] + tok - cu[req]
    inside = tok < cu[-1]
    slot = table[req, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    return {"table": table, "ring": ring,
            "state_out": torch.stack([(head + need.sum()) % size, count - need.sum() + gone.sum()]).int(),
            "kv_lens": torch.where(new < 0, torch.zeros_like(past), past + take).int(), "cu": cu.int(),
            "slots": torch.where(inside, slot, torch.full_like(slot, -1)).int(),
            "positions": torch.where(inside, pos, torch.zeros_like(pos)).int(),
            "refused": ((new > 0) & (take == 0)).sum().view(1).int()}


def _values(codes, scales):
    """Packed code bytes [..., n/2] and scale bytes [..., n/32] -> float32 [..., n]."""
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=DEV)
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    e = scales.float()
    return lut[nib.int()] * torch.where(e == 255, torch.nan, torch.exp2(e - 127.0)).repeat_interleave(32, -1)


def _plain_rows(s):
    page, d = s["page"], s["d"]
    kc, ks, vc, vs = _places(d)
    ok = s["slots"] >= 0
    slot = s["slots"].clamp(min=0).long()
    pg, ch, r = slot // page, slot % page // 16, slot % 16
    heads = torch.arange(s["hkv"], device=DEV)[None, :, None]
    cache = s["cache"]
    ix = lambda where, keep: (pg[keep, None, None], heads, ch[keep, None, None], where[r[keep]][:, None, :])  # noqa: E731
    if s["op"] == "append":
        c, e = _cells(s["k"])
        cache[ix(kc, ok)] = (c[..., 0::2] | c[..., 1::2] << 4)[ok]
        cache[ix(ks, ok)] = e[ok]
        c, e = _cells(s["v"])
        cache[ix(vc, ok)] = (c[..., 0::2] | c[..., 1::2] << 4)[ok]
        cache[ix(vs, ok)] = e[ok]
    every = torch.ones_like(ok)
    k = _values(cache[ix(kc, every)], cache[ix(ks, every)])
    v = _values(cache[ix(vc, every)], cache[ix(vs, every)])
    zero = ~ok[:, None, None]
    return {"k": k.masked_fill(zero, 0.0).bfloat16(), "v": v.masked_fill(zero, 0.0).bfloat16()}


def _plain_attention(s):
    b, q, hq, hkv, d, page = s["b"], s["q_max"], s["hq"], s["hkv"], s["d"], s["page"]
    kc, ks, vc, vs = _places(d)
    lens, cu = s["lens"].long(), s["cu"].long()
    n = s["width"] * page
    got = s["cache"][s["table"].long()].permute(0, 2, 1, 3, 4).flatten(2, 3)  # [b, hkv, chunks, bytes]
    k = _values(got[..., kc.reshape(-1)].reshape(b, hkv, n, d // 2), got[..., ks.reshape(-1)].reshape(b, hkv, n, d // 32))
    v = _values(got[..., vc.reshape(-1)].reshape(b, hkv, n, d // 2), got[..., vs.reshape(-1)].reshape(b, hkv, n, d // 32))
    key = torch.arange(n, device=DEV)
    v = v.masked_fill((key >= lens[:, None])[:, None, :, None], 0.0)
    i = torch.arange(q, device=DEV)[None]
    new = (cu[1:] - cu[:-1])[:, None]
    row = (cu[:-1, None] + i).clamp(max=max(s["total"] - 1, 0))
    x = s["q"][row].float().view(b, q, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [b, hkv, group * q, d]
    seen = (lens[:, None] - new + i + 1).clamp(min=0)  # keys that query i of the request sees
    dark = (key >= seen[..., None])[:, None, None]  # [b, 1, 1, q, n]
    z = (x @ k.transpose(-1, -2)).mul_(s["scale"]).view(b, hkv, -1, q, n).masked_fill_(dark, -torch.inf)
    top = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = z.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hkv, -1, n) @ v).view(b, hkv, -1, q, d) / total.clamp(min=1e-38)
    lse = torch.where(total > 0, top + total.log(), -torch.inf)
    mine = i < new
    back = lambda t: t.permute(0, 3, 1, 2, 4).flatten(2, 3)[mine]  # noqa: E731
    return {"out": back(o).bfloat16(), "lse": back(lse)[..., 0]}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "plan":
        return _plain_plan(s)
    return _plain_attention(s) if s["op"] == "attention" else _plain_rows(s)


# ---------------------------------------------------------------------------
# work, and the definition in 64 bits

def work(case):
    if case["op"] == "plan":
        b, t = case["b"], case["b"] * case["new"] + 8
        return {"bytes": 4 * (4 * b + 2 * t), "flops": 4 * t}
    cell = lambda d: 2 * (d // 2 + d // 32)  # noqa: E731  a key row and a value row of one head
    if case["op"] in ("append", "read"):
        n = case["t"] * case["hkv"]
        both = n * (2 * 2 * case["d"] + cell(case["d"])) + 4 * case["t"]
        return {"bytes": 2 * both if case["op"] == "append" else both, "flops": 4 * n * case["d"]}
    b, q, kv, hq, hkv, d = (case[k] for k in ("b", "q", "kv", "hq", "hkv", "d"))
    share = 0.5 if case["ragged"] and b > 1 else 1.0
    rows = b * q * share if q > 1 else b
    keys = kv * share
    seen = max(keys - q * share / 2, keys / 2)
    return {"bytes": b * keys * hkv * cell(d) + rows * hq * (4 * d + 4), "flops": 4 * rows * hq * seen * d}


def _wide(codes, scales):
    mag = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[(codes & 7).long()]
    return torch.where(codes > 7, -mag, mag) * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    if case["op"] == "append":
        s = prepare(case, seed)
        got = {}
        for name in ("k", "v"):
            x = s[name].double().unflatten(-1, (-1, 32))
            top = x.abs().amax(-1, keepdim=True)
            exp = torch.frexp(top).exponent - 3  # top = m 2^exponent with m in [1/2, 1): floor(log2 top) - 2
            unit = torch.ldexp(torch.ones_like(top), exp.clamp(min=-127))
            y = (x.abs() / unit).clamp(max=6.0)
            # steps of 1/2 below 2, of 1 below 4, of 2 above; torch.round takes ties to even, as the codes do
            step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0)).double()
            z = torch.round(y / step) * step * unit * torch.sign(x)
            got[name] = z.flatten(-2) * (s["slots"] >= 0).view(-1, 1, 1)
        return got
    if case["op"] == "read":
        g, pages, slots = _rows_inputs(case, seed)
        live = torch.ones(pages * case["page"], dtype=torch.bool, device=DEV)
        kc, ks, vc, vs = _contents(case, g, pages, live)
        at, ok = slots.clamp(min=0).long(), (slots >= 0).view(-1, 1, 1)
        return {"k": _wide(kc[at], ks[at]) * ok, "v": _wide(vc[at], vs[at]) * ok}
    a = _attention_inputs(case, seed)
    kc, ks, vc, vs = _contents(case, a["g"], a["pages"], a["live"].reshape(-1))
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    out = torch.zeros(a["total"], hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((a["total"], hq), -torch.inf, dtype=torch.float64, device=DEV)
    lens, cu = a["lens"].tolist(), a["cu"].tolist()
    for r in range(case["b"]):
        n, m = lens[r], cu[r + 1] - cu[r]
        if n == 0 or m == 0:
            continue
        tok = torch.arange(n, device=DEV)
        at = a["table"][r].long()[tok // page] * page + tok % page
        for h in range(hkv):
            k, v = _wide(kc[at, h], ks[at, h]), _wide(vc[at, h], vs[at, h])
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                z = a["qkv"][cu[r]: cu[r + 1], j].double() @ k.T / math.sqrt(d)
                ends = n - m + torch.arange(m, device=DEV)[:, None]
                z.masked_fill_(tok[None] > ends, -torch.inf)
                l = torch.logsumexp(z, -1)
                p = torch.exp(z - torch.where(l.isinf(), torch.zeros_like(l), l)[:, None])
                out[cu[r]: cu[r + 1], j] = p @ v
                lse[cu[r]: cu[r + 1], j] = l
    return {"out": out, "lse": lse}
