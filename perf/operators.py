"""Measured operators of a serving step over a paged cache held in 4 bits: block tables and slot
maps from request lengths, rotary positions with several axes joined to the cache append, and the
attention of ragged windows that reads the cache.

Where ``own`` is false, run() computes them from elementary torch operations in 32 bits (angles
and the choice of codes in 64); where it is true, it calls the package's entry points.  Both read
and write the same page bytes:

* a page holds ``page_size`` positions (a multiple of 16) of every kv head, [page][kv head][units
  of 16 positions][2304 bytes];
* a unit is K codes [4 blocks of 32 dimensions][16 positions][16 bytes] (dimension 2b of the block
  in the low nibble of byte b, 2b + 1 in the high one), V codes [64][16 bytes] (row d holds
  dimension d in the low nibbles and d + 64 in the high ones; position 4k + j at byte
  4k + (0, 2, 1, 3)[j]), K scales fp16 [16 positions][4 blocks], V scales fp16 [4 blocks][16];
* the value of code c is d * (c - 8), d one scale per 32 dimensions of a position with eight
  significant bits.
"""
import random

import numpy as np
import torch

own = False

D = 128          # head dimension
UNIT = 2304      # bytes of 16 positions of one kv head
V_BYTE = (0, 2, 1, 3)


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # a verify window of four tokens for eight requests: what every decode step pays
        {"name": "tables-decode", "op": "tables", "R": 8, "ctx": 32768, "page": 16, "new": 4, "ragged": False},
        # a busy server: windows of one to eight tokens for 256 requests of up to 32K
        {"name": "tables-serve", "op": "tables", "R": 256, "ctx": 32768, "page": 64, "new": 8, "ragged": True},
        # prompts arriving: up to 2048 new tokens for each of 48 requests, up to 128K each
        {"name": "tables-prompts", "op": "tables", "R": 48, "ctx": 131072, "page": 32, "new": 2048, "ragged": True},
        # one window of four text tokens after the q|k|v product of the 27B-shaped stack
        {"name": "append-window", "op": "append", "T": 4, "Hq": 40, "Hkv": 8, "page": 16, "axes": 1, "pairs": 64,
         "interleaved": False, "type": "f32"},
        # 64 windows of four tokens, positions in time, height and width
        {"name": "append-batch", "op": "append", "T": 256, "Hq": 40, "Hkv": 8, "page": 64, "axes": 3, "pairs": 64,
         "interleaved": False, "type": "f32"},
        # a prompt chunk with images, activations in bf16, rotary on half of each head
        {"name": "append-chunk", "op": "append", "T": 4099, "Hq": 32, "Hkv": 8, "page": 32, "axes": 3, "pairs": 32,
         "interleaved": True, "type": "bf16"},
        # a single token of one short request: latency
        {"name": "attend-token", "op": "attend", "R": 1, "ctx": 1500, "Hq": 40, "Hkv": 8, "page": 16, "new": 1,
         "ragged": False, "out": "bf16"},
        # the 27B-shaped window at 32K
        {"name": "attend-32k", "op": "attend", "R": 1, "ctx": 32768, "Hq": 40, "Hkv": 8, "page": 64, "new": 4,
         "ragged": False, "out": "bf16"},
        # the same at 262K, where the cache outweighs the weights
        {"name": "attend-262k", "op": "attend", "R": 1, "ctx": 262144, "Hq": 40, "Hkv": 8, "page": 128, "new": 4,
         "ragged": False, "out": "bf16"},
        # plain decoding of many short requests, small pages
        {"name": "attend-short", "op": "attend", "R": 200, "ctx": 2001, "Hq": 32, "Hkv": 8, "page": 16, "new": 1,
         "ragged": False, "out": "f32"},
        # ragged windows of 64 requests of up to 16K
        {"name": "attend-serve", "op": "attend", "R": 64, "ctx": 16384, "Hq": 40, "Hkv": 8, "page": 32, "new": 4,
         "ragged": True, "out": "bf16"},
        # two prompt chunks of 512 tokens behind 8K of cache
        {"name": "attend-chunk", "op": "attend", "R": 2, "ctx": 8704, "Hq": 40, "Hkv": 8, "page": 64, "new": 512,
         "ragged": False, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("tables", "append", "attend", "attend"))
    page = rng.choice((16, 32, 64, 128))
    heads = rng.choice(((40, 8), (32, 8), (16, 16), (8, 1), (24, 4), (12, 2)))
    if op == "tables":
        R = _log(rng, 1, 1024)
        ctx = _log(rng, 200, min(131072, (1 << 23) // R * page // 64))
        new = rng.choice((1, 4, 8, _log(rng, 9, 2048)))
        if R * new > 98304:
            new = max(1, 98304 // R)
        return {"op": op, "R": R, "ctx": max(ctx, new + 1), "page": page, "new": new, "ragged": rng.random() < 0.7}
    if op == "append":
        axes = rng.choice((1, 3, 3))
        return {"op": op, "T": _log(rng, 1, 4096), "Hq": heads[0], "Hkv": heads[1], "page": page, "axes": axes,
                "pairs": rng.choice((64, 64, 32, 16)), "interleaved": rng.random() < 0.4,
                "type": rng.choice(("f32", "bf16"))}
    R = _log(rng, 1, 256)
    ctx = _log(rng, 17, min(262144, (1 << 23) // (R * heads[1])))
    new = rng.choice((1, 2, 3, 4, 5, 8, _log(rng, 9, 400)))
    new = max(1, min(new, ctx, (1 << 28) // (R * ctx * heads[0])))
    return {"op": op, "R": R, "ctx": ctx, "Hq": heads[0], "Hkv": heads[1], "page": page, "new": new,
            "ragged": rng.random() < 0.6, "out": rng.choice(("bf16", "bf16", "f32"))}


def _lens(case):
    """Cache lengths (the new tokens counted) and new tokens of every request: the case's alone."""
    rng = random.Random(case["R"] * 1000003 + case["ctx"] * 31 + case["new"])
    R, ctx, new = case["R"], case["ctx"], case["new"]
    n = [rng.randint(1, new) if case["ragged"] else new for _ in range(R)]
    lens = [max(rng.randint(max(1, ctx // 8), ctx), n[r]) for r in range(R)]
    lens[0] = ctx
    return lens, n


def work(case):
    if case["op"] == "tables":
        lens, n = _lens(case)
        pages = sum(-(-(x + case["new"]) // case["page"]) for x in lens)
        # each held page id read and written once, the pool's free ids, slots and positions
        return {"bytes": 8.0 * pages + 8.0 * (pages // 4) + 12.0 * sum(n) + 28.0 * case["R"], "flops": 0}
    if case["op"] == "append":
        T, Hq, Hkv = case["T"], case["Hq"], case["Hkv"]
        b = 4 if case["type"] == "f32" else 2
        read = T * (Hq + 2 * Hkv) * D * b + T * (4 * case["axes"] + 8)
        wrote = T * Hq * D * 2 + T * Hkv * 144 + T * 2 * Hkv * D * 4
        return {"bytes": float(read + wrote), "flops": 3.0 * T * (Hq + Hkv) * 2 * case["pairs"]}
    lens, n = _lens(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    b = 2 if case["out"] == "bf16" else 4
    seen = sum(c * (x - c) + c * (c + 1) // 2 for x, c in zip(lens, n))
    cache = sum(lens) * Hkv * 144 + 4 * sum(-(-x // case["page"]) for x in lens)
    return {"bytes": float(cache + sum(n) * Hq * D * (2 + b)), "flops": 4.0 * D * Hq * seen}


# ---- page bytes --------------------------------------------------------------------------------
def _quantise(x):
    """Blocks of 32 along the last dimension: (codes uint8, scales fp16).  d is minus an eighth of
    the value of largest magnitude (the lowest dimension on ties), rounded to eight significant
    bits; c = x / d + 8 rounded half up, in 0..15.  What is not a number counts as 0, and
    magnitudes end at 65280 (where -8 d still fits fp16)."""
    b = torch.nan_to_num(x, nan=0.0, posinf=65280.0, neginf=-65280.0).clamp(-65280.0, 65280.0)
    b = b.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    mag = b.abs()
    at = torch.arange(32, device=x.device)
    first = torch.where(mag == mag.amax(-1, keepdim=True), at, 32).amin(-1, keepdim=True)
    frac, e = torch.frexp(b.gather(-1, first) * -0.125)
    d = torch.ldexp((frac * 256.0).round(), e - 8).to(torch.float16)
    df = d.to(b.dtype)
    ratio = torch.where(df != 0, b / df, torch.zeros_like(b))
    c = (ratio + 8.5).floor().clamp(0, 15).to(torch.uint8)
    return c.reshape(x.shape), d.squeeze(-1)


def _parts(pages, Hkv, page):
    """The four parts of every unit as views of the page bytes: K codes [N, Hkv, U, 4, 16, 16], V
    codes [N, Hkv, U, 64, 16], K scales [N, Hkv, U, 16, 4], V scales [N, Hkv, U, 4, 16]."""
    u = pages.view(-1, Hkv, page // 16, UNIT)
    half = u.view(torch.float16)
    return (u[..., :1024].unflatten(-1, (4, 16, 16)), u[..., 1024:2048].unflatten(-1, (64, 16)),
            half[..., 1024:1088].unflatten(-1, (16, 4)), half[..., 1088:].unflatten(-1, (4, 16)))


def _v_perm(device):
    p = torch.arange(16, device=device)
    return (p // 4) * 4 + torch.tensor(V_BYTE, device=device)[p % 4]


def _units(k, v):
    """fp32 [..., 16 positions, 128] keys and values -> unit bytes [..., 2304]."""
    kc, kd = _quantise(k)
    vc, vd = _quantise(v)
    kb = kc[..., 0::2] | (kc[..., 1::2] << 4)                       # [..., 16, 64]
    kb = kb.unflatten(-1, (4, 16)).transpose(-3, -2)                # [..., 4, 16, 16]
    vb = (vc[..., :64] | (vc[..., 64:] << 4)).transpose(-2, -1)     # [..., 64, 16]
    vb = vb[..., torch.argsort(_v_perm(k.device))]
    lead = k.shape[:-2]
    return torch.cat([kb.reshape(*lead, 1024), vb.reshape(*lead, 1024),
                      kd.contiguous().view(torch.uint8).reshape(*lead, 128),
                      vd.transpose(-2, -1).contiguous().view(torch.uint8).reshape(*lead, 128)], -1)


def _random_pages(n_pages, Hkv, page, g, dev):
    """A pool of pages that holds N(0, 1) keys and values, some key dimensions larger."""
    pages = torch.empty(n_pages * Hkv * (page // 16), UNIT, dtype=torch.uint8, device=dev)
    loud = torch.ones(D, device=dev)
    loud[5::32] = 3.0
    step = 1 << 14
    for i in range(0, pages.shape[0], step):
        n = min(step, pages.shape[0] - i)
        k = torch.randn(n, 16, D, generator=g, device=dev) * loud
        pages[i:i + n] = _units(k, torch.randn(n, 16, D, generator=g, device=dev))
    return pages.view(-1)


# ---- inputs ------------------------------------------------------------------------------------
def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case, "keep": {}}
    if case["op"] == "tables":
        R, page, new = case["R"], case["page"], case["new"]
        lens, n = _lens(case)
        rng = random.Random(int(seed) * 7919 + 13)
        before = [rng.randint(1, min(new, x)) if new <= 64 else 0 for x in lens]  # the last window
        kept = [rng.randint(1, b) if b else 0 for b in before]                   # of it, accepted
        held = torch.tensor(lens, device=dev)
        have = (held + page - 1) // page
        width = -(-(case["ctx"] + new) // page)
        total = int(have.sum())
        n_pages = total + max(total // 4, R * -(-new // page) + 8)
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
        table[torch.arange(width, device=dev) < have[:, None]] = order[:total]
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        free[:n_pages - total] = order[total:]
        tokens = R * new
        s |= {"held": held.to(torch.int32), "window": _i32(before, dev), "emitted": _i32(kept, dev),
              "new": _i32(n, dev), "table": table, "free": free, "n_free": _i32([n_pages - total], dev),
              "width": width, "n_pages": n_pages, "tokens": tokens}
        s["out"] = {"table": torch.empty_like(table), "free": torch.empty_like(free),
                    "n_free": torch.empty(1, dtype=torch.int32, device=dev),
                    "kv_len": torch.empty(R, dtype=torch.int32, device=dev),
                    "q_start": torch.empty(R + 1, dtype=torch.int32, device=dev),
                    "slots": torch.empty(tokens, dtype=torch.int64, device=dev),
                    "positions": torch.empty(tokens, dtype=torch.int32, device=dev),
                    "status": torch.empty(R, dtype=torch.int32, device=dev)}
        return s
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    if case["op"] == "append":
        T, axes, pairs = case["T"], case["axes"], case["pairs"]
        kind = torch.float32 if case["type"] == "f32" else torch.bfloat16
        qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=dev)
        qkv.view(T, -1, D)[:, Hq:Hq + Hkv, 5::32] *= 3.0
        n_pages = -(-T // page) + 8
        # tokens follow each other in pages that lie anywhere, from inside the first one on
        order = torch.randperm(n_pages, generator=g, device=dev)
        at = torch.arange(T, device=dev) + int(seed) % min(page, 8)
        slots = order[at // page] * page + at % page
        start = 200000 if seed % 2 else 1000
        text = start + torch.arange(T, device=dev)
        pos = text.repeat(axes, 1)
        if axes == 3 and T > 8:  # an image of 24 tokens a row after the first tokens
            i = torch.arange(T - 8, device=dev)
            pos[0, 8:], pos[1, 8:], pos[2, 8:] = start + 8, start + 8 + i // 24, start + 8 + i % 24
        inv = [10000000.0 ** (-i / pairs) for i in range(pairs)]
        axis = [0] * pairs if axes == 1 else [0 if i < pairs // 4 else 1 if i < 5 * pairs // 8 else 2 for i in range(pairs)]
        s |= {"qkv": qkv.to(kind), "slots": slots, "positions": pos.to(torch.int32).contiguous(), "inv": inv, "axis": axis,
              "inv_d": torch.tensor(inv, dtype=torch.float64, device=dev), "axis_d": torch.tensor(axis, device=dev),
              "pages": torch.zeros(n_pages * Hkv * (page // 16) * UNIT, dtype=torch.uint8, device=dev), "n_pages": n_pages,
              "q": torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev),
              "k": torch.empty(T, Hkv, D, dtype=torch.float32, device=dev),
              "v": torch.empty(T, Hkv, D, dtype=torch.float32, device=dev)}
        return s
    R = case["R"]
    lens, n = _lens(case)
    have = [-(-x // page) for x in lens]
    width, total = max(have), sum(have)
    n_pages = total + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
    table[torch.arange(width, device=dev) < torch.tensor(have, device=dev)[:, None]] = order[:total]
    T = sum(n)
    starts = [0]
    for c in n:
        starts.append(starts[-1] + c)
    q = torch.randn(T, Hq, D, generator=g, device=dev) * 1.5
    s |= {"q": q.to(torch.bfloat16), "pages": _random_pages(n_pages, Hkv, page, g, dev), "n_pages": n_pages, "table": table,
          "width": width, "kv_len": _i32(lens, dev), "q_start": _i32(starts, dev), "T": T, "most": max(n),
          "out": torch.empty(T, Hq, D, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=dev)}
    return s


# ---- plain forms -------------------------------------------------------------------------------
def _plain_tables(s):
    page, width, n_pages, most = s["case"]["page"], s["width"], s["n_pages"], s["tokens"]
    held, window, emitted, new = (s[k].long() for k in ("held", "window", "emitted", "new"))
    table, R = s["table"], s["case"]["R"]
    keep = held - window + emitted
    size = keep + new
    p0, p1 = (held + page - 1) // page, (size + page - 1) // page
    bad = (window < 0) | (emitted < 0) | (emitted > window) | (window > held) | (new < 0) | (p0 > width) | (p1 > width)
    ask = torch.where(bad, 0, new)
    full = ~bad & (ask > 0) & (ask.cumsum(0) > most)
    out = bad | full
    take = torch.where(out, 0, (p1 - p0).clamp(min=0))
    give = torch.where(out, 0, (p0 - p1).clamp(min=0))
    n_free = s["n_free"].long().clamp(0, n_pages)
    top = n_free + give.sum()
    none = (take > 0) & (take.cumsum(0) > top)
    ok = ~(out | none)
    granted = torch.where(ok, new, 0)
    first = take.cumsum(0) - take
    take = torch.where(none, 0, take)
    col = torch.arange(width, device=table.device)
    # the stack of free pages: what was free, then what is given back, in request and page order
    stack = torch.cat([s["free"], torch.zeros(R * width, dtype=torch.int32, device=table.device)])
    back = (col >= p1[:, None]) & (col < p0[:, None]) & ok[:, None]
    where = n_free + (give.cumsum(0) - give)[:, None] + col - p1[:, None]
    stack[where[back]] = table[back]
    q1 = torch.where(ok, p1, p0)
    got = stack[(top - 1 - first[:, None] - (col - p0[:, None])).clamp(0, stack.numel() - 1)]
    t = torch.where(col < torch.minimum(p0, q1)[:, None], table, torch.where(col < q1[:, None], got, -1))
    t = torch.where(bad[:, None], table, t).to(torch.int32)
    left = top - take.sum()
    free = torch.where(torch.arange(n_pages, device=table.device) < left, stack[:n_pages], -1).to(torch.int32)
    kv_len = torch.where(ok, size, torch.where(bad, 0, keep))
    q_start = torch.cat([granted.new_zeros(1), granted.cumsum(0)])
    i = torch.arange(most, device=table.device)
    r = torch.searchsorted(q_start, i, right=True).clamp(max=R) - 1
    at = keep[r] + i - q_start[r]
    live = i < q_start[-1]
    slot = t[r, (at // page).clamp(0, width - 1)].long() * page + at % page
    status = 32 * bad + 64 * none + 128 * full
    return {"table": t, "free": free, "n_free": left.to(torch.int32).reshape(1), "kv_len": kv_len.to(torch.int32),
            "q_start": q_start.to(torch.int32), "slots": torch.where(live, slot, -1),
            "positions": torch.where(live, at, -1).to(torch.int32), "status": status.to(torch.int32)}


def _rotate(x, cos, sin, pairs, interleaved):
    """x [T, heads, 128]; cos and sin [T, 1, pairs].  What lies past the pairs stays as it is."""
    turned, rest = x[..., :2 * pairs], x[..., 2 * pairs:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :pairs], turned[..., pairs:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _plain_append(s):
    c = s["case"]
    T, Hq, Hkv, page, pairs = c["T"], c["Hq"], c["Hkv"], c["page"], c["pairs"]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    angle = s["positions"].double()[s["axis_d"]].t() * s["inv_d"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    q = _rotate(x[:, :Hq], cos.float(), sin.float(), pairs, c["interleaved"])
    # in 64 bits: a key or value next to the border of two codes goes to the right one
    kc, kd = _quantise(_rotate(x[:, Hq:Hq + Hkv].double(), cos, sin, pairs, c["interleaved"]))
    vc, vd = _quantise(x[:, Hq + Hkv:].double())
    kp, vp, ks, vs = _parts(s["pages"], Hkv, page)
    at, off = s["slots"] // page, s["slots"] % page
    unit, i = off // 16, off % 16
    byte = _v_perm(x.device)[i]
    kp[at, :, unit, :, i] = (kc[..., 0::2] | (kc[..., 1::2] << 4)).unflatten(-1, (4, 16))
    vp[at, :, unit, :, byte] = vc[..., :64] | (vc[..., 64:] << 4)
    ks[at, :, unit, i] = kd
    vs[at, :, unit, :, i] = vd
    # the values that the pages now hold for these tokens, read back
    kb, vb = kp[at, :, unit, :, i], vp[at, :, unit, :, byte]
    k = torch.stack([kb & 15, kb >> 4], -1).reshape(T, Hkv, 4, 32).float() - 8.0
    v = torch.cat([vb & 15, vb >> 4], -1).reshape(T, Hkv, 4, 32).float() - 8.0
    return {"q": q.to(torch.bfloat16), "k": (k * ks[at, :, unit, i].float()[..., None]).reshape(T, Hkv, D),
            "v": (v * vs[at, :, unit, :, i].float()[..., None]).reshape(T, Hkv, D)}


def _plain_attend(s):
    c = s["case"]
    R, Hq, Hkv, page, C = c["R"], c["Hq"], c["Hkv"], c["page"], s["most"]
    G, L = Hq // Hkv, s["width"] * page
    kp, vp, ks, vs = _parts(s["pages"], Hkv, page)
    t = s["table"].clamp(min=0).long()
    kb = kp[t]                                                      # [R, P, Hkv, U, 4, 16, 16]
    k = torch.stack([kb & 15, kb >> 4], -1).flatten(-2).float() - 8.0
    k = (k * ks[t].transpose(-2, -1)[..., None].float()).transpose(-3, -2)
    k = k.permute(0, 2, 1, 3, 4, 5, 6).reshape(R, Hkv, L, D)
    vb = vp[t][..., _v_perm(t.device)]                              # [R, P, Hkv, U, 64, 16]
    v = torch.cat([vb & 15, vb >> 4], -2).float() - 8.0             # [..., 128, 16]
    v = (v.unflatten(-2, (4, 32)) * vs[t][..., None, :].float()).flatten(-3, -2)
    v = v.transpose(-2, -1).permute(0, 2, 1, 3, 4, 5).reshape(R, Hkv, L, D)
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(C, device=t.device)
    token = (s["q_start"][:-1].long()[:, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].float()[token].view(R, C, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, C * G, D)
    sc = (q @ k.transpose(-2, -1)) * (D ** -0.5)
    see = s["kv_len"].long()[:, None] - n[:, None] + i              # last position seen
    mask = torch.arange(L, device=t.device) <= see[..., None]       # [R, C, L]
    sc = sc.view(R, Hkv, C, G, L).masked_fill(~mask[:, None, :, None], float("-inf"))
    top = sc.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (sc - top).exp()
    o = p.view(R, Hkv, C * G, L) @ v
    total = p.sum(-1).view(R, Hkv, C * G, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.view(R, Hkv, C, G, D).permute(0, 2, 1, 3, 4).reshape(R, C, Hq, D)
    at = torch.arange(s["T"], device=t.device, dtype=torch.int32)
    r = torch.searchsorted(s["q_start"], at, right=True) - 1
    return o[r, at.long() - s["q_start"][r].long()].to(s["out"].dtype)


# ---- the package's calls -----------------------------------------------------------------------
def _own_tables(s):
    from speculative_decoding_verify_06_gb300 import svd
    o = s["out"]
    svd.svd_paged_tables(s["held"], s["window"], s["emitted"], s["new"], s["case"]["R"], s["case"]["page"], s["table"],
                         s["width"], s["free"], s["n_free"], s["n_pages"], o["table"], o["free"], o["n_free"], o["kv_len"],
                         o["q_start"], o["slots"], o["positions"], s["tokens"], o["status"])
    return o


def _own_append(s):
    from speculative_decoding_verify_06_gb300 import svd
    c, keep = s["case"], s["keep"]
    if not keep:
        keep["rope"] = svd.Rope(s["inv"], s["axis"], c["axes"], c["interleaved"])
    T, Hq, Hkv, page = c["T"], c["Hq"], c["Hkv"], c["page"]
    svd.svd_paged_append(s["qkv"], (Hq + 2 * Hkv) * D, T, Hq, Hkv, s["slots"], s["pages"], page, s["n_pages"], s["q"],
                         rope=keep["rope"], positions=s["positions"], positions_ld=T,
                         dtype=svd.SVD_F32 if c["type"] == "f32" else svd.SVD_BF16)
    svd.svd_paged_read(s["slots"], T, Hkv, s["pages"], page, s["n_pages"], s["k"], s["v"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _own_attend(s):
    from speculative_decoding_verify_06_gb300 import svd
    c, keep = s["case"], s["keep"]
    if not keep:
        keep["ws"] = torch.zeros(svd.svd_paged_attention_workspace_bytes(c["Hq"], c["Hkv"], c["R"], s["most"]),
                                 dtype=torch.uint8, device=s["q"].device)
    svd.svd_paged_attention(s["q"], s["T"], s["kv_len"], s["q_start"], c["R"], s["most"], s["table"], s["width"], s["pages"],
                            c["page"], s["n_pages"], c["Hq"], c["Hkv"], D ** -0.5, s["out"],
                            svd.SVD_BF16 if c["out"] == "bf16" else svd.SVD_F32, keep["ws"])
    return s["out"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attend": _own_attend}[op](state)
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[op](state)


# ---- from the definitions, in 64 bits ----------------------------------------------------------
def _blocks64(x):
    """The values that blocks of 32 of x (float64, [..., 128]) stand for once held in 4 bits."""
    b = x.reshape(*x.shape[:-1], 4, 32)
    first = np.abs(b).argmax(-1, keepdims=True)
    m = np.take_along_axis(b, first, -1) / -8.0
    frac, e = np.frexp(m)
    d = np.ldexp(np.rint(frac * 256.0), e - 8).astype(np.float16).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.where(d != 0, np.floor(b / d + 8.5), 8.0).clip(0, 15)
    return (d * (c - 8.0)).reshape(x.shape)


def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        T, Hq, Hkv, pairs = case["T"], case["Hq"], case["Hkv"], case["pairs"]
        x = s["qkv"].double().cpu().numpy().reshape(T, Hq + 2 * Hkv, D)
        pos = s["positions"].cpu().numpy().astype(np.float64)
        turn = np.exp(1j * pos[np.array(s["axis"])].T * np.array(s["inv"]))[:, None]
        lo, hi = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if case["interleaved"] else (slice(0, pairs), slice(pairs, 2 * pairs))
        z = (x[:, :Hq + Hkv, lo] + 1j * x[:, :Hq + Hkv, hi]) * turn
        y = x[:, :Hq + Hkv].copy()
        y[..., lo], y[..., hi] = z.real, z.imag
        return {"q": y[:, :Hq].copy(), "k": _blocks64(y[:, Hq:]), "v": _blocks64(x[:, Hq + Hkv:])}
    lens, n = _lens(case)
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    raw = s["pages"].view(-1, Hkv, page // 16, UNIT)
    order = [4 * (p // 4) + V_BYTE[p % 4] for p in range(16)]
    out, at = [], 0
    for r, (size, c) in enumerate(zip(lens, n)):
        u = raw[s["table"][r, :-(-size // page)].long()].permute(1, 0, 2, 3).reshape(Hkv, -1, UNIT)
        kd = u[..., 2048:2176].contiguous().view(torch.float16).double().view(Hkv, -1, 16, 4)
        vd = u[..., 2176:].contiguous().view(torch.float16).double().view(Hkv, -1, 4, 16)
        kb = u[..., :1024].reshape(Hkv, -1, 4, 16, 16).permute(0, 1, 3, 2, 4)    # [h, u, pos, blk, byte]
        k = torch.empty(*kb.shape[:4], 32, dtype=torch.float64, device=u.device)
        k[..., 0::2], k[..., 1::2] = (kb % 16).double() - 8, (kb // 16).double() - 8
        k = (k * kd[..., None]).reshape(Hkv, -1, D)[:, :size]
        vb = u[..., 1024:2048].reshape(Hkv, -1, 64, 16)[..., order].permute(0, 1, 3, 2)   # [h, u, pos, 64]
        v = torch.cat([(vb % 16).double() - 8, (vb // 16).double() - 8], -1)
        v = (v.view(Hkv, -1, 16, 4, 32) * vd.transpose(-2, -1)[..., None]).reshape(Hkv, -1, D)[:, :size]
        q = s["q"][at:at + c].double().view(c, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
        sc = torch.einsum("hgcd,hld->hgcl", q, k) / D ** 0.5
        seen = torch.arange(size, device=u.device) <= size - c + torch.arange(c, device=u.device)[:, None]
        p = torch.softmax(torch.where(seen, sc, -torch.inf), -1)
        out.append(torch.einsum("hgcl,hld->chgd", p, v).reshape(c, Hq, D))
        at += c
    return torch.cat(out)
