"""Measured operators of a paged cache held in 8 bits with one scale for each block of tokens and head,
and of moving pages: the append with rotary positions, the attention of ragged windows that reads the
cache, and forking requests and compacting a pool (of 8-bit or 4-bit pages) with the copies of the pages.

Where ``own`` is false, run() computes them from elementary torch operations in 32 bits (angles and the
choice of codes in 64); where it is true, it calls the package's entry points.  Both read and write
the same page bytes:

* a page holds ``page_size`` positions (a multiple of 16) of every kv head, [page][kv head][units of 16
  positions][4112 bytes];
* a unit is K codes [16 positions][128 bytes] (the 16 bytes of dimensions 16c .. 16c + 15 at place
  c ^ (position % 8)), V codes [128 dimensions][16 positions], the scales of K and of V (fp32), 8 bytes of 0;
* a code is an 8-bit float with 4 exponent and 3 fraction bits, largest 448; its value is code * scale,
  the scale a power of two from 2^-64 to 2^7, one for the keys and one for the values of a unit;
* an append gives a unit whose first position it writes the smallest scale s that covers its new values
  (448 s >= every magnitude), and a unit with earlier positions the larger of that and the scale it has; codes of
  earlier positions are rounded again where the scale grew.
"""
import random

import numpy as np
import torch

own = False

D = 128            # head dimension
UNIT8 = 4112       # bytes of 16 positions of one kv head, 8 bits
UNIT4 = 2304       # the same in 4 bits: moved as bytes only
E_LO, E_HI = -64, 7


def _dev():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


# ---- cases -------------------------------------------------------------------------------------
def listed():
    return [
        # one window of four text tokens after the q|k|v product of the 27B-shaped stack
        {"name": "append8-window", "op": "append", "R": 1, "new": 4, "ragged": False, "ctx": 1003, "Hq": 40, "Hkv": 8, "page": 16,
         "axes": 1, "pairs": 64, "interleaved": False, "type": "f32"},
        # 64 windows of four tokens, positions in time, height and width
        {"name": "append8-batch", "op": "append", "R": 64, "new": 4, "ragged": False, "ctx": 700, "Hq": 40, "Hkv": 8, "page": 64,
         "axes": 3, "pairs": 64, "interleaved": False, "type": "f32"},
        # a prompt chunk with images, activations in bf16, rotary on half of each head
        {"name": "append8-chunk", "op": "append", "R": 1, "new": 4099, "ragged": False, "ctx": 5000, "Hq": 32, "Hkv": 8, "page": 32,
         "axes": 3, "pairs": 32, "interleaved": True, "type": "bf16"},
        # a single token of one short request: latency
        {"name": "attend8-token", "op": "attend", "R": 1, "ctx": 1500, "Hq": 40, "Hkv": 8, "page": 16, "new": 1,
         "ragged": False, "out": "bf16"},
        # the 27B-shaped window at 32K
        {"name": "attend8-32k", "op": "attend", "R": 1, "ctx": 32768, "Hq": 40, "Hkv": 8, "page": 64, "new": 4,
         "ragged": False, "out": "bf16"},
        # the same at 262K, where the cache outweighs the weights
        {"name": "attend8-262k", "op": "attend", "R": 1, "ctx": 262144, "Hq": 40, "Hkv": 8, "page": 128, "new": 4,
         "ragged": False, "out": "bf16"},
        # plain decoding of many short requests, small pages, the o product in 32 bits
        {"name": "attend8-short", "op": "attend", "R": 200, "ctx": 2001, "Hq": 32, "Hkv": 8, "page": 16, "new": 1,
         "ragged": False, "out": "f32"},
        # ragged windows of 64 requests of up to 16K
        {"name": "attend8-serve", "op": "attend", "R": 64, "ctx": 16384, "Hq": 40, "Hkv": 8, "page": 32, "new": 4,
         "ragged": True, "out": "bf16"},
        # two prompt chunks of 512 tokens behind 8K of cache
        {"name": "attend8-chunk", "op": "attend", "R": 2, "ctx": 8704, "Hq": 40, "Hkv": 8, "page": 64, "new": 512,
         "ragged": False, "out": "bf16"},
        # a search keeps one of two short requests and continues it twice, 4-bit pages: latency
        {"name": "fork-pair", "op": "fork", "R": 2, "each": 2, "ctx": 301, "page": 16, "Hkv": 8, "bits": 4, "layers": 2},
        # eight prompts of up to 4K answered eight times each, 8-bit pages
        {"name": "fork-samples", "op": "fork", "R": 64, "each": 8, "ctx": 4096, "page": 64, "Hkv": 8, "bits": 8, "layers": 2},
        # a pool two thirds empty after long requests ended: what is left moves to its start
        {"name": "compact-pool", "op": "compact", "R": 48, "ctx": 16384, "page": 32, "Hkv": 8, "bits": 4, "layers": 2},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("append", "append", "attend", "attend", "attend", "fork", "compact"))
    page = rng.choice((16, 32, 64, 128))
    heads = rng.choice(((40, 8), (32, 8), (16, 16), (8, 1), (24, 4), (12, 2)))
    if op == "append":
        R = _log(rng, 1, 256)
        new = rng.choice((1, 2, 4, 8, _log(rng, 9, 4096)))
        new = max(1, min(new, 4096 // R))
        axes = rng.choice((1, 3, 3))
        return {"op": op, "R": R, "new": new, "ragged": rng.random() < 0.6, "ctx": new + _log(rng, 1, min(1000, 100000 // R)),
                "Hq": heads[0], "Hkv": heads[1], "page": page, "axes": axes, "pairs": rng.choice((64, 64, 32, 16)),
                "interleaved": rng.random() < 0.4, "type": rng.choice(("f32", "bf16"))}
    if op == "attend":
        R = _log(rng, 1, 256)
        ctx = _log(rng, 17, min(262144, (1 << 22) // (R * heads[1])))
        new = rng.choice((1, 2, 3, 4, 5, 8, _log(rng, 9, 400)))
        new = max(1, min(new, ctx, (1 << 28) // (R * ctx * heads[0])))
        return {"op": op, "R": R, "ctx": ctx, "Hq": heads[0], "Hkv": heads[1], "page": page, "new": new,
                "ragged": rng.random() < 0.6, "out": rng.choice(("bf16", "bf16", "f32"))}
    bits, layers = rng.choice((4, 8)), rng.choice((1, 2, 3))
    R = _log(rng, 2, 256)
    ctx = _log(rng, 17, max(18, min(16384, (1 << 21) // (R * heads[1] * layers))))
    if op == "fork":
        return {"op": op, "R": R, "each": rng.randint(2, min(R, 9)), "ctx": ctx, "page": page, "Hkv": heads[1], "bits": bits, "layers": layers}
    return {"op": op, "R": R, "ctx": ctx, "page": page, "Hkv": heads[1], "bits": bits, "layers": layers}


def _lens(case):
    """Cache lengths (the new tokens counted) and new tokens of every request: the case's alone."""
    rng = random.Random(case["R"] * 1000003 + case["ctx"] * 31 + case["new"])
    R, ctx, new = case["R"], case["ctx"], case["new"]
    n = [rng.randint(1, new) if case["ragged"] else new for _ in range(R)]
    lens = [max(rng.randint(max(1, ctx // 8), ctx), n[r]) for r in range(R)]
    lens[0] = ctx
    return lens, n


def _shares(case):
    """Of a fork or a compaction: lengths held, last windows, their tokens kept, and every request's
    parent (-1: it stays)."""
    R, ctx = case["R"], case["ctx"]
    rng = random.Random(R * 1000003 + ctx * 31 + case["page"])
    held = [rng.randint(max(1, ctx // 2 if case["op"] == "fork" else ctx // 8), ctx) for _ in range(R)]
    held[0] = ctx
    window = [rng.randint(0, min(4, h)) for h in held]
    kept = [rng.randint(1, w) if w else 0 for w in window]
    each = case.get("each", 1)
    parent = [-1 if r % each == 0 else r - r % each for r in range(R)]
    if case["op"] == "fork":  # what a request held that goes: mostly less than what its parent hands on
        held = [h if p < 0 else min(h, rng.randint(0, ctx)) for h, p in zip(held, parent)]
        window = [min(w, h) for w, h in zip(window, held)]
        kept = [min(k, w) for k, w in zip(kept, window)]
    return held, window, kept, parent


def _page_bytes(case):
    return case["Hkv"] * (case["page"] // 16) * (UNIT8 if case["bits"] == 8 else UNIT4)


def work(case):
    if case["op"] == "append":
        _, n = _lens(case)
        T, Hq, Hkv = sum(n), case["Hq"], case["Hkv"]
        b = 4 if case["type"] == "f32" else 2
        read = T * (Hq + 2 * Hkv) * D * b + T * 4 * case["axes"]
        wrote = T * Hq * D * 2 + T * Hkv * 257 + T * 2 * Hkv * D * 4
        return {"bytes": float(read + wrote), "flops": 3.0 * T * (Hq + Hkv) * 2 * case["pairs"]}
    if case["op"] == "attend":
        lens, n = _lens(case)
        Hq, Hkv = case["Hq"], case["Hkv"]
        b = 2 if case["out"] == "bf16" else 4
        seen = sum(c * (x - c) + c * (c + 1) // 2 for x, c in zip(lens, n))
        cache = sum(lens) * Hkv * 257 + 4 * sum(-(-x // case["page"]) for x in lens)
        return {"bytes": float(cache + sum(n) * Hq * D * (2 + b)), "flops": 4.0 * D * Hq * seen}
    held, window, kept, parent = _shares(case)
    page = case["page"]
    pages = [-(-h // page) for h in held]
    if case["op"] == "fork":
        need = [-(-(h - w + k) // page) for h, w, k in zip(held, window, kept)]
        wrote = sum(need[p] for p in parent if p >= 0)
        read = sum(need[p] for p in sorted({p for p in parent if p >= 0}))
    else:  # the pool is three times what is held: two of three held pages move
        wrote = read = sum(pages) * 2 // 3
    return {"bytes": float((read + wrote) * _page_bytes(case) * case["layers"] + 16 * sum(pages)), "flops": 0}


# ---- page bytes --------------------------------------------------------------------------------
def _pow2(e):
    """2^e in 64 bits, exactly (a power that a GPU computes need not be)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _table256(dev):
    """The values of the 256 codes (those of the two codes that are no numbers: 0)."""
    c = torch.arange(256, device=dev)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * _pow2(e - 7), m * 2.0 ** -9)
    v = torch.where((c & 127) == 127, 0.0, v)
    return torch.where(c > 127, -v, v)


def _encode(x):
    """float64 of magnitude up to 448 -> codes: to nearest, ties to even."""
    a = x.abs()
    _, e = torch.frexp(a)                                  # a = f 2^e, f in [1/2, 1)
    e = torch.where(a > 0, e - 1, -99).clamp(min=-6)
    n = (a * _pow2(3 - e)).round()                      # steps of 2^(e - 3)
    code = (n + 8 * (e + 6)).to(torch.uint8)               # (a carry into the next exponent counts itself)
    return code + 128 * torch.signbit(x).to(torch.uint8) * (code > 0)


def _exponent(top):
    """The smallest exponent e with 448 * 2^e >= top."""
    f, e = torch.frexp(top)                                # 448 = 0.875 * 2^9
    e = e - 9 + (f > 0.875).to(e.dtype)
    return torch.where(top > 0, e, E_LO).clamp(E_LO, E_HI)


def _clean(x):
    top = 448.0 * 2.0 ** E_HI
    return torch.nan_to_num(x, nan=0.0, posinf=top, neginf=-top).clamp(-top, top)


def _k_place(dev):
    """Byte of dimension d of position i: [16][128]."""
    i, d = torch.arange(16, device=dev)[:, None], torch.arange(D, device=dev)
    return i * D + (((d // 16) ^ (i % 8)) * 16) + d % 16


def _units(k, v):
    """float64 [..., 16 positions, 128] keys and values -> unit bytes [..., 4112]."""
    lead = k.shape[:-2]
    ek, ev = _exponent(k.abs().amax((-2, -1))), _exponent(v.abs().amax((-2, -1)))
    kc, vc = _encode(k * _pow2(-ek)[..., None, None]), _encode(v * _pow2(-ev)[..., None, None])
    u = torch.zeros(*lead, UNIT8, dtype=torch.uint8, device=k.device)
    u[..., _k_place(k.device).flatten()] = kc.flatten(-2)
    u[..., 2048:4096] = vc.transpose(-2, -1).flatten(-2)
    s = _pow2(torch.stack([ek, ev], -1)).float()
    u[..., 4096:4104] = s.contiguous().view(torch.uint8)
    return u


def _random_pages(n_pages, Hkv, page, g, dev):
    """A pool of pages that holds N(0, 1) keys and values, some key dimensions larger."""
    pages = torch.empty(n_pages * Hkv * (page // 16), UNIT8, dtype=torch.uint8, device=dev)
    loud = torch.ones(D, device=dev)
    loud[5::32] = 3.0
    step = 1 << 13
    for i in range(0, pages.shape[0], step):
        n = min(step, pages.shape[0] - i)
        k = torch.randn(n, 16, D, generator=g, device=dev) * loud
        pages[i:i + n] = _units(k.double(), torch.randn(n, 16, D, generator=g, device=dev).double())
    return pages.view(-1)


# ---- inputs ------------------------------------------------------------------------------------
def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def _rows(have, width, order, dev):
    """A table whose rows hold the first pages of `order`, one row after the other."""
    table = torch.full((len(have), width), -1, dtype=torch.int32, device=dev)
    table[torch.arange(width, device=dev) < torch.tensor(have, device=dev)[:, None]] = order[:sum(have)]
    return table


def prepare(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case, "keep": {}}
    page, Hkv, R = case["page"], case["Hkv"], case["R"]
    if case["op"] in ("fork", "compact"):
        held, window, kept, parent = _shares(case)
        have = [-(-h // page) for h in held]
        need = [have[r] if parent[r] < 0 else -(-(held[parent[r]] - window[parent[r]] + kept[parent[r]]) // page) for r in range(R)]
        total = sum(have)
        n_pages = 3 * total if case["op"] == "compact" else total + sum(max(0, b - a) for a, b in zip(have, need)) + 5
        width = -(-case["ctx"] // page) + 1
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        free = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        free[:n_pages - total] = order[total:]
        table = _rows(have, width, order, dev)
        nbytes = n_pages * _page_bytes(case)
        pools = [torch.randint(0, 256, (nbytes,), dtype=torch.uint8, generator=g, device=dev) for _ in range(case["layers"])]
        one = lambda *n: torch.empty(*n, dtype=torch.int32, device=dev)  # noqa: E731
        return s | {"held": _i32(held, dev), "window": _i32(window, dev), "emitted": _i32(kept, dev), "parent": _i32(parent, dev),
                    "table": table, "width": width, "free": free, "n_free": _i32([n_pages - total], dev), "n_pages": n_pages,
                    "pools": pools,
                    "out": {"table": one(R, width), "free": one(n_pages), "n_free": one(1), "held": one(R), "window": one(R),
                            "from": one(n_pages), "to": one(n_pages), "n": one(1), "status": one(R)}}
    lens, n = _lens(case)
    Hq, T = case["Hq"], sum(n)
    starts = [0]
    for c in n:
        starts.append(starts[-1] + c)
    have = [-(-x // page) for x in lens]
    width, n_pages = max(have), sum(have) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    s |= {"pages": _random_pages(n_pages, Hkv, page, g, dev), "n_pages": n_pages, "table": _rows(have, width, order, dev),
          "width": width, "kv_len": _i32(lens, dev), "q_start": _i32(starts, dev), "T": T, "most": max(n)}
    if case["op"] == "attend":
        q = torch.randn(T, Hq, D, generator=g, device=dev) * 1.5
        return s | {"q": q.to(torch.bfloat16),
                    "out": torch.empty(T, Hq, D, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=dev)}
    axes, pairs = case["axes"], case["pairs"]
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=dev)
    x = qkv.view(T, -1, D)
    x[:, Hq:Hq + Hkv, 5::32] *= 3.0
    # a few tokens louder than what the cache holds, so that scales of units grow
    x[:, Hq:] *= torch.where(torch.rand(T, 1, 1, generator=g, device=dev) < 0.1, 6.0, 1.0)
    at = [torch.arange(a - c, a, device=dev) for a, c in zip(lens, n)]
    text = torch.cat(at) + (200000 if seed % 2 else 1000)
    pos = text.repeat(axes, 1)
    if axes == 3 and case["new"] > 8:  # images of 24 tokens a row
        i = torch.arange(T, device=dev)
        pos[1], pos[2] = text[0] + i // 24, text[0] + i % 24
    inv = [10000000.0 ** (-i / pairs) for i in range(pairs)]
    axis = [0] * pairs if axes == 1 else [0 if i < pairs // 4 else 1 if i < 5 * pairs // 8 else 2 for i in range(pairs)]
    # what is read back: the new positions, and the earlier ones of their units
    first = [(a - c) // 16 * 16 for a, c in zip(lens, n)]
    r = torch.cat([torch.full((a - f,), j, device=dev) for j, (a, f) in enumerate(zip(lens, first))])
    p = torch.cat([torch.arange(f, a, device=dev) for a, f in zip(lens, first)])
    slots = s["table"][r, p // page].long() * page + p % page
    return s | {"qkv": qkv.to(torch.float32 if case["type"] == "f32" else torch.bfloat16), "positions": pos.to(torch.int32).contiguous(),
                "inv": inv, "axis": axis, "inv_d": torch.tensor(inv, dtype=torch.float64, device=dev),
                "axis_d": torch.tensor(axis, device=dev), "slots": slots,
                "q": torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev),
                "k": torch.empty(len(slots), Hkv, D, dtype=torch.float32, device=dev),
                "v": torch.empty(len(slots), Hkv, D, dtype=torch.float32, device=dev)}


# ---- plain forms -------------------------------------------------------------------------------
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
    T, Hq, Hkv, page, pairs, R = s["T"], c["Hq"], c["Hkv"], c["page"], c["pairs"], c["R"]
    dev = s["qkv"].device
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    angle = s["positions"].double()[s["axis_d"]].t() * s["inv_d"]
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    q = _rotate(x[:, :Hq], cos.float(), sin.float(), pairs, c["interleaved"])
    # in 64 bits: a key next to the border of two codes goes to the right one
    k = _rotate(x[:, Hq:Hq + Hkv].double(), cos, sin, pairs, c["interleaved"])
    both = _clean(torch.stack([k, x[:, Hq + Hkv:].double()], 2))              # [T, Hkv, 2, 128]
    # the units that get tokens, [R, U] of them, and each one's 16 places
    kv, q0 = s["kv_len"].long(), s["q_start"].long()
    n = q0[1:] - q0[:-1]
    begin = kv - n
    U = (s["most"] + 30) // 16
    pos = ((begin // 16) * 16)[:, None] + torch.arange(U * 16, device=dev)     # [R, U * 16]
    new = (pos >= begin[:, None]) & (pos < kv[:, None])
    at = (q0[:-1, None] + pos - begin[:, None]).clamp(0, T - 1)
    y = torch.where(new[..., None, None, None], both[at], 0.0).view(R, U, 16, Hkv, 2, D)
    new = new.view(R, U, 16)
    live, earlier = new.any(-1), pos.view(R, U, 16)[..., 0] < begin[:, None]
    col = (pos[:, ::16] // page).clamp(max=s["width"] - 1)
    which = s["table"].gather(1, col).long()
    units = s["pages"].view(-1, Hkv, page // 16, UNIT8)
    here = torch.where(live, which, 0), pos[:, ::16] % page // 16
    old = units[here[0], :, here[1]]                                           # [R, U, Hkv, 4112]
    kp = _k_place(dev)
    codes = torch.stack([old[..., kp], old[..., 2048:4096].unflatten(-1, (D, 16)).transpose(-2, -1)], -3)  # [R, U, Hkv, 2, 16, D]
    _, e0 = torch.frexp(old[..., 4096:4104].contiguous().view(torch.float32))  # [R, U, Hkv, 2]
    e0 = (e0 - 1).clamp(E_LO, E_HI)
    e = _exponent(y.abs().amax((2, -1)))
    e = torch.where(earlier[..., None, None], torch.maximum(e, e0), e)
    y = y.permute(0, 1, 3, 4, 2, 5)
    value = _table256(dev)[codes.long()]
    again = _encode(value * _pow2((e0 - e).clamp(max=0))[..., None, None])
    fresh = _encode(y * _pow2(-e)[..., None, None])
    is_new = new[:, :, None, None, :, None]
    before = (pos.view(R, U, 1, 1, 16, 1) < begin.view(R, 1, 1, 1, 1, 1)) & (e > e0)[..., None, None]
    codes = torch.where(is_new, fresh, torch.where(before, again, codes))
    out = old.clone()
    out[..., kp.flatten()] = codes[..., 0, :, :].flatten(-2)
    out[..., 2048:4096] = codes[..., 1, :, :].transpose(-2, -1).flatten(-2)
    out[..., 4096:4104] = _pow2(e).float().view(torch.uint8)
    units[here[0][live], :, here[1][live]] = out[live]
    # the values that the pages now hold
    held, off = s["slots"] // page, s["slots"] % page
    u, i = units[held, :, off // 16], off % 16
    scale = u[..., 4096:4104].contiguous().view(torch.float32)
    of = _table256(dev).float()
    kc = u.gather(-1, kp[i][:, None].expand(-1, Hkv, -1))
    vc = u.gather(-1, (2048 + torch.arange(D, device=dev) * 16 + i[:, None])[:, None].expand(-1, Hkv, -1))
    return {"q": q.to(torch.bfloat16), "k": of[kc.long()] * scale[..., :1], "v": of[vc.long()] * scale[..., 1:]}


def _plain_attend(s):
    c = s["case"]
    R, Hq, Hkv, page, C = c["R"], c["Hq"], c["Hkv"], c["page"], s["most"]
    G, L = Hq // Hkv, s["width"] * page
    dev = s["q"].device
    u = s["pages"].view(-1, Hkv, page // 16, UNIT8)[s["table"].clamp(min=0).long()]     # [R, P, Hkv, U, 4112]
    scale = u[..., 4096:4104].contiguous().view(torch.float32)
    value = _table256(dev).float()
    k = value[u[..., _k_place(dev)].int()] * scale[..., :1, None]
    k = k.permute(0, 2, 1, 3, 4, 5).reshape(R, Hkv, L, D)
    v = value[u[..., 2048:4096].int()].unflatten(-1, (D, 16)) * scale[..., 1:, None]
    v = v.transpose(-2, -1).permute(0, 2, 1, 3, 4, 5).reshape(R, Hkv, L, D)
    del u
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    i = torch.arange(C, device=dev)
    token = (s["q_start"][:-1].long()[:, None] + i).clamp(max=s["T"] - 1)
    q = s["q"].float()[token].view(R, C, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, C * G, D)
    sc = (q @ k.transpose(-2, -1)) * (D ** -0.5)
    see = s["kv_len"].long()[:, None] - n[:, None] + i              # last position seen
    mask = torch.arange(L, device=dev) <= see[..., None]            # [R, C, L]
    sc = sc.view(R, Hkv, C, G, L).masked_fill(~mask[:, None, :, None], float("-inf"))
    top = sc.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (sc - top).exp()
    o = p.view(R, Hkv, C * G, L) @ v
    total = p.sum(-1).view(R, Hkv, C * G, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.view(R, Hkv, C, G, D).permute(0, 2, 1, 3, 4).reshape(R, C, Hq, D)
    at = torch.arange(s["T"], device=dev, dtype=torch.int32)
    r = torch.searchsorted(s["q_start"], at, right=True) - 1
    return o[r, at.long() - s["q_start"][r].long()].to(s["out"].dtype)


def _listed_moves(src, dst, n_pages):
    """Page ids of the copies at the front of [n_pages] entries, -1 behind them."""
    pad = torch.full((n_pages,), -1, dtype=torch.int32, device=src.device)
    return torch.cat([src.int(), pad])[:n_pages], torch.cat([dst.int(), pad])[:n_pages]


def _move(s, src, dst):
    out = []
    for pool in s["pools"]:
        p = pool.view(s["n_pages"], -1)
        p[dst.long()] = p[src.long()]
        out.append(pool)
    return out


def _plain_fork(s):
    page, width, n_pages, R = s["case"]["page"], s["width"], s["n_pages"], s["case"]["R"]
    held, window, emitted, parent = (s[k].long() for k in ("held", "window", "emitted", "parent"))
    table, dev = s["table"], s["table"].device
    r = torch.arange(R, device=dev)
    win, emi = window.abs(), torch.where(window > 0, emitted, 0)
    keep = held - win + emi
    fine = (emi >= 0) & (emi <= win) & (win <= held) & (held <= width * page)
    child = (parent >= 0) & (parent != r)
    who = parent.clamp(0, R - 1)
    bad = child & ((parent >= R) | child[who] | ~fine[who] | (held < 0) | (held > width * page))
    go = child & ~bad
    p0 = (held + page - 1) // page
    p1 = torch.where(go, (keep[who] + page - 1) // page, p0)
    take, give = (p1 - p0).clamp(min=0), (p0 - p1).clamp(min=0)
    n_free = s["n_free"].long().clamp(0, n_pages)
    top = n_free + give.sum()
    none = (take > 0) & (take.cumsum(0) > top)
    first = take.cumsum(0) - take
    take = torch.where(none, 0, take)
    ok = go & ~none
    col = torch.arange(width, device=dev)
    stack = torch.cat([s["free"], torch.zeros(R * width, dtype=torch.int32, device=dev)])
    back = (col >= p1[:, None]) & (col < p0[:, None]) & ok[:, None]
    stack[(n_free + (give.cumsum(0) - give)[:, None] + col - p1[:, None])[back]] = table[back]
    got = stack[(top - 1 - first[:, None] - (col - p0[:, None])).clamp(0, stack.numel() - 1)]
    t = torch.where(col < torch.minimum(p0, p1)[:, None], table, torch.where(col < p1[:, None], got, -1))
    t = torch.where(ok[:, None], t, table).to(torch.int32)
    left = top - take.sum()
    free = torch.where(torch.arange(n_pages, device=dev) < left, stack[:n_pages], -1).to(torch.int32)
    use = ok[:, None] & (col < p1[:, None])
    src, dst = table[who][use], t[use]
    pools = _move(s, src, dst)
    a, b = _listed_moves(src, dst, n_pages)
    return {"table": t, "free": free, "n_free": left.to(torch.int32).reshape(1), "held": torch.where(ok, keep[who], held).to(torch.int32),
            "window": torch.where(ok, 0, window).to(torch.int32), "from": a, "to": b,
            "n": use.sum().to(torch.int32).reshape(1), "status": (32 * bad + 64 * (go & none)).to(torch.int32), "pools": pools}


def _plain_compact(s):
    page, width, n_pages = s["case"]["page"], s["width"], s["n_pages"]
    table, dev = s["table"], s["table"].device
    have = ((s["held"].long() + page - 1) // page).clamp(0, width)
    inside = torch.arange(width, device=dev) < have[:, None]
    live = inside & (table >= 0) & (table < n_pages)
    used = torch.zeros(n_pages, dtype=torch.bool, device=dev)
    used[table[live].long()] = True
    count = used.sum()
    ids = torch.arange(n_pages, device=dev)
    src, dst = ids[used & (ids >= count)], ids[~used & (ids < count)]
    to = ids.clone()
    to[src] = dst
    t = torch.where(live, to[table.clamp(0, n_pages - 1).long()], torch.where(inside, table.long(), -1)).to(torch.int32)
    left = n_pages - count
    free = torch.where(ids < left, n_pages - 1 - ids, -1).to(torch.int32)
    pools = _move(s, src, dst)
    a, b = _listed_moves(src, dst, n_pages)
    return {"table": t, "free": free, "n_free": left.to(torch.int32).reshape(1), "from": a, "to": b,
            "n": (used & (ids >= count)).sum().to(torch.int32).reshape(1), "pools": pools}


# ---- the package's calls -----------------------------------------------------------------------
def _own_append(s):
    from speculative_decoding_verify_06_gb300 import svd
    c, keep = s["case"], s["keep"]
    if not keep:
        keep["rope"] = svd.Rope(s["inv"], s["axis"], c["axes"], c["interleaved"])
    T, Hq, Hkv, page = s["T"], c["Hq"], c["Hkv"], c["page"]
    svd.svd_paged8_append(s["qkv"], (Hq + 2 * Hkv) * D, T, Hq, Hkv, s["kv_len"], s["q_start"], c["R"], s["table"], s["width"],
                          s["pages"], page, s["n_pages"], s["q"], rope=keep["rope"], positions=s["positions"], positions_ld=T,
                          dtype=svd.SVD_F32 if c["type"] == "f32" else svd.SVD_BF16)
    svd.svd_paged8_read(s["slots"], s["slots"].numel(), Hkv, s["pages"], page, s["n_pages"], s["k"], s["v"])
    return {"q": s["q"], "k": s["k"], "v": s["v"]}


def _own_attend(s):
    from speculative_decoding_verify_06_gb300 import svd
    c, keep = s["case"], s["keep"]
    if not keep:
        keep["ws"] = torch.zeros(svd.svd_paged8_attention_workspace_bytes(c["Hq"], c["Hkv"], c["R"], s["most"]),
                                 dtype=torch.uint8, device=s["q"].device)
    svd.svd_paged8_attention(s["q"], s["T"], s["kv_len"], s["q_start"], c["R"], s["most"], s["table"], s["width"], s["pages"],
                             c["page"], s["n_pages"], c["Hq"], c["Hkv"], D ** -0.5, s["out"],
                             svd.SVD_BF16 if c["out"] == "bf16" else svd.SVD_F32, keep["ws"])
    return s["out"]


def _own_pools(s):
    from speculative_decoding_verify_06_gb300 import svd
    if "pools" not in s["keep"]:
        s["keep"]["pools"] = svd.Pools(s["pools"], _page_bytes(s["case"]))
    return s["keep"]["pools"]


def _own_fork(s):
    from speculative_decoding_verify_06_gb300 import svd
    c, o, pools = s["case"], s["out"], _own_pools(s)
    svd.svd_paged_fork(s["held"], s["window"], s["emitted"], s["parent"], c["R"], c["page"], s["table"], s["width"], s["free"],
                       s["n_free"], s["n_pages"], o["held"], o["window"], o["table"], o["free"], o["n_free"], o["from"], o["to"],
                       o["n"], o["status"])
    svd.svd_paged_copy(pools, s["n_pages"], o["from"], o["to"], o["n"], s["n_pages"])
    return o | {"pools": s["pools"]}


def _own_compact(s):
    from speculative_decoding_verify_06_gb300 import svd
    c, o, pools = s["case"], s["out"], _own_pools(s)
    svd.svd_paged_compact(s["held"], c["R"], c["page"], s["table"], s["width"], s["n_pages"], o["table"], o["free"], o["n_free"],
                          o["from"], o["to"], o["n"])
    svd.svd_paged_copy(pools, s["n_pages"], o["from"], o["to"], o["n"], s["n_pages"])
    return {k: o[k] for k in ("table", "free", "n_free", "from", "to", "n")} | {"pools": s["pools"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "fork": _own_fork, "compact": _own_compact}[op](state)
    return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact}[op](state)


# ---- from the definitions, in 64 bits ----------------------------------------------------------
def _grid64(x, e):
    """Numpy float64 x as multiples of the 8-bit float's steps under the scale 2^e."""
    a = np.ldexp(np.abs(x), -e)
    step = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(a, 2.0 ** -30))[1] - 1, -6) - 3)
    return np.copysign(np.ldexp(np.rint(a / step) * step, e), x)


def _held64(units):
    """The keys and values of units (numpy uint8 [n, Hkv, 4112]) and their exponents: [n, Hkv, 16, 128] each,
    [n, Hkv, 2]."""
    byte = np.arange(256)
    e, m = byte // 8 % 16, byte % 8
    value = np.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9) * np.where(byte > 127, -1.0, 1.0)
    value[127] = value[255] = 0
    scale = np.ascontiguousarray(units[..., 4096:4104]).view(np.float32).astype(np.float64)
    rows = units[..., :2048].reshape(*units.shape[:-1], 16, 8, 16)
    k = np.stack([rows[..., i, [c ^ (i & 7) for c in range(8)], :] for i in range(16)], -3).reshape(*units.shape[:-1], 16, D)
    v = np.swapaxes(units[..., 2048:4096].reshape(*units.shape[:-1], D, 16), -1, -2)
    return value[k] * scale[..., 0, None, None], value[v] * scale[..., 1, None, None], np.frexp(np.maximum(scale, 2.0 ** E_LO))[1] - 1


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None
    s = prepare(case, seed)
    lens, n = _lens(case)
    Hq, Hkv, page = case["Hq"], case["Hkv"], case["page"]
    raw = s["pages"].view(-1, Hkv, page // 16, UNIT8)
    out, at = [], 0
    if case["op"] == "append":
        T, pairs = s["T"], case["pairs"]
        x = s["qkv"].double().cpu().numpy().reshape(T, Hq + 2 * Hkv, D)
        pos = s["positions"].cpu().numpy().astype(np.float64)
        turn = np.exp(1j * pos[np.array(s["axis"])].T * np.array(s["inv"]))[:, None]
        lo, hi = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if case["interleaved"] else (slice(0, pairs), slice(pairs, 2 * pairs))
        z = (x[:, :Hq + Hkv, lo] + 1j * x[:, :Hq + Hkv, hi]) * turn
        y = x.copy()
        y[:, :Hq + Hkv, lo], y[:, :Hq + Hkv, hi] = z.real, z.imag
        kv = np.stack([y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]], 1)                     # [T, 2, Hkv, 128]
        found = []
        for r, (size, c) in enumerate(zip(lens, n)):
            row = s["table"][r].cpu().numpy()
            for u in range((size - c) // 16, (size + 15) // 16):
                b, e = max(size - c, 16 * u), min(size, 16 * u + 16)
                new = kv[at + b - (size - c):at + e - (size - c)].transpose(2, 1, 0, 3)    # [Hkv, 2, new, 128]
                top = np.abs(new).max((-1, -2))
                frac, want = np.frexp(np.maximum(top, 2.0 ** -99))
                want = np.clip(np.where(frac * 512 > 448, want - 8, want - 9), E_LO, E_HI)
                if b > 16 * u:
                    k0, v0, e0 = _held64(raw[int(row[16 * u // page]), :, 16 * u % page // 16][None].cpu().numpy())
                    want = np.maximum(want, e0[0])
                    new = np.concatenate([np.stack([k0[0], v0[0]], 1)[:, :, :b - 16 * u], new], 2)
                found.append(_grid64(new, want[..., None, None]))
            at += c
        found = np.concatenate(found, 2).transpose(1, 2, 0, 3)                      # [2, positions, Hkv, 128]
        return {"q": y[:, :Hq].copy(), "k": found[0].copy(), "v": found[1].copy()}
    for r, (size, c) in enumerate(zip(lens, n)):
        u = raw[s["table"][r, :-(-size // page)].long()].permute(1, 0, 2, 3).reshape(Hkv, -1, UNIT8)
        e, m = (torch.arange(256, device=u.device) // 8 % 16).double(), (torch.arange(256, device=u.device) % 8).double()
        value = torch.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)
        value[128:] *= -1
        scale = u[..., 4096:4104].contiguous().view(torch.float32).double()
        rows = u[..., :2048].reshape(Hkv, -1, 16, 8, 16)
        k = torch.stack([rows[:, :, i][:, :, [j ^ (i & 7) for j in range(8)]] for i in range(16)], 2).reshape(Hkv, -1, 16, D)
        k = (value[k.int()] * scale[..., :1, None]).reshape(Hkv, -1, D)[:, :size]
        v = (value[u[..., 2048:4096].int()].reshape(Hkv, -1, D, 16) * scale[..., 1:, None]).transpose(-1, -2).reshape(Hkv, -1, D)[:, :size]
        q = s["q"][at:at + c].double().view(c, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3)
        sc = torch.einsum("hgcd,hld->hgcl", q, k) / D ** 0.5
        seen = torch.arange(size, device=u.device) <= size - c + torch.arange(c, device=u.device)[:, None]
        p = torch.softmax(torch.where(seen, sc, -torch.inf), -1)
        out.append(torch.einsum("hgcl,hld->chgd", p, v).reshape(c, Hq, D))
        at += c
    return torch.cat(out)
