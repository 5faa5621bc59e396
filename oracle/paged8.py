"""fp64 reference of the paged 8-bit cache (append, read-back, attention) and of moving pages (fork, compact).

Written from the definitions in include/svd.h, one request, unit and page at a time; shares no code with the
kernels.
"""
from __future__ import annotations

import numpy as np

from . import paged

D, UNIT = 128, 4112
E_LO, E_HI = -64, 7
LARGEST = 448.0 * 2.0 ** E_HI
BAD_REQUEST, NO_PAGES, NONFINITE, BAD_SLOT = 32, 64, 256, 512

# The value of every code; the two codes that are no numbers are NaN.
VALUE = np.array([(-1.0 if c & 128 else 1.0) * ((8 + c % 8) * 2.0 ** (c // 8 % 16 - 10) if c // 8 % 16 else c % 8 * 2.0 ** -9)
                  if c % 128 != 127 else np.nan for c in range(256)])


def encode(x):
    """float64 -> codes, to nearest, ties to even; magnitudes end at 448."""
    x = np.asarray(x, np.float64)
    positive = VALUE[:127]                                  # ascending
    a = np.minimum(np.abs(x), 448.0)
    above = np.clip(np.searchsorted(positive, a), 1, 126)   # positive[above - 1] <= a <= positive[above]
    lo, hi = a - positive[above - 1], positive[above] - a   # exact
    code = np.where(lo < hi, above - 1, np.where(lo > hi, above, above - (above & 1)))
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def exponent(top):
    """The smallest e in E_LO..E_HI with 448 * 2^e >= top."""
    for e in range(E_LO, E_HI):
        if 448.0 * 2.0 ** e >= top:
            return e
    return E_HI


def clean(x):
    """What is no number counts as 0, and magnitudes end."""
    return np.clip(np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf), -LARGEST, LARGEST)


def k_bytes(i):
    """Byte of every dimension of position i among a unit's K codes."""
    d = np.arange(D)
    return i * D + (((d // 16) ^ (i % 8)) * 16) + d % 16


def v_bytes(i):
    return 2048 + np.arange(D) * 16 + i


def stored_exponent(scale):
    frac, e = np.frexp(np.float64(scale))
    return int(np.clip(e - 1, E_LO, E_HI)) if scale > 0 else E_LO


def append(pages, k, v, kv_len, q_start, table, page):
    """Stores fp64 keys and values [T, Hkv, 128] in pages uint8 [n, Hkv, page/16, 4112]; returns the tokens that have no page."""
    T = len(k)
    k, v = clean(k), clean(v)
    lost = []
    for r in range(len(kv_len)):
        n = int(q_start[r + 1]) - int(q_start[r])
        begin = int(kv_len[r]) - n
        units = {}
        for i in range(n):
            t, p = int(q_start[r]) + i, begin + i
            if t >= T:
                continue
            pg = int(table[r, p // page]) if 0 <= p < table.shape[1] * page else -1
            if not 0 <= pg < len(pages):
                lost.append(t)
                continue
            units.setdefault((pg, p % page // 16), []).append((p % 16, t))
        for (pg, u), rows in units.items():
            first = rows[0][0]
            for h in range(pages.shape[1]):
                unit = pages[pg, h, u]
                scales = unit[4096:4104].view(np.float32)
                for part, (x, place) in enumerate(((k, k_bytes), (v, v_bytes))):
                    e = exponent(max(np.abs(x[t, h]).max() for _, t in rows))
                    if first > 0:
                        had = stored_exponent(scales[part])
                        e = max(e, had)
                        if e > had:
                            for i in range(first):
                                unit[place(i)] = encode(VALUE[unit[place(i)]] * 2.0 ** (had - e))
                    for i, t in rows:
                        unit[place(i)] = encode(x[t, h] * 2.0 ** -e)
                    scales[part] = 2.0 ** e
    return lost


def get(pages, slots, page):
    """The fp64 keys and values at slots, [T, Hkv, 128] each; 0 outside the pool."""
    T, H = len(slots), pages.shape[1]
    k, v = np.zeros((T, H, D)), np.zeros((T, H, D))
    s = np.asarray(slots, np.int64)
    ok = np.flatnonzero((s >= 0) & (s < pages.shape[0] * page))
    s = s[ok]
    unit = pages[s // page, :, s % page // 16]                                  # [t, H, 4112]
    scale = np.ascontiguousarray(unit[:, :, 4096:4104]).view(np.float32).astype(np.float64)
    kb, vb = (np.array([f(i) for i in s % 16], np.int64).reshape(-1, D) for f in (k_bytes, v_bytes))
    tt, hh = np.arange(len(ok))[:, None, None], np.arange(H)[:, None]
    k[ok] = VALUE[unit[tt, hh, kb[:, None]]] * scale[..., :1]
    v[ok] = VALUE[unit[tt, hh, vb[:, None]]] * scale[..., 1:]
    return k, v


def attention(q, pages, page, table, kv_len, q_start, scale, max_new=None):
    """As paged.attention, over this format: (o, a, e), and per output row the largest magnitude among the values that it sees."""
    T, Hq, _ = q.shape
    H = pages.shape[1]
    G = Hq // H
    o, a = np.full(q.shape, np.nan), np.zeros(q.shape)
    e, big = np.zeros((T, Hq)), np.zeros((T, Hq))
    for r in range(len(kv_len)):
        t0, n = int(q_start[r]), int(q_start[r + 1] - q_start[r])
        size = min(max(int(kv_len[r]), 0), table.shape[1] * page)
        pos = np.arange(size)
        pg = table[r, pos // page].astype(np.int64)
        there = (pg >= 0) & (pg < pages.shape[0])
        k, v = get(pages, np.where(there, pg * page + pos % page, -1), page)
        for i in range(min(n, T - t0) if max_new is None else min(n, max_new, T - t0)):
            seen = there & (pos <= int(kv_len[r]) - n + i)
            for h in range(Hq):
                x, kk, vv = q[t0 + i, h], k[seen, h // G], v[seen, h // G]
                if not len(kk):
                    o[t0 + i, h] = 0
                    continue
                s = kk @ x * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                o[t0 + i, h], a[t0 + i, h] = p @ vv, p @ np.abs(vv)
                e[t0 + i, h] = (np.abs(kk) @ np.abs(x)).max() * scale
                big[t0 + i, h] = (p[:, None] * np.abs(vv)).max()
    return o, a, e, big


# ---- moving pages ----------------------------------------------------------------------------------
def fork(held, window, emitted, parent, page, table, free, n_free):
    """Returns dict(held, window, table, free, n_free, moves [(from, to)], status)."""
    R, width = table.shape
    n_pages, room = len(free), width * page
    window = np.zeros(R, int) if window is None else window
    child = [0 <= int(parent[r]) != r for r in range(R)]
    keep, status, p0, p1 = [0] * R, [0] * R, [0] * R, [0] * R
    for r in range(R):
        if not child[r]:
            continue
        s = int(parent[r])
        ok = s < R and 0 <= held[r] <= room and not child[s]
        if ok:
            w = int(window[s])
            e = (w if emitted is None else int(emitted[s])) if w > 0 else 0
            ok = 0 <= e <= abs(w) <= held[s] <= room
            keep[r] = int(held[s]) - abs(w) + e
        if not ok:
            status[r] = BAD_REQUEST
            continue
        p0[r], p1[r] = -(-int(held[r]) // page), -(-keep[r] // page)
    stack = [int(x) for x in free[:min(max(int(n_free), 0), n_pages)]]
    for r in range(R):
        stack += [int(table[r, c]) for c in range(p1[r], p0[r])]
    available, wanted = len(stack), 0
    out, moves = table.copy(), []
    held_out, window_out = np.array(held, np.int32), np.array(window, np.int32)
    for r in range(R):
        if not child[r] or status[r]:
            continue
        need = max(0, p1[r] - p0[r])
        wanted += need
        if need and wanted > available:
            status[r] = NO_PAGES
            continue
        for c in range(p0[r], p1[r]):
            out[r, c] = stack.pop()
        out[r, p1[r]:] = -1
        held_out[r], window_out[r] = keep[r], 0
        moves += [(int(table[int(parent[r]), c]), int(out[r, c])) for c in range(p1[r])]
    free_out = np.full(n_pages, -1, np.int32)
    free_out[:len(stack)] = stack
    return dict(held=held_out, window=window_out, table=out, free=free_out, n_free=len(stack), moves=moves,
                status=np.array(status, np.int32))


def compact(held, page, table, n_pages):
    """Returns dict(table, free, n_free, moves)."""
    R, width = table.shape
    have = [min(max(-(-int(h) // page), 0), width) for h in held]
    used = sorted({int(table[r, c]) for r in range(R) for c in range(have[r]) if 0 <= table[r, c] < n_pages})
    U, held_ids = len(used), set(used)
    src = [i for i in used if i >= U]
    moves = list(zip(src, [i for i in range(U) if i not in held_ids]))
    to = dict(moves)
    out = np.full_like(table, -1)
    for r in range(R):
        for c in range(have[r]):
            out[r, c] = to.get(int(table[r, c]), int(table[r, c]))
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - U] = np.arange(n_pages - 1, U - 1, -1)
    return dict(table=out, free=free, n_free=n_pages - U, moves=moves)


def rotate(x, positions, inv_freq, axis, interleaved):
    return paged.rotate(x, positions, inv_freq, axis, interleaved)
