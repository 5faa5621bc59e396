"""fp64 reference of the paged 4-bit cache: tables from request lengths, rotary append, attention.

Written from the definitions in include/svd.h, one request and one block at a time; shares no code
with the kernels.
"""
from __future__ import annotations

import numpy as np

D, UNIT = 128, 2304
BAD_REQUEST, NO_PAGES, NO_TOKENS, NONFINITE, BAD_SLOT = 32, 64, 128, 256, 512
LARGEST = 65280.0  # magnitudes end here: -8 d still fits fp16


def tables(held, window, emitted, n_new, page, table, free, n_free, max_tokens):
    """Returns dict(table, free, n_free, kv_len, q_start, slots, positions, status)."""
    R, width = table.shape
    n_pages = len(free)
    keep, p0, p1, status = [], [], [], []
    asked = 0
    for r in range(R):
        w, e, h, n = int(window[r]), int(emitted[r]), int(held[r]), int(n_new[r])
        k = h - w + e
        a, b = -(-h // page), -(-(k + n) // page)
        st = 0
        if not (0 <= e <= w <= h) or n < 0 or a > width or b > width:
            st = BAD_REQUEST
        else:
            asked += n
            if n > 0 and asked > max_tokens:
                st = NO_TOKENS
        keep.append(k)
        p0.append(a)
        p1.append(a if st else b)
        status.append(st)
    stack = [int(x) for x in free[:min(max(int(n_free), 0), n_pages)]]
    out = table.copy()
    for r in range(R):
        if status[r] == 0:
            stack += [int(table[r, c]) for c in range(p1[r], p0[r])]
    available, wanted = len(stack), 0
    for r in range(R):
        if status[r] == BAD_REQUEST:
            continue
        need = max(0, p1[r] - p0[r])
        wanted += need
        if need and wanted > available:
            status[r], p1[r] = NO_PAGES, p0[r]
        for c in range(p0[r], p1[r]):
            out[r, c] = stack.pop()
        out[r, p1[r]:] = -1
    left = len(stack)
    free_out = np.full(n_pages, -1, np.int32)
    free_out[:min(left, n_pages)] = stack[:n_pages]
    slots = np.full(max_tokens, -1, np.int64)
    positions = np.full(max_tokens, -1, np.int32)
    kv_len, q_start, t = [], [0], 0
    for r in range(R):
        n = int(n_new[r]) if status[r] == 0 else 0
        kv_len.append(0 if status[r] == BAD_REQUEST else keep[r] + n)
        for i in range(n):
            p = keep[r] + i
            slots[t], positions[t] = int(out[r, p // page]) * page + p % page, p
            t += 1
        q_start.append(t)
    return dict(table=out, free=free_out, n_free=left, kv_len=np.array(kv_len, np.int32),
                q_start=np.array(q_start, np.int32), slots=slots, positions=positions,
                status=np.array(status, np.int32))


def advance(held, window, emitted, n_new, max_new, page, table, free, n_free, max_tokens):
    """tables() with the state carried: also held and window of the next call.  A request for more than
    max_new tokens asks for nothing and gives nothing back."""
    R = len(held)
    room = table.shape[1] * page
    win, kept, odd, over = [], [], [], []
    for r in range(R):
        w, h = int(window[r]), int(held[r])
        e = (w if emitted is None else int(emitted[r])) if w > 0 else 0
        win.append(abs(w))
        kept.append(e)
        odd.append(not 0 <= e <= abs(w) <= h)
        over.append(not odd[r] and max(h, h - win[r] + e + int(n_new[r])) <= room and int(n_new[r]) > max_new)
    still = np.array(over)
    o = tables(held, np.where(still, 0, win), np.where(still, 0, kept), np.where(still, 0, n_new), page, table, free,
               n_free, max_tokens)
    o["status"][still] = NO_TOKENS
    o["held"], o["window"] = np.zeros(R, np.int32), np.zeros(R, np.int32)
    for r in range(R):
        keep = int(held[r]) - win[r] + (0 if odd[r] else kept[r])
        if o["status"][r] == 0:
            o["held"][r], o["window"][r] = keep + int(n_new[r]), int(n_new[r])
        else:
            o["held"][r], o["window"][r] = held[r], window[r] if odd[r] else kept[r] - win[r]
            o["kv_len"][r] = max(keep, 0)
    return o


def rotate(x, positions, inv_freq, axis, interleaved):
    """x [T, heads, 128] fp64; positions [axes, T]."""
    y = x.copy()
    n = len(inv_freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        t = positions[axis[i]].astype(np.float64) * inv_freq[i]
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def quantise(x):
    """Blocks of 32 of the last dimension: codes uint8 [..., 128] and scales float64 [..., 4]."""
    x = np.clip(np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=np.inf, neginf=-np.inf),
                -LARGEST, LARGEST)
    b = x.reshape(-1, 32)
    codes = np.empty(b.shape, np.uint8)
    scales = np.empty(len(b))
    for i, row in enumerate(b):
        m = row[np.abs(row).argmax()] / -8.0
        frac, e = np.frexp(m)
        d = float(np.float16(np.ldexp(np.rint(frac * 256), e - 8)))
        scales[i] = d
        codes[i] = np.clip(np.floor(row / d + 8.5), 0, 15) if d != 0 else 8
    return codes.reshape(x.shape), scales.reshape(*x.shape[:-1], x.shape[-1] // 32)


def put(pages, slots, k, v, page):
    """Writes quantised keys and values fp64 [T, Hkv, 128] into pages uint8 [n, Hkv, page/16, 2304];
    slots outside the pool are passed over."""
    kc, kd = quantise(k)
    vc, vd = quantise(v)
    half = pages.view(np.uint16)
    for t, s in enumerate(slots):
        if not 0 <= s < pages.shape[0] * page:
            continue
        pg, u, i = int(s) // page, int(s) % page // 16, int(s) % 16
        vb = 4 * (i // 4) + (0, 2, 1, 3)[i % 4]
        for h in range(pages.shape[1]):
            for blk in range(4):
                c = kc[t, h, 32 * blk:32 * blk + 32]
                pages[pg, h, u, blk * 256 + i * 16:blk * 256 + i * 16 + 16] = c[0::2] | (c[1::2] << 4)
                half[pg, h, u, 1024 + 4 * i + blk] = np.float16(kd[t, h, blk]).view(np.uint16)
                half[pg, h, u, 1088 + 16 * blk + i] = np.float16(vd[t, h, blk]).view(np.uint16)
            pages[pg, h, u, 1024 + vb:2048:16] = vc[t, h, :64] | (vc[t, h, 64:] << 4)
    return pages


@np.errstate(invalid="ignore")  # (bytes of positions that nobody asked for may be signalling NaNs)
def get(pages, slots, page):
    """The fp64 keys and values that pages hold at slots: [T, Hkv, 128] each; 0 outside the pool."""
    T, H = len(slots), pages.shape[1]
    k, v = np.zeros((T, H, D)), np.zeros((T, H, D))
    f16 = pages.view(np.float16)
    ok = [t for t, s in enumerate(slots) if 0 <= s < pages.shape[0] * page]
    s = np.asarray(slots, np.int64)[ok]
    pg, u, i = s // page, s % page // 16, s % 16
    unit = pages[pg, :, u]                                   # [t, H, 2304]
    half = f16[pg, :, u].astype(np.float64)
    tt = np.arange(len(ok))
    kb = unit[:, :, :1024].reshape(-1, H, 4, 16, 16)[tt, :, :, i]         # [t, H, 4, 16]
    kd = half[:, :, 1024:1088].reshape(-1, H, 16, 4)[tt, :, i]            # [t, H, 4]
    codes = np.stack([kb & 15, kb >> 4], -1).reshape(-1, H, 4, 32).astype(np.float64)
    k[ok] = ((codes - 8) * kd[..., None]).reshape(-1, H, D)
    vb = unit[:, :, 1024:2048].reshape(-1, H, 64, 16)[tt, :, :, (i // 4) * 4 + np.array([0, 2, 1, 3])[i % 4]]
    vd = half[:, :, 1088:].reshape(-1, H, 4, 16)[tt, :, :, i]
    codes = np.concatenate([vb & 15, vb >> 4], -1).reshape(-1, H, 4, 32).astype(np.float64)
    v[ok] = ((codes - 8) * vd[..., None]).reshape(-1, H, D)
    return k, v


def attention(q, pages, page, table, kv_len, q_start, scale, max_new=None):
    """q fp64 [T, Hq, 128].  Returns (o, a, e): the outputs, sum_j p_j |v_j|, and per output row the
    largest sum_i |q_i k_ji| scale over the positions it sees; rows of no request are NaN."""
    T, Hq, _ = q.shape
    H = pages.shape[1]
    G = Hq // H
    o, a = np.full(q.shape, np.nan), np.zeros(q.shape)
    e = np.zeros((T, Hq))
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
    return o, a, e
