"""Pins of the paged cache's fp64 reference against things other than itself: hand-worked tables, the
quantiser's defining properties, complex rotation, the byte layout spelled out, and a softmax over
a plain cache; and the refusals of the library's entry points, which need no GPU."""
import ctypes

import numpy as np
import pytest

from oracle import paged
from speculative_decoding_verify_06_gb300 import build, svd


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return svd.load()


def test_tables_by_hand():
    # pages of 16; request 0 loses a page (held 33 -> keeps 30, adds 2), request 1 grows into two,
    # request 2 stays inside its page
    table = np.array([[7, 3, 5, -1], [2, -1, -1, -1], [9, -1, -1, -1]], np.int32)
    free = np.array([0, 1, 4, -1, -1, -1, -1, -1, -1, -1], np.int32)
    o = paged.tables([33, 16, 3], [4, 1, 1], [1, 1, 1], [2, 17, 1], 16, table, free, 3, 24)
    assert o["kv_len"].tolist() == [32, 33, 4] and o["q_start"].tolist() == [0, 2, 19, 20]
    # page 5 goes back first and, on top of the stack, is taken first; then 4
    assert o["table"].tolist() == [[7, 3, -1, -1], [2, 5, 4, -1], [9, -1, -1, -1]]
    assert o["n_free"] == 2 and o["free"].tolist() == [0, 1] + [-1] * 8
    assert o["slots"].tolist() == ([3 * 16 + 14, 3 * 16 + 15] + [5 * 16 + i for i in range(16)] + [4 * 16] +
                                   [9 * 16 + 3] + [-1] * 4)
    assert o["positions"][:20].tolist() == [30, 31] + list(range(16, 33)) + [3]
    assert o["status"].tolist() == [0, 0, 0]


def test_tables_refusals_by_hand():
    table = np.full((4, 2), -1, np.int32)
    table[0, 0] = 1
    free = np.array([2, 3, -1, -1], np.int32)
    # 0: emitted > window; 1: takes one; 2: wants two more than are left; 3: wants nothing
    o = paged.tables([5, 0, 0, 0], [1, 0, 0, 0], [2, 0, 0, 0], [1, 16, 32, 0], 16, table, free, 2, 64)
    assert o["status"].tolist() == [paged.BAD_REQUEST, 0, paged.NO_PAGES, 0]
    assert o["kv_len"].tolist() == [0, 16, 0, 0] and o["q_start"].tolist() == [0, 0, 16, 16, 16]
    assert o["table"].tolist() == [[1, -1], [3, -1], [-1, -1], [-1, -1]] and o["n_free"] == 1
    o = paged.tables([5, 0, 0, 0], [0] * 4, [0] * 4, [1, 16, 2, 0], 16, table, free, 2, 10)
    assert o["status"].tolist() == [0, paged.NO_TOKENS, paged.NO_TOKENS, 0]


def test_quantiser_properties():
    g = np.random.default_rng(0)
    x = g.normal(0, 1, (50, 128)) * g.uniform(0.01, 50, (50, 1))
    c, d = paged.quantise(x)
    b, cb = x.reshape(50, 4, 32), c.reshape(50, 4, 32).astype(float)
    ext = np.take_along_axis(b, np.abs(b).argmax(-1)[..., None], -1)[..., 0]
    assert np.all(np.abs(d / (ext / -8) - 1) <= 2.0 ** -8)          # eight significant bits
    frac, _ = np.frexp(d)
    assert np.all(frac * 256 == np.rint(frac * 256))
    at = np.take_along_axis(cb, np.abs(b).argmax(-1)[..., None], -1)
    assert np.all(at == 0)                                          # the extreme is code 0, value -8 d
    y = d[..., None] * (cb - 8)
    # within half a step, or the clip of the far side by up to one step and the scale's rounding
    assert np.all(np.abs(y - b) <= np.abs(d)[..., None] * (0.5 + (cb == 15) * 0.54) + 8 * np.abs(d)[..., None] * 2.0 ** -8)
    # exact in fp16
    assert np.all(y == y.astype(np.float16))
    z, dz = paged.quantise(np.zeros((1, 32)))
    assert np.all(z == 8) and np.all(dz == 0)
    # ties of magnitude: the lower dimension's sign; halves go up; not-finite values
    t = np.zeros((1, 32))
    t[0, 3], t[0, 9], t[0, 5] = 8.0, -8.0, -0.5
    c, d = paged.quantise(t)
    assert d[0, 0] == -1.0 and c[0, 3] == 0 and c[0, 9] == 15 and c[0, 5] == 9
    t[0, 3], t[0, 9] = np.nan, np.inf
    c, d = paged.quantise(t)
    assert d[0, 0] == -8160.0 and c[0, 3] == 8 and c[0, 9] == 0


def test_rotation_is_complex_multiplication():
    g = np.random.default_rng(1)
    x = g.normal(size=(5, 2, 128))
    pos = g.integers(0, 1000, (3, 5))
    inv = 10000.0 ** (-np.arange(32) / 32)
    axis = g.integers(0, 3, 32)
    for inter in (False, True):
        y = paged.rotate(x, pos, inv, axis, inter)
        lo, hi = (slice(0, 64, 2), slice(1, 64, 2)) if inter else (slice(0, 32), slice(32, 64))
        z = (x[..., lo] + 1j * x[..., hi]) * np.exp(1j * pos[axis].T * inv)[:, None]
        assert np.allclose(y[..., lo], z.real, atol=1e-12) and np.allclose(y[..., hi], z.imag, atol=1e-12)
        assert np.array_equal(y[..., 64:], x[..., 64:])


def test_bytes_and_read_back():
    page, H = 32, 2
    pages = np.full((3, H, 2, paged.UNIT), 0xA5, np.uint8)
    k, v = np.zeros((2, H, 128)), np.zeros((2, H, 128))
    k[0, 1, 33], v[0, 1, 70], v[0, 1, 6] = 8.0, 4.0, 2.0  # d -1 in K block 1; -0.5 in V block 2; -0.25
    paged.put(pages, [2 * 32 + 16 + 6, -1], k, v, page)
    u = pages[2, 1, 1]
    assert u[256 + 6 * 16] == 0x08 and u[6 * 16] == 0x88      # block 1: dim 33 in the high nibble, code 0
    assert u[2048:2176].view(np.float16)[6 * 4 + 1] == -1.0
    # position 6 = 4 + 2 sits at byte 5; row 6 holds dims 6 (low: code 0) and 70 (high: code 0)
    assert u[1024 + 6 * 16 + 5] == 0x00 and u[1024 + 7 * 16 + 5] == 0x88
    assert u[2176:].view(np.float16)[2 * 16 + 6] == -0.5 and u[2176:].view(np.float16)[6] == -0.25
    assert np.all(pages[:2] == 0xA5) and u[1024 + 6 * 16 + 4] == 0xA5 and u[7 * 16] == 0xA5
    kk, vv = paged.get(pages, [2 * 32 + 22, -1, 96], page)
    assert np.array_equal(kk[0], k[0]) and np.array_equal(vv[0], v[0])
    assert not kk[1:].any() and not vv[1:].any()


def test_attention_against_a_plain_cache():
    g = np.random.default_rng(2)
    page, H, G, n = 16, 2, 3, 4
    pages = np.zeros((6, H, 1, paged.UNIT), np.uint8)
    table = np.array([[4, 1, 5], [0, -1, -1]], np.int32)
    slots = [4 * 16 + i for i in range(16)] + [16 + i for i in range(16)] + [5 * 16 + i for i in range(3)] + [0, 1]
    paged.put(pages, slots, g.normal(size=(37, H, 128)), g.normal(size=(37, H, 128)), page)
    k, v = paged.get(pages, slots, page)
    q = g.normal(size=(n + 3, H * G, 128))
    # request 1 has two positions but three tokens: its first sees nothing
    o, a, _ = paged.attention(q, pages, page, table, [35, 2], [0, n, n + 3], 0.1)
    for t, (size, base) in enumerate([(32, 0), (33, 0), (34, 0), (35, 0), (0, 35), (1, 35), (2, 35)]):
        for h in range(H * G):
            s = np.exp(q[t, h] @ k[base:base + size, h // G].T * 0.1)
            want = s @ v[base:base + size, h // G] / s.sum() if size else np.zeros(128)
            assert np.allclose(o[t, h], want, atol=1e-12)


# ---- refusals, before anything touches the GPU ---------------------------------------------------
TABLES = dict(held=16, window=16, emitted=16, n_new=16, R=2, page=16, table=32, width=4, free_ids=48, n_free=64, n_pages=8,
              table_out=80, free_out=96, n_free_out=112, kv_len=128, q_start=144, slots=160, positions=176, tokens=8,
              status=192, stream=None)


@pytest.mark.parametrize("change", [
    dict(held=None), dict(n_new=None), dict(window=None), dict(emitted=None), dict(table=None), dict(free_ids=None),
    dict(n_free=None), dict(table_out=None), dict(slots=None), dict(status=None), dict(R=0), dict(R=4097), dict(page=8),
    dict(page=24), dict(page=272), dict(page=0), dict(width=0), dict(width=1 << 27), dict(n_pages=0), dict(tokens=0),
    dict(table_out=32), dict(free_out=48), dict(n_free_out=64), dict(R=4096, width=1 << 20)])
def test_tables_refusals(lib, change):
    assert lib.svd_paged_tables(*{**TABLES, **change}.values()) == svd.SVD_ERR_INVALID_ARG


def rope(n=64, axes=1, **kw):
    r = svd.Rope([0.5] * n, kw.get("axis"), axes)
    if "inv" in kw:
        r._s.inv_freq[1] = kw["inv"]
    return r


APPEND = dict(qkv=16, dtype=0, ld=56 * 128, T=2, Hq=40, Hkv=8, rope=None, positions=16, positions_ld=2, slots=16, pages=16,
              page=16, n_pages=4, q=16, status=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(qkv=8), dict(dtype=2), dict(ld=56 * 128 - 4), dict(ld=56 * 128 + 2), dict(T=-1), dict(Hq=-1),
    dict(Hkv=0), dict(slots=None), dict(pages=None), dict(pages=24), dict(page=20), dict(n_pages=0), dict(q=None), dict(q=4),
    dict(rope=rope(), positions=None), dict(rope=rope(62)), dict(rope=rope(0)), dict(rope=rope(64, 0)), dict(rope=rope(64, 5)),
    dict(rope=rope(64, 2), positions_ld=1), dict(rope=rope(64, 1, axis=[1] * 64)), dict(rope=rope(64, 1, inv=float("nan"))),
    dict(rope=rope(64, 1, inv=2.0 ** 32))])
def test_append_refusals(lib, change):
    a = {**APPEND, **change}
    a["rope"] = None if a["rope"] is None else a["rope"]._p
    assert lib.svd_paged_append(*a.values()) == svd.SVD_ERR_INVALID_ARG


def test_rope_refuses_what_does_not_fit():
    for bad in (dict(inv_freq=[1.0] * 65), dict(inv_freq=[1.0] * 4, axis=[0] * 3), dict(inv_freq=[1.0], axis=[256])):
        with pytest.raises(ValueError):
            svd.Rope(**bad)


READ = dict(slots=16, T=2, Hkv=8, pages=16, page=16, n_pages=4, k=16, v=16, stream=None)


@pytest.mark.parametrize("change", [dict(slots=None), dict(T=-1), dict(Hkv=0), dict(pages=None), dict(pages=8), dict(page=17),
                                    dict(n_pages=0), dict(k=None), dict(k=8), dict(v=None), dict(v=4)])
def test_read_refusals(lib, change):
    assert lib.svd_paged_read(*{**READ, **change}.values()) == svd.SVD_ERR_INVALID_ARG


ATTEND = dict(q=16, T=2, kv_len=16, q_start=16, R=2, max_new=1, table=16, width=4, pages=16, page=16, n_pages=8, Hq=40, Hkv=8,
              scale=0.1, out=16, dtype=1, ws=16, ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=8), dict(T=-1), dict(kv_len=None), dict(q_start=None), dict(R=0), dict(R=4097), dict(max_new=0),
    dict(table=None), dict(width=0), dict(width=1 << 27), dict(pages=None), dict(pages=8), dict(page=40), dict(n_pages=0),
    dict(Hq=0), dict(Hq=41), dict(Hkv=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(out=None), dict(out=8), dict(dtype=2), dict(ws=8)])
def test_attention_refusals(lib, change):
    assert lib.svd_paged_attention(*{**ATTEND, **change}.values()) == svd.SVD_ERR_INVALID_ARG


def test_attention_workspace_and_empty_calls(lib):
    assert lib.svd_paged_attention(*{**ATTEND, "ws": None}.values()) == svd.SVD_ERR_WORKSPACE
    assert svd.svd_paged_attention_workspace_bytes(41, 8, 1, 1) == 0
    assert svd.svd_paged_attention_workspace_bytes(40, 8, 0, 1) == 0
    assert lib.svd_paged_attention(*{**ATTEND, "T": 0}.values()) == svd.SVD_OK
    assert lib.svd_paged_append(*{**APPEND, "T": 0}.values()) == svd.SVD_OK
    assert lib.svd_paged_read(*{**READ, "T": 0}.values()) == svd.SVD_OK


def test_cache_bytes(lib):
    # 4.5 bits a value: 144 bytes per position and kv head for 2 x 128 values
    assert svd.svd_paged_cache_bytes(8, 64, 10) == 10 * 64 * 8 * 144
    for bad in ((0, 64, 1), (8, 8, 1), (8, 24, 1), (8, 272, 1), (8, 64, 0)):
        assert svd.svd_paged_cache_bytes(*bad) == 0
    assert ctypes.sizeof(svd._Rope) == 64 * 8 + 64 + 12 + 4  # the C struct, padded to its 8-byte alignment
