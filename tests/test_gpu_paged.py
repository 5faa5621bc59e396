"""The paged 4-bit cache on the GPU against the fp64 reference: tables and appends bit for bit (the
whole pool's bytes, so that nothing else was touched), attention within bounds counted from its
roundings, at the lengths, pages, masks and contents where it can go wrong."""
import numpy as np
import pytest
import torch

from oracle import paged
from speculative_decoding_verify_06_gb300 import svd
from tests.gpu_helpers import DEV, lib, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


# ---- tables ------------------------------------------------------------------------------------
def gpu_tables(held, window, emitted, n_new, page, table, free, n_free, tokens, stream=None):
    R, width = table.shape
    n_pages = len(free)
    i32 = lambda a: None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
    mk = lambda n, t=torch.int32: torch.full((n,), -77, dtype=t, device=DEV)  # noqa: E731
    o = dict(table=mk(R * width), free=mk(n_pages), n_free=mk(1), kv_len=mk(R), q_start=mk(R + 1),
             slots=mk(tokens, torch.int64), positions=mk(tokens), status=mk(R))
    ins = [i32(held), i32(window), i32(emitted), i32(n_new), i32(table), i32(free), i32([n_free])]
    svd.svd_paged_tables(*ins[:4], R, page, ins[4], width, ins[5], ins[6], n_pages, o["table"], o["free"], o["n_free"],
                         o["kv_len"], o["q_start"], o["slots"], o["positions"], tokens, o["status"], stream=stream)
    torch.cuda.synchronize()
    o = {k: v.cpu().numpy() for k, v in o.items()}
    o["table"], o["n_free"] = o["table"].reshape(R, width), int(o["n_free"][0])
    return o


def same_tables(got, want):
    for k in want:
        assert np.array_equal(got[k], want[k]), k


def random_state(g, R, page, width, spare):
    held = g.integers(0, width * page + 1, R)
    have = -(-held // page)
    ids = g.permutation(int(have.sum()) + spare).astype(np.int32)
    table = np.full((R, width), -1, np.int32)
    table[np.arange(width) < have[:, None]] = ids[:have.sum()]
    free = np.full(len(ids), -1, np.int32)
    free[:spare] = ids[have.sum():]
    return held, table, free


@pytest.mark.parametrize("R,page,width,spare,most,tokens", [
    (1, 16, 1, 1, 3, 1), (1, 64, 5, 0, 70, 64), (3, 16, 40, 7, 5, 64), (8, 32, 17, 3, 40, 200), (33, 48, 9, 20, 300, 5000),
    (511, 16, 6, 100, 4, 2000), (513, 256, 3, 40, 9, 600), (1025, 16, 1030, 60, 8, 6000), (4096, 16, 3, 900, 8, 9000)])
def test_tables(R, page, width, spare, most, tokens):
    g = np.random.default_rng(R * 7 + page)
    held, table, free = random_state(g, R, page, width, spare)
    window = np.minimum(held, g.integers(0, 9, R))
    emitted = g.integers(0, window + 1)
    n_new = g.integers(0, most + 1, R)
    # a few contradictions
    for r in g.integers(0, R, R // 8):
        [lambda: window.__setitem__(r, held[r] + 1), lambda: emitted.__setitem__(r, window[r] + 1),
         lambda: n_new.__setitem__(r, -1), lambda: emitted.__setitem__(r, -1)][g.integers(0, 4)]()
    args = (held, window, emitted, n_new, page, table, free, spare, tokens)
    want = paged.tables(*args)
    same_tables(gpu_tables(*args), want)
    if R > 500:
        assert {0, paged.BAD_REQUEST} <= set(want["status"].tolist())


def test_tables_without_a_window_and_with_a_count_past_the_pool():
    g = np.random.default_rng(5)
    held, table, free = random_state(g, 20, 32, 12, 30)
    free[:] = g.permutation(len(free))  # every entry valid, so that a clamped count is well defined
    args = (held, np.zeros(20, int), np.zeros(20, int), np.full(20, 3), 32, table, free)
    want = paged.tables(*args, 10 ** 6, 100)
    got = gpu_tables(held, None, None, np.full(20, 3), 32, table, free, 10 ** 6, 100)
    same_tables(got, want)
    got = gpu_tables(held, None, None, np.full(20, 3), 32, table, free, -5, 100)
    same_tables(got, paged.tables(*args, -5, 100))


def test_tables_keep_every_page_in_one_place():
    g = np.random.default_rng(9)
    R, page, width, pool = 40, 16, 30, 500
    table, free = np.full((R, width), -1, np.int32), g.permutation(pool).astype(np.int32)
    held, n_free, window = np.zeros(R, int), pool, np.zeros(R, int)
    for step in range(25):
        emitted = g.integers(0, window + 1)
        done = g.random(R) < 0.05  # a request that ends gives everything back
        window, emitted = np.where(done, held, window), np.where(done, 0, emitted)
        n_new = np.where(done, 0, g.integers(0, 40, R))
        args = (held, window, emitted, n_new, page, table, free, n_free, R * 40)
        o = gpu_tables(*args)
        same_tables(o, paged.tables(*args))
        table, free, n_free = o["table"], o["free"], o["n_free"]
        held = np.where(o["status"] == 0, o["kv_len"], held)
        window = np.where(o["status"] == 0, n_new, 0)
        have = -(-held // page)
        ids = np.concatenate([table[r, :have[r]] for r in range(R)] + [free[:n_free]])
        assert np.array_equal(np.sort(ids), np.arange(pool))
        live = o["slots"][o["slots"] >= 0]
        assert len(np.unique(live)) == len(live) == o["q_start"][-1]


# ---- append and read ---------------------------------------------------------------------------
def as_type(x, dtype):
    t = torch.from_numpy(np.asarray(x, np.float32))
    return t if dtype == svd.SVD_F32 else t.to(torch.bfloat16)


def gpu_append(x, dtype, ld, T, Hq, Hkv, slots, pool, page, **kw):
    """x [T, heads, 128] float32 -> q fp32, pool bytes, status."""
    n_pages = pool.shape[0]
    buf = torch.full((max(T, 1), ld), float("nan"), dtype=torch.float32 if dtype == svd.SVD_F32 else torch.bfloat16, device=DEV)
    buf[:T, :x[0].size if T else 0] = as_type(x.reshape(T, -1), dtype).to(DEV)
    pages = to_dev(pool.reshape(-1))
    q = torch.full((T, Hq, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(T, dtype=torch.int32, device=DEV)
    if kw.get("positions") is not None:
        kw["positions"] = to_dev(np.ascontiguousarray(kw["positions"], dtype=np.int32))
        kw["positions_ld"] = kw["positions"].shape[1]
    sl = torch.tensor(np.asarray(slots), dtype=torch.int64, device=DEV)
    svd.svd_paged_append(buf, ld, T, Hq, Hkv, sl, pages, page, n_pages, q if Hq else None, dtype=dtype, status=status, **kw)
    torch.cuda.synchronize()
    return q.float().cpu().numpy(), pages.cpu().numpy().reshape(pool.shape), status.cpu().numpy()


def check_q(q, want):
    # bf16 rounding 2^-8, and the fp32 angle and rotation before it: 2^-20 of |x_a| + |x_b|
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * np.abs(want).max(initial=0.0) * 4 + 1e-30
    assert np.all(np.abs(q - want) <= bound)


@pytest.mark.parametrize("dtype", [svd.SVD_F32, svd.SVD_BF16])
@pytest.mark.parametrize("T,Hq,Hkv,page,pairs,axes,inter,pad", [
    (1, 40, 8, 16, 64, 1, False, 0), (4, 40, 8, 64, 64, 3, False, 128), (37, 5, 1, 48, 32, 3, True, 4), (65, 2, 2, 256, 4, 2, True, 0),
    (29, 3, 3, 32, 60, 4, False, 12), (16, 0, 4, 16, 64, 1, True, 0), (7, 1, 1, 128, 16, 1, False, 8)])
def test_append(dtype, T, Hq, Hkv, page, pairs, axes, inter, pad):
    g = np.random.default_rng(T * 100 + pairs)
    heads = Hq + 2 * Hkv
    x = g.normal(0, 1, (T, heads, 128)).astype(np.float32)
    x[:, Hq:, 5::32] *= 30
    x = as_type(x, dtype).float().numpy()
    n_pages = -(-T // page) + 2
    pool = g.integers(0, 256, (n_pages, Hkv, page // 16, paged.UNIT)).astype(np.uint8)
    slots = g.permutation(n_pages * page)[:T]
    if T > 6:
        slots[[1, 4]] = -1, -5
    pos = g.integers(0, 300000, (axes, T))
    pos[:, 0] = 0  # an angle of zero: keys as they came, many next to or on a border
    inv = 1e6 ** (-np.arange(pairs) / pairs)
    axis = g.integers(0, axes, pairs)
    q, got, st = gpu_append(x, dtype, heads * 128 + pad, T, Hq, Hkv, slots, pool, page, rope=svd.Rope(inv, axis, axes, inter), positions=pos)
    y = paged.rotate(x.astype(np.float64), pos, inv, axis, inter)
    want = paged.put(pool.copy(), slots, y[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], page)
    assert np.array_equal(got, want)
    assert not st.any()
    check_q(q, y[:, :Hq])
    # without rotation
    q, got, st = gpu_append(x, dtype, heads * 128 + pad, T, Hq, Hkv, slots, pool, page)
    assert np.array_equal(got, paged.put(pool.copy(), slots, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], page))
    assert np.array_equal(q, as_type(x[:, :Hq], svd.SVD_BF16).float().numpy()) and not st.any()


def test_append_next_to_the_borders_of_codes():
    """Values on and one ulp off every border of a block, both signs of the scale, all magnitudes."""
    rows = []
    for e in (-20, -12, -3, 0, 7, 12):
        for d in (1.0, -1.0, 1.0078125, -1.984375):
            for u in (-1, 0, 1):
                b = ((np.arange(32) % 16) - 7.5) * d * 2.0 ** e
                b = np.nextafter(b.astype(np.float32), np.float32(np.inf) * u) if u else b.astype(np.float32)
                b[0] = -8 * d * 2.0 ** e
                rows.append(b)
    x = np.array(rows, np.float32).reshape(-1, 128)
    T = x.shape[0]
    full = np.stack([x, x], 1)
    pool = np.zeros((T // 16 + 1, 1, 1, paged.UNIT), np.uint8)
    _, got, st = gpu_append(full, svd.SVD_F32, 256, T, 0, 1, np.arange(T), pool, 16)
    assert np.array_equal(got, paged.put(pool.copy(), np.arange(T), full[:, :1].astype(float), full[:, 1:].astype(float), 16))
    assert not st.any()


def test_append_rotated_keys_at_the_borders_of_scales():
    """Many rotated blocks: scales whose rounding or sign is nearly a tie come out as in fp64."""
    g = np.random.default_rng(77)
    T, H = 600, 2
    x = g.normal(0, 1, (T, 2 * H, 128)).astype(np.float32)
    a = np.abs(x[:, :H]).max(-1)
    x[:, :H, 17] = a * 1.5  # two extremes of opposite signs, rotated by the same angle
    x[:, :H, 18] = -a * 1.5
    pos = g.integers(0, 4, (1, T))
    inv = np.zeros(64)
    inv[::3] = 0.25
    pool = np.zeros((T // 64 + 1, H, 4, paged.UNIT), np.uint8)
    _, got, _ = gpu_append(x, svd.SVD_F32, 2 * H * 128, T, 0, H, np.arange(T), pool, 64, rope=svd.Rope(inv), positions=pos)
    y = paged.rotate(x.astype(np.float64), pos, inv, [0] * 64, False)
    assert np.array_equal(got, paged.put(pool.copy(), np.arange(T), y[:, :H], x[:, H:], 64))


def test_append_reports_what_is_not_finite_and_bad_slots():
    x = np.ones((6, 3, 128), np.float32)
    x[1, 1, 4], x[2, 2, 9], x[3, 1, 100], x[4, 0, 0] = np.nan, np.inf, -np.inf, np.nan
    pool = np.zeros((1, 1, 1, paged.UNIT), np.uint8)
    _, got, st = gpu_append(x, svd.SVD_F32, 384, 6, 1, 1, [0, 1, 2, 3, 4, 16], pool, 16)
    assert st.tolist() == [0, paged.NONFINITE, paged.NONFINITE, paged.NONFINITE, 0, paged.BAD_SLOT]
    assert np.array_equal(got, paged.put(pool.copy(), [0, 1, 2, 3, 4], x[:5, 1:2].astype(float), x[:5, 2:].astype(float), 16))
    assert np.all(np.isfinite(got.view(np.float16)[..., 1024:]))


def test_far_positions_keep_their_angle():
    """At position 2^20 - 1 an angle reduced in fp32 would be off by 0.06 rad."""
    x = np.zeros((3, 3, 128), np.float32)
    x[:, 0, :64] = 1.0
    pos = np.array([[2 ** 20 - 1, 123457, -7]])
    inv = np.linspace(1.0, 1e-4, 64)
    pool = np.zeros((1, 1, 1, paged.UNIT), np.uint8)
    q, _, _ = gpu_append(x, svd.SVD_F32, 384, 3, 1, 1, [0, 1, 2], pool, 16, rope=svd.Rope(inv), positions=pos)
    check_q(q, paged.rotate(x.astype(np.float64), pos, inv, [0] * 64, False)[:, :1])


@pytest.mark.parametrize("page,H", [(16, 1), (48, 3), (128, 8)])
def test_read(page, H):
    g = np.random.default_rng(page)
    pool = g.integers(0, 256, (4, H, page // 16, paged.UNIT)).astype(np.uint8)
    pool.view(np.float16)[..., 1024:] = g.normal(0, 1, (4, H, page // 16, 128))
    slots = np.concatenate([g.permutation(4 * page)[:50], [-1, 4 * page, 2 ** 40]])
    k = torch.full((len(slots), H, 128), float("nan"), device=DEV)
    v = torch.full_like(k, float("nan"))
    svd.svd_paged_read(torch.tensor(slots, device=DEV), len(slots), H, to_dev(pool.reshape(-1)), page, 4, k, v)
    kk, vv = paged.get(pool, slots, page)
    assert np.array_equal(k.double().cpu().numpy(), kk) and np.array_equal(v.double().cpu().numpy(), vv)


# ---- attention ---------------------------------------------------------------------------------
class Case:
    def __init__(self, lens, new, Hq, Hkv, page, seed=0, spread=1.0, width=None):
        g = np.random.default_rng(seed)
        self.g, self.lens, self.new, self.Hq, self.Hkv, self.page = g, lens, new, Hq, Hkv, page
        R = len(lens)
        have = [-(-max(x, 0) // page) for x in lens]
        self.n_pages = sum(have) + 2
        # 0xFF everywhere else: scales of positions past the lengths are NaN
        self.pool = np.full((self.n_pages, Hkv, page // 16, paged.UNIT), 0xFF, np.uint8)
        ids = g.permutation(self.n_pages)
        self.table = np.full((R, width or max(1, max(have))), -1, np.int32)
        at = 0
        units = self.pool.reshape(-1, paged.UNIT)
        for r, n in enumerate(have):
            self.table[r, :n] = ids[at:at + n]
            at += n
        half = self.pool.view(np.uint16)
        for r, x in enumerate(lens):  # random codes and eight-bit scales, written part by part
            for c in range(have[r]):
                pg, m = self.table[r, c], min(page, x - c * page)
                for u in range(-(-m // 16)):
                    p = min(16, m - 16 * u)
                    vb = [4 * (i // 4) + (0, 2, 1, 3)[i % 4] for i in range(p)]
                    self.pool[pg, :, u, :1024].reshape(Hkv, 4, 16, 16)[:, :, :p] = g.integers(0, 256, (Hkv, 4, p, 16))
                    codes = self.pool[pg, :, u, 1024:2048].reshape(Hkv, 64, 16)
                    codes[:, :, vb] = g.integers(0, 256, (Hkv, 64, p))
                    sc = lambda *s: (g.integers(128, 256, s) / 1024 * g.choice([-1, 1], s)).astype(np.float16)  # noqa: E731
                    half[pg, :, u, 1024:1088].reshape(Hkv, 16, 4)[:, :p] = (sc(Hkv, p, 4) * np.float16(spread)).view(np.uint16)
                    half[pg, :, u, 1088:].reshape(Hkv, 4, 16)[:, :, :p] = sc(Hkv, 4, p).view(np.uint16)
        assert units.base is not None
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T = int(self.q_start[-1])
        q = torch.from_numpy(g.normal(0, 1, (max(self.T, 1), Hq, 128))).to(torch.bfloat16)
        self.q = q
        self.scale = 128 ** -0.5
        self.largest = 8 * 255 / 1024  # of the values

    def run(self, out_dtype, max_new=None, T=None, ws=None, stream=None, table=None, out=None):
        T = self.T if T is None else T
        most = max(1, max(self.new)) if max_new is None else max_new
        dt = torch.bfloat16 if out_dtype == svd.SVD_BF16 else torch.float32
        q = torch.zeros((T, self.Hq, 128), dtype=torch.bfloat16)
        q[:self.T] = self.q[:self.T]
        if out is None:
            out = torch.full((T, self.Hq, 128), -7.0, dtype=dt, device=DEV)
        if ws is None:
            ws = torch.zeros(svd.svd_paged_attention_workspace_bytes(self.Hq, self.Hkv, len(self.lens), most),
                             dtype=torch.uint8, device=DEV)
        tab = to_dev(self.table if table is None else table)
        self.keep = (q.to(DEV), to_dev(np.array(self.lens, np.int32)), to_dev(self.q_start), tab, to_dev(self.pool.reshape(-1)), ws)
        torch.cuda.synchronize()
        svd.svd_paged_attention(self.keep[0], T, self.keep[1], self.keep[2], len(self.lens), most, tab, tab.shape[1],
                                self.keep[4], self.page, self.n_pages, self.Hq, self.Hkv, self.scale, out, out_dtype, ws,
                                stream=stream)
        torch.cuda.synchronize()
        assert ws[:4].view(torch.int32).item() == 0
        return out.double().cpu().numpy()

    def reference(self, **kw):
        return paged.attention(self.q.double().numpy(), self.pool, self.page, kw.pop("table", self.table), self.lens,
                               self.q_start, self.scale, **kw)

    def check(self, out_dtype, got, ref):
        o, a, e = ref
        n = max(max(self.lens), 1)
        # scores: 128 products added with 2^-23 each; p: that, its exponent's 2^-20, and for bf16 outputs
        # its rounding to fp16 (2^-11), for fp32 outputs what its two parts leave (2^-21); the sums over
        # positions: 2^-23 an addition (fp32 outputs: within a tile, then over the tiles); and fp16's
        # smallest step: p is held to 2^-25 where the largest p is 2^7 or more, so what a position adds is
        # good to 2^-32 of its value
        score = 2.0 ** -16 * e[..., None]
        if out_dtype == svd.SVD_BF16:
            bound = 2.0 ** -8 * np.abs(o) + a * (2.0 ** -11 + 2 * score + n * 2.0 ** -23 + 2.0 ** -19)
        else:
            bound = a * (2.0 ** -21 + 2 * score + (256 + n / 128) * 2.0 ** -23 + 2.0 ** -19)
        bound = bound + n * 2.0 ** -32 * self.largest
        there = ~np.isnan(o)
        assert np.all(np.isfinite(got[there]))
        err = np.abs(got - o)
        assert np.all(err[there] <= bound[there] + 1e-30), float(np.max((err / (bound + 1e-30))[there]))
        assert np.all(got[~there] == -7.0)  # rows that no request has are left alone


BOTH = pytest.mark.parametrize("out_dtype", [svd.SVD_BF16, svd.SVD_F32])


@BOTH
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (10, 2), (13, 1), (24, 2), (32, 1), (40, 1)])
@pytest.mark.parametrize("new", [1, 4])
def test_attention_heads(out_dtype, Hq, Hkv, new):
    c = Case([70, 200], [new, new], Hq, Hkv, 32, seed=Hq)
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
@pytest.mark.parametrize("page", [16, 48, 128, 256])
def test_attention_lengths(out_dtype, page):
    """Lengths around units, pages and tiles; a request without tokens, one without positions."""
    lens = [1, 2, 15, 16, 17, 0, 31, 33, 127, 128, 129, 255, 256, 257, 90, 385]
    new = [1, 2, 3, 1, 2, 0, 3, 1, 2, 1, 3, 1, 2, 3, 0, 1]
    c = Case(lens, new, 6, 2, page, seed=page)
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
@pytest.mark.parametrize("new", [5, 13, 21, 33, 100, 150])
def test_attention_windows_of_several_row_tiles(out_dtype, new):
    c = Case([new, new + 100, 290, 150], [new, new, min(new, 7), new], 6, 2, 64, seed=new)
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
def test_attention_over_many_ctas(out_dtype):
    """A long cache, split between CTAs and joined; beside short ones."""
    c = Case([9000, 40, 3000], [2, 1, 1], 5, 1, 64, seed=3)
    c.check(out_dtype, c.run(out_dtype), c.reference())


def test_attention_many_requests():
    g = np.random.default_rng(4)
    lens = g.integers(1, 60, 700).tolist()
    c = Case(lens, g.integers(0, 2, 700).tolist(), 2, 1, 16, seed=5)
    c.check(svd.SVD_BF16, c.run(svd.SVD_BF16), c.reference())
    c = Case([20] * 4096, [1] * 4096, 1, 1, 16, seed=6)
    c.check(svd.SVD_BF16, c.run(svd.SVD_BF16), c.reference())


@BOTH
def test_rows_that_see_nothing_are_zero(out_dtype):
    """Fewer positions than tokens: the first tokens' positions are negative."""
    c = Case([2, 0, 130], [5, 3, 131], 4, 2, 32, seed=7)
    got = c.run(out_dtype)
    c.check(out_dtype, got, c.reference())
    assert not got[:3].any() and not got[5:8].any() and not got[8].any() and got[9].any()


@BOTH
def test_pages_outside_the_pool_take_no_part(out_dtype):
    c = Case([300, 200, 100], [2, 1, 4], 5, 1, 32, seed=8)
    t = c.table.copy()
    t[0, 0], t[0, 4], t[0, 9], t[1, :], t[2, 1] = -1, c.n_pages, 2 ** 31 - 1, -9, -2 ** 31
    got = c.run(out_dtype, table=t)
    c.check(out_dtype, got, c.reference(table=t))
    assert not got[2].any()  # every page of request 1


@BOTH
def test_max_new_and_padding(out_dtype):
    """Tokens past max_new, and past the last request, are not written."""
    c = Case([50, 60], [4, 6], 4, 1, 16, seed=9)
    got = c.run(out_dtype, max_new=4, T=c.T + 3)
    o, a, e = c.reference(max_new=4)
    pad = np.full((3, 4, 128), np.nan)
    c.check(out_dtype, got, (np.concatenate([o, pad]), np.concatenate([a, pad]), np.concatenate([e, pad[..., 0]])))


@BOTH
@pytest.mark.parametrize("spread", [0.0, 2.0 ** -6, 32.0])
def test_scores_of_any_spread(out_dtype, spread):
    """Equal scores; scores near 0; scores of some hundred, so that one position takes all."""
    c = Case([700, 1300], [3, 1], 5, 1, 64, seed=10, spread=spread)
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
def test_rising_scores_move_the_reference(out_dtype):
    """Key scales that grow along the cache: the largest score rises from tile to tile."""
    c = Case([1500], [4], 5, 1, 16, seed=11)
    half = c.pool.view(np.uint16)
    for p in range(1500):
        pg, u, i = c.table[0, p // 16], 0, p % 16
        d = np.float16(2.0 ** (-8 + p // 128))
        half[pg, 0, u, 1024 + 4 * i:1028 + 4 * i] = d.view(np.uint16)
    c.check(out_dtype, c.run(out_dtype), c.reference())


def test_a_query_that_is_not_a_number_stays_in_its_row():
    c = Case([300], [4], 5, 1, 64, seed=12)
    ref = c.reference()
    c.q[2, 3, 7] = float("nan")
    c.q[1, 0, :] = float("inf")
    for out_dtype in (svd.SVD_BF16, svd.SVD_F32):
        got = c.run(out_dtype)
        assert np.isnan(got[2, 3]).all() and np.isnan(got[1, 0]).all()
        got[2, 3], got[1, 0] = ref[0][2, 3], ref[0][1, 0]
        c.check(out_dtype, got, ref)


def test_offsets_past_32_bits():
    """A pool of 5 GB with the request's pages at its end."""
    c = Case([100], [2], 8, 8, 256, seed=13)
    small = c.run(svd.SVD_BF16)
    per = 8 * 16 * paged.UNIT
    n_pages = 5 * 2 ** 30 // per
    pool = torch.empty(n_pages * per, dtype=torch.uint8, device=DEV)
    pool[(n_pages - 1) * per:] = to_dev(c.pool[c.table[0, 0]].reshape(-1))
    tab = torch.tensor([[n_pages - 1]], dtype=torch.int32, device=DEV)
    out = torch.empty((2, 8, 128), dtype=torch.bfloat16, device=DEV)
    svd.svd_paged_attention(c.keep[0], 2, c.keep[1], c.keep[2], 1, 2, tab, 1, pool, 256, n_pages, 8, 8, c.scale, out,
                            svd.SVD_BF16, c.keep[5])
    assert np.array_equal(out.double().cpu().numpy(), small)
    # append and read there too
    x = torch.randn((1, 24 * 128), device=DEV)
    slot = torch.tensor([n_pages * 256 - 1], device=DEV)
    k, v = torch.empty((1, 8, 128), device=DEV), torch.empty((1, 8, 128), device=DEV)
    svd.svd_paged_append(x, 24 * 128, 1, 8, 8, slot, pool, 256, n_pages, torch.empty((1, 8, 128), dtype=torch.bfloat16, device=DEV))
    svd.svd_paged_read(slot, 1, 8, pool, 256, n_pages, k, v)
    codes, d = paged.quantise(x.double().cpu().numpy().reshape(24, 128)[8:])
    want = (codes.reshape(16, 4, 32).astype(float) - 8) * d[..., None]
    assert np.array_equal(torch.cat([k[0], v[0]]).double().cpu().numpy(), want.reshape(16, 128))


def test_the_same_bits_every_time_and_in_a_graph_on_another_stream():
    c = Case([5000, 17, 800], [3, 1, 2], 10, 2, 32, seed=14)
    first = c.run(svd.SVD_BF16)
    assert np.array_equal(c.run(svd.SVD_BF16), first)
    q, lens, starts, tab, pool, ws = c.keep
    s = torch.cuda.Stream()
    out = torch.zeros((c.T, 10, 128), dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    svd.svd_graph_begin(s)
    for _ in range(3):
        svd.svd_paged_attention(q, c.T, lens, starts, 3, 3, tab, tab.shape[1], pool, 32, c.n_pages, 10, 2, c.scale, out,
                                svd.SVD_BF16, ws, stream=s)
    g = svd.svd_graph_end(s)
    g.launch(s)
    g.launch(s)
    s.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), first)


def test_a_wait_that_runs_out_is_reported_and_does_not_hang():
    """The second word of the workspace lets every wait that is not satisfied at once give up."""
    c = Case([5000, 600], [4, 2], 10, 2, 32, seed=15)
    want = c.run(svd.SVD_BF16)
    ws = c.keep[5]
    for out_dtype in (svd.SVD_BF16, svd.SVD_F32):
        out = torch.zeros((c.T, 10, 128), dtype=torch.bfloat16 if out_dtype == svd.SVD_BF16 else torch.float32, device=DEV)
        ws[:8].view(torch.int32)[1] = 1
        svd.svd_paged_attention(*[c.keep[0], c.T, c.keep[1], c.keep[2], 2, 4, c.keep[3], c.keep[3].shape[1], c.keep[4], 32,
                                  c.n_pages, 10, 2, c.scale, out, out_dtype, ws])
        torch.cuda.synchronize()
        assert ws[:8].view(torch.int32)[0].item() == 1
        ws[:8] = 0
    assert np.array_equal(c.run(svd.SVD_BF16, ws=ws), want)


def test_nothing_is_written_beside_the_outputs():
    c = Case([400, 30], [3, 2], 10, 2, 32, seed=16)
    big = torch.full((c.T * 10 * 128 + 512,), -7.0, dtype=torch.bfloat16, device=DEV)
    most = 3
    n = svd.svd_paged_attention_workspace_bytes(10, 2, 2, most)
    ws = torch.full((n + 512,), 0, dtype=torch.uint8, device=DEV)
    ws[n:] = 0xEE
    c.run(svd.SVD_BF16, ws=ws[:n], out=big[256:256 + c.T * 1280].view(c.T, 10, 128))
    assert (big[:256] == -7).all() and (big[-256:] == -7).all() and (ws[n:] == 0xEE).all()
