"""The paged 8-bit cache on the GPU against the fp64 reference: appends and read-back bit for bit (the whole
pool's bytes, so that nothing else was touched), attention within bounds counted from its roundings, at the
lengths, pages, masks and contents where it can go wrong."""
import numpy as np
import pytest
import torch

from oracle import paged, paged8
from speculative_decoding_verify_06_gb300 import svd
from tests.gpu_helpers import DEV, lib, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def same_zeros(pool):
    """Pool bytes with one code for zero: -0 and 0 are the same value."""
    p = pool.copy()
    codes = p[..., :4096]
    codes[codes == 0x80] = 0
    return p


def layout(lens, new, page, g, spare=2):
    """A table of random pages, and the first token of every request."""
    have = [-(-max(x, 0) // page) for x in lens]
    ids = g.permutation(sum(have) + spare)
    table = np.full((len(lens), max(1, max(have))), -1, np.int32)
    at = 0
    for r, n in enumerate(have):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, np.concatenate([[0], np.cumsum(new)]).astype(np.int32), len(ids)


def random_pool(g, n_pages, H, page, e_lo=-3, e_hi=2):
    pool = g.integers(0, 255, (n_pages, H, page // 16, paged8.UNIT)).astype(np.uint8)
    codes = pool[..., :4096]
    codes[codes % 128 == 127] = 3
    pool.view(np.float32)[..., 1024:1026] = 2.0 ** g.integers(e_lo, e_hi, (n_pages, H, page // 16, 2))
    return pool


def as_type(x, dtype):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return t.to(torch.bfloat16) if dtype == svd.SVD_BF16 else t


def gpu_append(x, dtype, Hq, Hkv, lens, q_start, table, pool, page, rope=None, positions=None, ld=None, T=None, stream=None):
    heads = Hq + 2 * Hkv
    T = len(x) if T is None else T
    ld = heads * 128 if ld is None else ld
    rows = torch.zeros((T, ld), dtype=torch.float32)
    rows[:len(x), :heads * 128] = torch.from_numpy(np.ascontiguousarray(x.reshape(len(x), -1)))
    rows = rows.to(torch.bfloat16 if dtype == svd.SVD_BF16 else torch.float32).to(DEV)
    q = torch.full((T, max(Hq, 1), 128), -7.0, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(T, dtype=torch.int32, device=DEV)
    p = to_dev(pool.reshape(-1).copy())
    pos = None if positions is None else to_dev(np.ascontiguousarray(positions, np.int32))
    tab = to_dev(np.ascontiguousarray(table, np.int32))
    svd.svd_paged8_append(rows, ld, T, Hq, Hkv, to_dev(np.array(lens, np.int32)), to_dev(q_start), len(lens), tab, tab.shape[1], p,
                          page, len(pool), q, rope=rope, positions=pos, positions_ld=0 if pos is None else pos.shape[-1],
                          dtype=dtype, status=status, stream=stream)
    torch.cuda.synchronize()
    return q.double().cpu().numpy(), p.cpu().numpy().reshape(pool.shape), status.cpu().numpy()


def check_q(got, want):
    """One rounding to bf16 (2^-9 relative is half its step) of a sum of two fp32 products (2^-22 of their magnitudes)."""
    mag = np.abs(want).max(-1, keepdims=True)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * mag + 1e-30)


# lens (with the new tokens), new tokens
FEW = ([17, 5, 64, 33, 16, 130, 3], [1, 5, 4, 1, 2, 7, 0])
MANY = ([700, 33, 300, 16, 90, 1], [640, 17, 128, 16, 33, 1])


@pytest.mark.parametrize("dtype", [svd.SVD_F32, svd.SVD_BF16])
@pytest.mark.parametrize("lens,new,Hq,Hkv,page,axes,pairs,inter,pad", [
    (*FEW, 5, 1, 16, 1, 64, False, 0), (*FEW, 0, 2, 48, 2, 12, True, 8), (*FEW, 3, 3, 256, 4, 32, False, 1024),
    (*MANY, 3, 5, 32, 3, 64, True, 0), (*MANY, 9, 8, 128, 3, 32, False, 16), (*MANY, 1, 5, 16, 1, 4, False, 0)])
def test_append(dtype, lens, new, Hq, Hkv, page, axes, pairs, inter, pad):
    g = np.random.default_rng(page + axes)
    table, q_start, n_pages = layout(lens, new, page, g)
    pool = random_pool(g, n_pages, Hkv, page)
    T, heads = int(q_start[-1]), Hq + 2 * Hkv
    x = g.normal(0, 1, (T, heads, 128)).astype(np.float32) * 2.0 ** g.integers(-4, 5, (T, 1, 1))
    x = as_type(x, dtype).float().numpy()
    pos = g.integers(0, 300000, (axes, T))
    pos[:, 0] = 0  # an angle of zero: keys as they came, many of them on a border
    pos[:, T // 2] = 0
    inv = 1e6 ** (-np.arange(pairs) / pairs)
    axis = g.integers(0, axes, pairs)
    args = (lens, q_start, table)
    q, got, st = gpu_append(x, dtype, Hq, Hkv, *args, pool, page, rope=svd.Rope(inv, axis, axes, inter), positions=pos, ld=heads * 128 + pad)
    y = paged.rotate(x.astype(np.float64), pos, inv, axis, inter)
    want = pool.copy()
    assert not paged8.append(want, y[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *args, page)
    assert np.array_equal(same_zeros(got), same_zeros(want))
    assert not st.any()
    if Hq:
        check_q(q, y[:, :Hq])
    # without rotation
    q, got, st = gpu_append(x, dtype, Hq, Hkv, *args, pool, page, ld=heads * 128 + pad)
    want = pool.copy()
    paged8.append(want, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], *args, page)
    assert np.array_equal(same_zeros(got), same_zeros(want)) and not st.any()
    if Hq:
        assert np.array_equal(q, as_type(x[:, :Hq], svd.SVD_BF16).double().numpy())


@pytest.mark.parametrize("dtype", [svd.SVD_F32, svd.SVD_BF16])
@pytest.mark.parametrize("Hq,new", [(37, 4), (40, None)])
def test_append_of_many_windows(dtype, Hq, new):
    """256 tokens of 64 requests, begun at every place of a unit, behind positions whose scales they raise or not: query heads that are
    no multiple of a CTA's, two of them to a warp; rows behind the last token stay as they are."""
    g = np.random.default_rng(Hq)
    n_new = np.full(64, 4) if new else np.bincount(np.repeat(np.arange(64), 4)[g.integers(0, 256, 253)], minlength=64)
    lens = n_new + np.arange(64) + g.integers(0, 3, 64) * 16
    table, q_start, n_pages = layout(lens.tolist(), n_new.tolist(), 32, g)
    pool = random_pool(g, n_pages, 8, 32, e_lo=-9, e_hi=-5)
    T, pad = int(q_start[-1]), 256 - int(q_start[-1])
    x = as_type(g.normal(0, 1, (T, Hq + 16, 128)).astype(np.float32) * 2.0 ** g.integers(-3, 4, (T, 1, 1)), dtype).float().numpy()
    pos = np.zeros((1, 256), np.int64)
    pos[0, :T] = np.concatenate([np.arange(n - k, n) for n, k in zip(lens, n_new)])
    inv = 1e4 ** (-np.arange(64) / 64)
    args = (lens.tolist(), q_start, table)
    q, got, st = gpu_append(x, dtype, Hq, 8, *args, pool, 32, rope=svd.Rope(inv), positions=pos, T=T + pad)
    y = paged.rotate(x.astype(np.float64), pos[:, :T], inv, [0] * 64, False)
    want = pool.copy()
    assert not paged8.append(want, y[:, Hq:Hq + 8], x[:, Hq + 8:], *args, 32)
    assert np.array_equal(same_zeros(got), same_zeros(want)) and not st.any()
    check_q(q[:T], y[:, :Hq])
    assert np.all(q[T:] == -7.0)


def test_append_next_to_the_borders_of_codes_and_scales():
    """Values on and one ulp off every border between two codes, and blocks whose largest is 448 scales or one ulp off."""
    v = paged8.VALUE[:127]
    borders = (v[1:] + v[:-1]) / 2
    rows = []
    for e in (-30, -6, 0, 7):
        for u in (-1, 0, 1):
            for top in (448.0, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(1000)), 232.0):
                b = (borders * 2.0 ** e).astype(np.float32)
                b = np.nextafter(b, np.float32(np.inf) * u) if u else b
                b[np.abs(b) > top * 2.0 ** e] = 1.0 * 2.0 ** e
                b = np.concatenate([b, [np.float32(top * 2.0 ** e), -b[40]]])
                rows.append(np.stack([b, -b]))
    x = np.array(rows, np.float32)                                   # [T, 2, 128]: a key and a value each
    T = len(x)
    lens, q_start = [1] * T, np.arange(T + 1, dtype=np.int32)       # a unit to each
    table = np.arange(T, dtype=np.int32)[:, None]
    pool = np.zeros((T, 1, 1, paged8.UNIT), np.uint8)
    _, got, st = gpu_append(x, svd.SVD_F32, 0, 1, lens, q_start, table, pool, 16)
    want = pool.copy()
    paged8.append(want, x[:, :1].astype(float), x[:, 1:].astype(float), lens, q_start, table, 16)
    assert np.array_equal(got, want) and not st.any()


def test_append_rotated_keys_at_the_borders():
    """Many rotated keys: turned back onto borders of codes and of scales, they come out as in fp64."""
    g = np.random.default_rng(78)
    T, H = 512, 2
    inv = np.zeros(64)
    inv[::3] = 0.25
    pos = g.integers(0, 40, (1, T))
    v = paged8.VALUE[:127]
    borders = (v[1:] + v[:-1]) / 2
    y = g.choice(borders, (T, 2 * H, 128)) * g.choice([-1, 1], (T, 2 * H, 128))
    y[:, :, 5] = 448.0
    x = paged.rotate(y, -pos, inv, [0] * 64, False).astype(np.float32)  # (rounded: next to the borders)
    table, q_start, n = np.arange(T // 64, dtype=np.int32)[None], np.array([0, T], np.int32), T // 64
    pool = np.zeros((n, H, 4, paged8.UNIT), np.uint8)
    _, got, _ = gpu_append(x, svd.SVD_F32, 0, H, [T], q_start, table, pool, 64, rope=svd.Rope(inv), positions=pos)
    turned = paged.rotate(x.astype(np.float64), pos, inv, [0] * 64, False)
    want = pool.copy()
    paged8.append(want, turned[:, :H], x[:, H:], [T], q_start, table, 64)
    # a key whose exact value lies within 2^-44 of a border may fall on either side in the reference's own arithmetic
    assert np.array_equal(got[..., 2048:], want[..., 2048:])
    assert np.mean(same_zeros(got) != same_zeros(want)) == 0.0


def test_a_scale_grows_once_and_earlier_codes_follow():
    """Tokens one by one into a unit, each four times the last: the scale grows, codes become subnormal and 0."""
    g = np.random.default_rng(3)
    pool = np.zeros((1, 2, 1, paged8.UNIT), np.uint8)
    want = pool.copy()
    table = np.zeros((1, 1), np.int32)
    for i in range(16):
        x = (g.normal(0, 1, (1, 4, 128)) * 4.0 ** (i - 8)).astype(np.float32)
        _, pool, st = gpu_append(x, svd.SVD_F32, 0, 2, [i + 1], np.array([0, 1], np.int32), table, pool, 16)
        paged8.append(want, x[:, :2].astype(float), x[:, 2:].astype(float), [i + 1], [0, 1], table, 16)
        assert np.array_equal(same_zeros(pool), same_zeros(want)) and not st.any()
    # a shorter request begins the unit anew
    x = g.normal(0, 1, (1, 4, 128)).astype(np.float32) * 2.0 ** -9
    _, pool, _ = gpu_append(x, svd.SVD_F32, 0, 2, [1], np.array([0, 1], np.int32), table, pool, 16)
    paged8.append(want, x[:, :2].astype(float), x[:, 2:].astype(float), [1], [0, 1], table, 16)
    assert np.array_equal(same_zeros(pool), same_zeros(want))


def test_append_reports_what_is_not_finite_and_positions_without_a_page():
    x = np.ones((8, 3, 128), np.float32)
    x[1, 1, 4], x[2, 2, 9], x[3, 1, 100], x[4, 0, 0], x[5, 1, 7] = np.nan, np.inf, -np.inf, np.nan, 1e30
    pool = np.zeros((2, 1, 1, paged8.UNIT), np.uint8)
    # request 0: six positions; request 1: a page outside the pool; request 2: a position before 0
    lens, q_start = [6, 1, 0], np.array([0, 6, 7, 8], np.int32)
    for bad in (-1, 2, 2 ** 31 - 1):
        table = np.array([[1], [bad], [0]], np.int32)
        _, got, st = gpu_append(x, svd.SVD_F32, 1, 1, lens, q_start, table, pool, 16)
        assert st.tolist() == [0, paged8.NONFINITE, paged8.NONFINITE, paged8.NONFINITE, 0, 0, paged8.BAD_SLOT, paged8.BAD_SLOT]
        want = pool.copy()
        assert paged8.append(want, x[:, 1:2].astype(float), x[:, 2:].astype(float), lens, q_start, table, 16) == [6, 7]
        assert np.array_equal(got, want)
        assert not np.isin(got[..., :4096] % 128, 127).any()


@pytest.mark.parametrize("dtype", [svd.SVD_F32, svd.SVD_BF16])
@pytest.mark.parametrize("inter", [False, True])
def test_append_rotates_what_is_not_finite_as_the_formula_says(dtype, inter):
    """NaN, infinities and magnitudes up to fp32's largest among rotated keys, and among values; beside them ordinary tokens."""
    g = np.random.default_rng(31)
    T, H = 80, 3
    x = as_type(g.normal(0, 1, (T, 2 * H, 128)).astype(np.float32), dtype).float().numpy()
    odd = np.array([np.nan, np.inf, -np.inf, 1e30, -3e38, 60000.0, 1e-40, 0.0, -0.0], np.float32)
    for t in range(0, T, 3):
        for _ in range(4):
            x[t, g.integers(0, 2 * H), g.integers(0, 128)] = odd[g.integers(0, len(odd))]
    x = as_type(x, dtype).float().numpy()
    pos = g.integers(0, 1000, (1, T))
    pos[0, ::7] = 0
    inv = 100.0 ** (-np.arange(32) / 32)
    lens, new = [T, 9], [T - 9, 9]
    table, q_start, n_pages = layout(lens, new, 32, g)
    pool = random_pool(g, n_pages, H, 32)
    _, got, st = gpu_append(x, dtype, 0, H, lens, q_start, table, pool, 32, rope=svd.Rope(inv, interleaved=inter), positions=pos)
    with np.errstate(invalid="ignore", over="ignore"):
        y = paged.rotate(x.astype(np.float64), pos, inv, [0] * 32, inter)
    want = pool.copy()
    paged8.append(want, y[:, :H], x[:, H:], lens, q_start, table, 32)
    assert np.array_equal(same_zeros(got), same_zeros(want))
    assert np.array_equal(st, np.where(np.isfinite(x).all((1, 2)), 0, paged8.NONFINITE))


@pytest.mark.parametrize("T", [40, 700])
def test_rows_behind_the_last_request_are_left_alone(T):
    g = np.random.default_rng(T)
    lens, new = [T - 20, 9], [T - 25, 9]
    table, q_start, n_pages = layout(lens, new, 32, g)
    pool = random_pool(g, n_pages, 6, 32)
    x = g.normal(0, 1, (int(q_start[-1]), 16, 128)).astype(np.float32)
    q, got, st = gpu_append(x, svd.SVD_F32, 4, 6, lens, q_start, table, pool, 32, T=T)
    want = pool.copy()
    paged8.append(want, x[:, 4:10].astype(float), x[:, 10:].astype(float), lens, q_start, table, 32)
    assert np.array_equal(same_zeros(got), same_zeros(want)) and not st.any()
    assert (q[len(x):] == -7).all() and (q[:len(x)] != -7).any()


def test_append_of_many_requests():
    g = np.random.default_rng(8)
    R = 4096
    lens = g.integers(1, 40, R)
    new = np.minimum(lens, g.integers(0, 3, R))
    table, q_start, n_pages = layout(lens, new, 16, g)
    pool = random_pool(g, n_pages, 1, 16)
    x = g.normal(0, 1, (int(q_start[-1]), 2, 128)).astype(np.float32)
    _, got, st = gpu_append(x, svd.SVD_F32, 0, 1, lens, q_start, table, pool, 16)
    want = pool.copy()
    paged8.append(want, x[:, :1].astype(float), x[:, 1:].astype(float), lens, q_start, table, 16)
    assert np.array_equal(same_zeros(got), same_zeros(want)) and not st.any()


@pytest.mark.parametrize("page,H", [(16, 1), (48, 3), (128, 8)])
def test_read(page, H):
    g = np.random.default_rng(page)
    pool = random_pool(g, 4, H, page)
    slots = np.concatenate([g.permutation(4 * page)[:50], [-1, 4 * page, 2 ** 40]])
    k = torch.full((len(slots), H, 128), float("nan"), device=DEV)
    v = torch.full_like(k, float("nan"))
    svd.svd_paged8_read(torch.tensor(slots, device=DEV), len(slots), H, to_dev(pool.reshape(-1)), page, 4, k, v)
    kk, vv = paged8.get(pool, slots, page)
    assert np.array_equal(k.double().cpu().numpy(), kk) and np.array_equal(v.double().cpu().numpy(), vv)


# ---- attention ---------------------------------------------------------------------------------
class Case:
    def __init__(self, lens, new, Hq, Hkv, page, seed=0, k_exp=(-4, -1), v_exp=(-4, -1)):
        g = np.random.default_rng(seed)
        self.g, self.lens, self.new, self.Hq, self.Hkv, self.page = g, lens, new, Hq, Hkv, page
        self.table, self.q_start, self.n_pages = layout(lens, new, page, g)
        # 0xFF everywhere else: codes and scales that are no numbers
        self.pool = np.full((self.n_pages, Hkv, page // 16, paged8.UNIT), 0xFF, np.uint8)
        for r, x in enumerate(lens):  # values of both signs up to about 4 * 2^e, and codes of all sizes
            for c in range(-(-max(x, 0) // page)):
                for u in range(-(-min(page, x - c * page) // 16)):
                    unit = self.pool[self.table[r, c], :, u]
                    m = min(16, x - c * page - 16 * u)
                    codes = g.integers(0x28, 0x50, (2, Hkv, m, 128)) | g.choice([0, 128], (2, Hkv, m, 128))
                    codes[..., 5] = g.integers(0, 127, (2, Hkv, m))
                    for i in range(m):
                        unit[:, paged8.k_bytes(i)] = codes[0, :, i]
                        unit[:, paged8.v_bytes(i)] = codes[1, :, i]
                    scales = 2.0 ** np.stack([g.integers(*k_exp, Hkv), g.integers(*v_exp, Hkv)], -1)
                    unit[:, 4096:4104] = scales.astype(np.float32).view(np.uint8)
        self.T = int(self.q_start[-1])
        self.q = torch.from_numpy(g.normal(0, 1, (max(self.T, 1), Hq, 128))).to(torch.bfloat16)
        self.scale = 128 ** -0.5
        self.largest = 448 * 2.0 ** (v_exp[1] - 1)  # of the values

    def run(self, out_dtype, max_new=None, T=None, ws=None, stream=None, table=None, out=None):
        T = self.T if T is None else T
        most = max(1, max(self.new)) if max_new is None else max_new
        dt = torch.bfloat16 if out_dtype == svd.SVD_BF16 else torch.float32
        q = torch.zeros((T, self.Hq, 128), dtype=torch.bfloat16)
        q[:self.T] = self.q[:self.T]
        if out is None:
            out = torch.full((T, self.Hq, 128), -7.0, dtype=dt, device=DEV)
        if ws is None:
            ws = torch.zeros(svd.svd_paged8_attention_workspace_bytes(self.Hq, self.Hkv, len(self.lens), most),
                             dtype=torch.uint8, device=DEV)
        tab = to_dev(self.table if table is None else table)
        self.keep = (q.to(DEV), to_dev(np.array(self.lens, np.int32)), to_dev(self.q_start), tab, to_dev(self.pool.reshape(-1)), ws)
        torch.cuda.synchronize()
        svd.svd_paged8_attention(self.keep[0], T, self.keep[1], self.keep[2], len(self.lens), most, tab, tab.shape[1],
                                 self.keep[4], self.page, self.n_pages, self.Hq, self.Hkv, self.scale, out, out_dtype, ws,
                                 stream=stream)
        torch.cuda.synchronize()
        assert ws[:4].view(torch.int32).item() == 0
        return out.double().cpu().numpy()

    def reference(self, **kw):
        return paged8.attention(self.q.double().numpy(), self.pool, self.page, kw.pop("table", self.table), self.lens,
                                self.q_start, self.scale, **kw)

    def check(self, out_dtype, got, ref):
        o, a, e = ref[:3]
        n = max(max(self.lens), 1)
        # scores: 128 products of each part added with 2^-23 each, the parts and the factors 2^-22; p: that,
        # its exponent's 2^-20, and for bf16 outputs its rounding to fp16 (2^-11), for fp32 outputs what
        # its two parts leave (2^-21); the sums over positions: 2^-23 an addition (fp32 outputs: within a tile, then
        # over the tiles); and fp16's smallest step: the weight of a code is held to 2^-25 where the largest one is
        # 2^7 or more, so what a position adds is good to 2^-32 of the largest value
        score = 2.0 ** -15 * e[..., None]
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
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (8, 1), (10, 2), (13, 1), (24, 2), (32, 1), (40, 1), (70, 70)])
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


@BOTH
def test_a_long_window_over_many_ctas(out_dtype):
    c = Case([5000, 300], [90, 130], 3, 1, 64, seed=21)
    c.check(out_dtype, c.run(out_dtype), c.reference())


def test_attention_many_requests():
    g = np.random.default_rng(4)
    lens = g.integers(1, 60, 700).tolist()
    c = Case(lens, g.integers(0, 2, 700).tolist(), 2, 1, 16, seed=5)
    c.check(svd.SVD_BF16, c.run(svd.SVD_BF16), c.reference())
    c = Case([20] * 4096, [1] * 4096, 1, 1, 16, seed=6)
    c.check(svd.SVD_BF16, c.run(svd.SVD_BF16), c.reference())


@BOTH
def test_many_row_tiles_split_between_two_ctas(out_dtype):
    g = np.random.default_rng(22)
    lens = g.integers(300, 900, 95).tolist()
    c = Case(lens, [1] * 95, 4, 4, 64, seed=23)
    c.check(out_dtype, c.run(out_dtype), c.reference())


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
    o, a, e, _ = c.reference(max_new=4)
    pad = np.full((3, 4, 128), np.nan)
    c.check(out_dtype, got, (np.concatenate([o, pad]), np.concatenate([a, pad]), np.concatenate([e, pad[..., 0]])))


@BOTH
@pytest.mark.parametrize("k_exp", [(-64, -63), (-12, -10), (2, 3)])
def test_scores_of_any_spread(out_dtype, k_exp):
    """Scores of 0; scores near 0; scores of some hundred, so that one position takes all."""
    c = Case([700, 1300], [3, 1], 5, 1, 64, seed=10, k_exp=k_exp)
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
def test_scales_of_values_far_apart(out_dtype):
    """Blocks of values whose scales lie between 2^-64 and 2^7, beside scores of all sizes."""
    c = Case([1000, 290], [3, 2], 5, 1, 64, seed=18, k_exp=(-2, 2), v_exp=(-64, 8))
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
def test_small_values_behind_large_ones_that_weigh_nothing(out_dtype):
    """The first block's values are 2^20 times the others', and its scores so low that it takes no part."""
    c = Case([400], [1], 4, 1, 16, seed=19, k_exp=(0, 1), v_exp=(-16, -15))
    unit = c.pool[c.table[0, 0], 0, 0]
    for i in range(16):
        unit[paged8.k_bytes(i)] = np.where(c.q[0, 0].float().numpy() > 0, 0xF0, 0x70)  # against the query
    unit[4100:4104] = np.array([2.0 ** 4], np.float32).view(np.uint8)
    c.q[:] = c.q[:1, :1]
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
def test_rising_scores_move_the_reference(out_dtype):
    """Key scales that grow along the cache: the largest score rises from tile to tile."""
    c = Case([1500], [4], 5, 1, 16, seed=11)
    for p in range(0, 1500, 16):
        c.pool[c.table[0, p // 16], 0, 0, 4096:4100] = np.array([2.0 ** (-10 + p // 128)], np.float32).view(np.uint8)
    c.check(out_dtype, c.run(out_dtype), c.reference())


@BOTH
def test_queries_of_any_magnitude(out_dtype):
    """Rows up to 2^60 and down to 2^-60, and rows with one large element, beside ordinary ones."""
    c = Case([300, 150], [4, 2], 5, 1, 64, seed=20, k_exp=(-3, -2))
    for t, e in ((0, 60), (1, -60), (2, -130)):
        c.q[t, 2] = c.q[t, 2] * 2.0 ** e
    k_small = Case([300, 150], [4, 2], 5, 1, 64, seed=20, k_exp=(-64, -63))
    k_small.q = c.q.clone()
    k_small.check(out_dtype, k_small.run(out_dtype), k_small.reference())
    c.q[0, 2] = 0
    c.q[3, 1, 7] *= 2.0 ** 7
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


@BOTH
@pytest.mark.parametrize("Hq,most", [(8, 1), (32, 4), (24, 7), (72, 7)])
def test_many_short_segments(out_dtype, Hq, most):
    """700 requests of one or two tiles and eight heads: some twenty segments to a CTA, more than there are descriptors of
    them in flight, in row tiles of 8, 16, 24 and 64 (fp32: 32) rows; some requests without positions or tokens."""
    g = np.random.default_rng(Hq)
    new = g.integers(0, most + 1, 700)
    lens = np.where(g.random(700) < 0.05, new, new + g.integers(0, 200, 700))
    c = Case(lens.tolist(), new.tolist(), Hq, 8, 256, seed=Hq)
    c.check(out_dtype, c.run(out_dtype), c.reference())


@pytest.mark.parametrize("new", [12, 40, 129])
@pytest.mark.parametrize("content", ["magnitudes", "small", "not finite", "rising", "scales", "spread", "missing pages"])
def test_contents_in_long_row_tiles(content, new):
    """What the tests above bring to windows, in row tiles of 64 and of 128 rows, the last ones part full."""
    k_exp, v_exp = {"magnitudes": ((-64, -63), (-4, -1)), "small": ((-40, -30), (-4, -1)), "scales": ((-2, 2), (-64, 8)),
                    "spread": ((2, 3), (-4, -1))}.get(content, ((-4, -1), (-4, -1)))
    c = Case([300, 150, 700], [new, 3, min(new, 60)], 5, 1, 32, seed=30 + new, k_exp=k_exp, v_exp=v_exp)
    if content == "magnitudes":  # k_exp keeps the scores of the largest rows finite
        for t in range(c.T):
            c.q[t, t % 5] = c.q[t, t % 5] * 2.0 ** (60, -60, -130, 7)[t % 4]
        c.q[4, 1, 7] *= 2.0 ** 7
        c.q[5, 3] = 0
    if content == "rising":
        for p in range(0, 700, 16):
            c.pool[c.table[2, p // 32], 0, p % 32 // 16, 4096:4100] = np.array([2.0 ** (-10 + p // 64)], np.float32).view(np.uint8)
    if content == "missing pages":
        c.table[0, 0], c.table[0, 7], c.table[2, 3:12], c.table[1] = -1, c.n_pages, 2 ** 31 - 1, -9
    ref = c.reference()
    if content == "not finite":
        c.q[2, 3, 7], c.q[new + 1, 0, :] = float("nan"), float("inf")
    got = c.run(svd.SVD_BF16)
    if content == "not finite":
        assert np.isnan(got[2, 3]).all() and np.isnan(got[new + 1, 0]).all()
        got[2, 3], got[new + 1, 0] = ref[0][2, 3], ref[0][new + 1, 0]
    c.check(svd.SVD_BF16, got, ref)


def test_offsets_past_32_bits():
    """A pool of 5 GB with the request's pages at its end."""
    c = Case([100], [2], 8, 8, 256, seed=13)
    small = c.run(svd.SVD_BF16)
    per = 8 * 16 * paged8.UNIT
    n_pages = 5 * 2 ** 30 // per
    pool = torch.empty(n_pages * per, dtype=torch.uint8, device=DEV)
    pool[(n_pages - 1) * per:] = to_dev(c.pool[c.table[0, 0]].reshape(-1))
    tab = torch.tensor([[n_pages - 1]], dtype=torch.int32, device=DEV)
    out = torch.empty((2, 8, 128), dtype=torch.bfloat16, device=DEV)
    svd.svd_paged8_attention(c.keep[0], 2, c.keep[1], c.keep[2], 1, 2, tab, 1, pool, 256, n_pages, 8, 8, c.scale, out,
                             svd.SVD_BF16, c.keep[5])
    assert np.array_equal(out.double().cpu().numpy(), small)
    # append and read there too
    x = torch.randn((1, 24 * 128), device=DEV)
    slot = torch.tensor([n_pages * 256 - 16], device=DEV)
    k, v = torch.empty((1, 8, 128), device=DEV), torch.empty((1, 8, 128), device=DEV)
    one = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    svd.svd_paged8_append(x, 24 * 128, 1, 8, 8, one(241), one(0, 1), 1, tab, 1, pool, 256, n_pages,
                          torch.empty((1, 8, 128), dtype=torch.bfloat16, device=DEV))
    svd.svd_paged8_read(slot, 1, 8, pool, 256, n_pages, k, v)
    want = np.zeros((1, 8, 16, paged8.UNIT), np.uint8)
    rows = x.double().cpu().numpy().reshape(1, 24, 128)
    paged8.append(want, rows[:, 8:16], rows[:, 16:], [241], [0, 1], np.zeros((1, 1), int), 256)
    kk, vv = paged8.get(want, [240], 256)
    assert np.array_equal(k.double().cpu().numpy(), kk) and np.array_equal(v.double().cpu().numpy(), vv)


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
        svd.svd_paged8_attention(q, c.T, lens, starts, 3, 3, tab, tab.shape[1], pool, 32, c.n_pages, 10, 2, c.scale, out,
                                 svd.SVD_BF16, ws, stream=s)
    g = svd.svd_graph_end(s)
    g.launch(s)
    g.launch(s)
    s.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), first)


def test_a_wait_that_runs_out_is_reported_and_does_not_hang():
    """The second word of the workspace lets every wait that is not satisfied at once give up."""
    for lens, new in (([5000, 600], [4, 2]), ([5000, 600], [60, 2])):
        c = Case(lens, new, 10, 2, 32, seed=15)
        want = c.run(svd.SVD_BF16)
        ws = c.keep[5]
        for out_dtype in (svd.SVD_BF16, svd.SVD_F32):
            out = torch.zeros((c.T, 10, 128), dtype=torch.bfloat16 if out_dtype == svd.SVD_BF16 else torch.float32, device=DEV)
            ws[:8].view(torch.int32)[1] = 1
            svd.svd_paged8_attention(c.keep[0], c.T, c.keep[1], c.keep[2], 2, max(new), c.keep[3], c.keep[3].shape[1], c.keep[4], 32,
                                     c.n_pages, 10, 2, c.scale, out, out_dtype, ws)
            torch.cuda.synchronize()
            assert ws[:8].view(torch.int32)[0].item() == 1
            ws[:8] = 0
        assert np.array_equal(c.run(svd.SVD_BF16, ws=ws), want)


def test_nothing_is_written_beside_the_outputs():
    c = Case([400, 30], [3, 2], 10, 2, 32, seed=16)
    big = torch.full((c.T * 10 * 128 + 512,), -7.0, dtype=torch.bfloat16, device=DEV)
    n = svd.svd_paged8_attention_workspace_bytes(10, 2, 2, 3)
    ws = torch.full((n + 512,), 0, dtype=torch.uint8, device=DEV)
    ws[n:] = 0xEE
    c.run(svd.SVD_BF16, ws=ws[:n], out=big[256:256 + c.T * 1280].view(c.T, 10, 128))
    assert (big[:256] == -7).all() and (big[-256:] == -7).all() and (ws[n:] == 0xEE).all()
