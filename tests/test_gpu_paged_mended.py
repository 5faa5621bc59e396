"""The paged calls on the GPU in cases that once went wrong, against the fp64 reference: waits that give up
with the copies of a short range in flight; one row of positions for several axes; rotated keys that are not finite or too
large for fp32; masks of many heads far behind the window; small
probabilities in fp32 outputs; keys of very small and very large scales; queries
beyond fp16."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from speculative_decoding_verify_06_gb300 import paged, svd
from tests.gpu_helpers import DEV, lib, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def random_pool(g, n_pages, Hkv, page):
    """Pages of normal keys and values."""
    pool = np.zeros((n_pages, Hkv, page // 16, ref.UNIT), np.uint8)
    n = n_pages * page
    return ref.put(pool, np.arange(n), g.normal(size=(n, Hkv, 128)), g.normal(size=(n, Hkv, 128)), page)


class Attend:
    """One attention call: lens and new tokens of each request, its pages in order unless a table is given."""

    def __init__(self, lens, new, Hq, Hkv, page, out_dtype=svd.SVD_BF16, seed=0, pool=None, table=None, q=None):
        g = np.random.default_rng(seed)
        have = [-(-x // page) for x in lens]
        if table is None:
            table = np.full((len(lens), max(have)), -1, np.int32)
            for r, n in enumerate(have):
                table[r, :n] = sum(have[:r]) + np.arange(n)
        self.lens, self.page, self.Hq, self.Hkv, self.out_dtype, self.table = lens, page, Hq, Hkv, out_dtype, table
        self.pool = random_pool(g, sum(have), Hkv, page) if pool is None else pool
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.T, self.most, self.scale = int(self.q_start[-1]), max(new), 128 ** -0.5
        self.q = torch.from_numpy(g.normal(size=(self.T, Hq, 128)) if q is None else q).to(torch.bfloat16)
        self.dev = [self.q.to(DEV), to_dev(np.array(lens, np.int32)), to_dev(self.q_start), to_dev(table), to_dev(self.pool.reshape(-1))]
        self.ws = torch.zeros(svd.svd_paged_attention_workspace_bytes(Hq, Hkv, len(lens), self.most), dtype=torch.uint8, device=DEV)
        self.out = torch.full((self.T, Hq, 128), -7.0, dtype=torch.bfloat16 if out_dtype == svd.SVD_BF16 else torch.float32,
                              device=DEV)

    def run(self):
        q, lens, starts, table, pool = self.dev
        svd.svd_paged_attention(q, self.T, lens, starts, len(self.lens), self.most, table, table.shape[1], pool, self.page,
                                self.pool.shape[0], self.Hq, self.Hkv, self.scale, self.out, self.out_dtype, self.ws)
        torch.cuda.synchronize()
        return self.out.double().cpu().numpy()

    def reference(self):
        return ref.attention(self.q.double().numpy(), self.pool, self.page, self.table, self.lens, self.q_start, self.scale)


@pytest.mark.parametrize("polls", [1, 2, 5])
@pytest.mark.parametrize("lens,new,Hq", [([130, 260], [1, 4], 10), ([100] * 40, [3] * 40, 10), ([700, 900], [40, 70], 8), ([40], [1], 2)])
def test_waits_that_give_up_after_the_last_copy_is_issued(lens, new, Hq, polls):
    """Ranges of no more tiles than the ring has stages: the copying warp never waits.  It must still let
    its copies land, and the next calls (over the same shared memory) give what they gave before."""
    c = Attend(lens, new, Hq, 2, 32)
    want = c.run()
    for _ in range(3):
        c.ws[:8].view(torch.int32)[1] = polls
        c.run()
        c.ws[:8] = 0
        assert np.array_equal(c.run(), want) and not c.ws[:4].any()


@pytest.mark.parametrize("given", [None, "row", "axes"])
def test_a_step_with_several_axes(given):
    """Text tokens turn by the same position on every axis, image tokens by each axis' own."""
    g = np.random.default_rng(2)
    T, Hq, Hkv, page, n = 9, 3, 1, 16, 64
    inv, axis = 100.0 ** (-np.arange(n) / n), np.arange(n) % 3
    b = paged.PagedBatch(2, 1, n_pages=8, page_size=page, max_len=64, max_window=5, n_q_heads=Hq, n_kv_heads=Hkv,
                         rope=svd.Rope(inv, axis, 3))
    b.begin(torch.tensor([4, 5], dtype=torch.int32, device=DEV))
    text = np.array([0, 1, 2, 3, 0, 1, 2, 3, 4])
    pos = {None: np.stack([text] * 3), "row": np.stack([text + 7] * 3), "axes": g.integers(0, 5000, (3, T))}[given]
    x = g.normal(size=(T, 5, 128)).astype(np.float32)
    arg = None if given is None else to_dev(pos[0].astype(np.int32) if given == "row" else pos.astype(np.int32))
    out = torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device=DEV)
    b.layer(0, to_dev(x.reshape(T, -1)), out, n_tokens=T, positions=arg)
    y = ref.rotate(x.astype(np.float64), pos, inv, axis, False)
    q = b.q[:T].double().cpu().numpy()
    # bf16's rounding, and the rotation before it
    assert np.all(np.abs(q - y[:, :Hq]) <= 2.0 ** -8 * np.abs(y[:, :Hq]) + 2.0 ** -17)
    want = ref.put(np.zeros((8, Hkv, 1, ref.UNIT), np.uint8), b.slots[:T].cpu().numpy(), y[:, Hq:Hq + 1], x[:, Hq + 1:].astype(float), page)
    assert np.array_equal(b.pools[0].cpu().numpy().reshape(want.shape), want) and not b.bad.any()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pairs", [64, 20])
def test_rotated_keys_that_are_not_finite(pairs, interleaved):
    """An infinite key is infinite after the rotation (the largest magnitude), not a NaN (0); finite ones that
    leave fp32's range are not reported; blocks beside them get the codes of exact arithmetic."""
    g = np.random.default_rng(pairs + interleaved)
    T, page = 600, 64
    x = g.normal(size=(T, 2, 128)).astype(np.float32)
    odd = g.random(T) < 0.5
    for t in range(T):
        big = [np.inf, -np.inf, np.nan, 3.3e38, -3e38, 7e4]
        for d in g.integers(0, 128, g.integers(0, 4)):
            x[t, 0, d] = big[g.integers(0, 6)] if odd[t] else big[g.integers(3, 6)]
        # a block of values near the borders of its codes, wherever it is
        x[t, 0, 96:] = ((np.arange(32) % 16) - 7.5).astype(np.float32) if pairs == 20 else x[t, 0, 96:]
    pos = g.integers(1, 4000, (1, T))
    inv = g.uniform(0.05, 1.0, pairs)
    pool = torch.zeros(10 * 4 * ref.UNIT, dtype=torch.uint8, device=DEV)
    status = torch.zeros(T, dtype=torch.int32, device=DEV)
    svd.svd_paged_append(to_dev(x.reshape(T, -1)), 256, T, 0, 1, torch.arange(T, device=DEV), pool, page, 10, None,
                         rope=svd.Rope(inv, interleaved=interleaved), positions=to_dev(pos.astype(np.int32)), positions_ld=T,
                         status=status)
    with np.errstate(invalid="ignore", over="ignore"):
        y = ref.rotate(x.astype(np.float64), pos, inv, [0] * pairs, interleaved)
    want = ref.put(np.zeros((10, 1, 4, ref.UNIT), np.uint8), np.arange(T), y[:, :1], x[:, 1:].astype(float), page)
    assert np.array_equal(pool.cpu().numpy().reshape(want.shape), want)
    assert np.array_equal(status.cpu().numpy() != 0, ~np.isfinite(x).all((1, 2)))


@pytest.mark.parametrize("out_dtype", [svd.SVD_BF16, svd.SVD_F32])
def test_a_missing_page_far_behind_a_window_of_many_heads(out_dtype):
    """8.5 million positions before the window, 256 heads to a kv head: the product of both passes 32 bits.
    The first page is missing; the second, which shares its tile, holds about half of the weight."""
    page, G, cols = 64, 256, 132800
    g = np.random.default_rng(4)
    k, v = np.zeros((2 * page, 1, 128)), g.normal(size=(2 * page, 1, 128))
    k[:page] = 1.0
    pool = ref.put(np.zeros((2, 1, 4, ref.UNIT), np.uint8), np.arange(2 * page), k, v, page)
    table = np.ones((1, cols), np.int32)
    table[0, :2] = -1, 0
    q = np.full((1, G, 128), 11.8 / 128 * 128 ** 0.5)
    q += g.normal(0, 0.05, q.shape)
    c = Attend([cols * page], [1], G, 1, page, out_dtype, pool=pool, table=table, q=q)
    got = c.run()[0]
    kk, vv = ref.get(pool, np.arange(2 * page), page)
    times = np.repeat([1.0, cols - 2.0], page)
    s = c.q[0].double().numpy() @ kk[:, 0].T * c.scale
    p = np.exp(s - s.max(1, keepdims=True)) * times
    p /= p.sum(1, keepdims=True)
    assert np.all((p[:, :page].sum(1) > 0.2) & (p[:, :page].sum(1) < 0.8))
    # the output's 2^-8, P's 2^-11, scores of 12 good to 2^-16 (twice), 2^14 truncated additions: below 2^-7 together
    assert np.all(np.abs(got - p @ vv[:, 0]) <= 2.0 ** -7 * (p @ np.abs(vv[:, 0])))


def test_a_long_tail_behind_one_large_probability():
    """fp32 outputs: one position takes nearly all, 4096 others 2^-21.6 of it each, between two steps of fp16's
    subnormals.  Its value is 0 and theirs are 1, so the output is the tail's share of the sum.  Requests
    enough that a CTA holds the first position and a long tail."""
    page, n, R, scale = 64, 4096, 256, 128 ** -0.5
    for key in range(128, 256):  # an eight-bit key for which the tail lies about half way between two steps
        m = 5.5 * key / 128 * 16 * scale / np.log(2.0)
        steps = 2.0 ** (31 - m)
        if 300 < steps < 900 and 0.45 < steps % 1 < 0.55:
            break
    assert 300 < steps < 900 and 0.45 < steps % 1 < 0.55
    k, v = np.zeros((2 * page, 1, 128)), np.ones((2 * page, 1, 128))
    k[page, :, :16], v[page] = key / 128, 0.0
    pool = ref.put(np.zeros((2, 1, 4, ref.UNIT), np.uint8), np.arange(2 * page), k, v, page)
    kk, vv = ref.get(pool, np.arange(2 * page), page)
    assert np.array_equal(kk, k) and np.array_equal(vv, v)
    table = np.zeros((R, n // page + 1), np.int32)
    table[:, 0] = 1
    c = Attend([n + 1] * R, [1] * R, 4, 1, page, svd.SVD_F32, pool=pool, table=table, q=np.full((R, 4, 128), 5.5))
    got = c.run()
    tail = n * 2.0 ** -m
    # fp32 additions of equal numbers: n / 128 within a lane and 16 across them and the segments, for the sum and
    # for the output; p: its exponent's 2^-20, the exponential's and the split's 2^-22
    bound = 2 * (n / 128 + 16) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -21
    assert np.all(np.abs(got / (tail / (1 + tail)) - 1) <= bound)


def check(c, got, small_keys):
    """Bounds counted from the roundings: scores 2^-16 of sum |q k| (fp32 additions in the tensor core), small
    keys eight steps of half of 2^-22, P's 2^-11 (fp32 outputs: its two parts' 2^-21), a position's 2^-32, the sums,
    the output."""
    o, a, e = c.reference()
    n = max(c.lens)
    score = 2.0 ** -16 * e[..., None]
    if small_keys:
        score = score + 2.0 ** -20 * c.scale * np.abs(c.q.double().numpy()).sum(-1, keepdims=True)
    if c.out_dtype == svd.SVD_BF16:
        bound = 2.0 ** -8 * np.abs(o) + a * (2.0 ** -11 + 2 * score + n * 2.0 ** -23 + 2.0 ** -19) + n * 2.0 ** -32 * 8
    else:
        bound = a * (2.0 ** -21 + 2 * score + (256 + n / 128) * 2.0 ** -23 + 2.0 ** -19) + n * 2.0 ** -43 * 8
    err = np.abs(got - o)
    assert np.all(err <= bound + 1e-30), float(np.max(err / (bound + 1e-30)))


@pytest.mark.parametrize("out_dtype", [svd.SVD_BF16, svd.SVD_F32])
@pytest.mark.parametrize("new,Hq", [(4, 5), (40, 5)])
@pytest.mark.parametrize("size", [2.0 ** -23, 2.0 ** -19, 2.0 ** -15, 2.0 ** -13, 2.0 ** 9, 2.0 ** 11])
def test_keys_of_any_scale(out_dtype, new, Hq, size):
    """Keys around 8 d for d from fp16's subnormals to its largest; queries that make their scores a few units.
    Scales from 2^-15 on are exact, smaller ones rounded to multiples of 2^-22."""
    page, n = 32, 400
    g = np.random.default_rng(6)
    k = g.normal(size=(416, 1, 128))
    k *= np.minimum(2.5 * size, 60000 / np.abs(k).max())
    pool = ref.put(np.zeros((13, 1, 2, ref.UNIT), np.uint8), np.arange(416), k, g.normal(size=k.shape), page)
    d = pool.view(np.float16)[..., 1024:1088].astype(float)
    assert np.median(np.abs(d)) < 2 * size and (size < 2.0 ** 11 or np.abs(d).max() > 2720)
    q = g.normal(size=(new, Hq, 128)) * min(0.6 / size, 12000.0)
    c = Attend([n], [new], Hq, 1, page, out_dtype, pool=pool, q=q)
    check(c, c.run(), (np.abs(d) < 2.0 ** -15).any())


@pytest.mark.parametrize("lens,new", [([70, 3000], [1, 2]), ([900, 40], [300, 30])])
@pytest.mark.parametrize("value,told", [(65280.0, 0), (65536.0, 2), (-3e38, 2), (np.inf, 0), (np.nan, 0)])
def test_queries_beyond_fp16_are_reported(lens, new, value, told):
    """One such value makes its row NaN and no other; what is not finite to begin with is not reported."""
    g = np.random.default_rng(9)
    q = g.normal(size=(sum(new), 10, 128))
    c = Attend(lens, new, 10, 2, 32, q=q)
    want = c.run()
    assert c.ws[:4].view(torch.int32).item() == 0
    q[-1, 6, 77] = value
    c.dev[0].copy_(torch.from_numpy(q).to(torch.bfloat16))
    got = c.run()
    assert c.ws[:4].view(torch.int32).item() == told
    assert np.isfinite(got[-1, 6]).all() if abs(value) < 65504 else np.isnan(got[-1, 6]).all()
    got[-1, 6] = want[-1, 6]
    assert np.array_equal(got, want)
