"""PagedBatch over 8-bit pools: steps with rejected drafts, forks, compactions and requests that end, against the reference's
own pools, pages and tables; steps recorded and replayed; two batches at once."""
import numpy as np
import pytest
import torch

from oracle import paged, paged8
from speculative_decoding_verify_06_gb300 import paged as pg
from speculative_decoding_verify_06_gb300 import svd
from tests.gpu_helpers import DEV, lib
from tests.test_gpu_paged8 import same_zeros

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Model:
    """The reference beside a batch: its state, and its pools."""

    def __init__(self, b, inv):
        self.b, self.inv = b, inv
        self.held, self.window = np.zeros(b.R, np.int32), np.zeros(b.R, np.int32)
        self.table = np.full((b.R, b.width), -1, np.int32)
        self.free, self.n_free = np.arange(b.n_pages - 1, -1, -1, dtype=np.int32), b.n_pages
        shape = (b.n_pages, b.Hkv, b.page // 16, paged8.UNIT if b.bits == 8 else paged.UNIT)
        self.pools = [np.zeros(shape, np.uint8) for _ in b.pools]

    def begin(self, n_new, emitted):
        b = self.b
        o = paged.advance(self.held, self.window, emitted, n_new, b.max_window, b.page, self.table, self.free, self.n_free, b.max_tokens)
        self.held, self.window, self.table, self.free, self.n_free = (o[k] for k in ("held", "window", "table", "free", "n_free"))
        self.kv_len, self.q_start = o["kv_len"], o["q_start"]
        self.slots = o["slots"]

    def fork(self, parent, emitted):
        o = paged8.fork(self.held, self.window, emitted, parent, self.b.page, self.table, self.free, self.n_free)
        self.held, self.window, self.table, self.free, self.n_free = (o[k] for k in ("held", "window", "table", "free", "n_free"))
        self.move(o["moves"])
        return o["status"]

    def compact(self):
        o = paged8.compact(self.held, self.b.page, self.table, self.b.n_pages)
        self.table, self.free, self.n_free = o["table"], o["free"], o["n_free"]
        self.move(o["moves"])

    def move(self, moves):
        for p in self.pools:
            was = p.copy()
            for a, c in moves:
                p[c] = was[a]

    def layer(self, l, x):
        """x fp32 [T, heads, 128] as the batch got it."""
        b, T = self.b, len(x)
        pos = np.concatenate([np.arange(self.kv_len[r] - (self.q_start[r + 1] - self.q_start[r]), self.kv_len[r]) for r in range(b.R)])
        y = paged.rotate(x.astype(np.float64), pos[None], self.inv, [0] * 64, False)
        k, v = y[:, b.Hq:b.Hq + b.Hkv], x[:, b.Hq + b.Hkv:].astype(np.float64)
        if b.bits == 8:
            assert not paged8.append(self.pools[l], k, v, self.kv_len, self.q_start, self.table, b.page)
        else:
            paged.put(self.pools[l], self.slots[:T], k, v, b.page)
        return y[:, :b.Hq]

    def same_state(self):
        b = self.b
        now = b.now
        assert np.array_equal(b.table[now].cpu().numpy(), self.table) and np.array_equal(b.held[now].cpu().numpy(), self.held)
        assert np.array_equal(b.window.cpu().numpy(), self.window) and int(b.n_free[now]) == self.n_free
        assert np.array_equal(b.free[now].cpu().numpy()[:self.n_free], self.free[:self.n_free])

    def same_pools(self):
        for got, want in zip(self.b.pools, self.pools):
            got = got.cpu().numpy().reshape(want.shape)
            if self.b.bits == 8:
                got, want = same_zeros(got), same_zeros(want)
            assert np.array_equal(got, want)


def step(b, m, g, n_new, emitted, out_type=torch.bfloat16):
    b.begin(i32(n_new), None if emitted is None else i32(emitted))
    m.begin(n_new, emitted)
    m.same_state()
    assert not b.status.any()
    T = int(np.sum(n_new))
    for l in range(len(b.pools)):
        x = g.normal(0, 1, (T, b.Hq + 2 * b.Hkv, 128)).astype(np.float32) * np.float32(2.0) ** g.integers(-2, 3, (T, 1, 1))
        x = x.astype(np.float32)
        out = torch.full((max(T, 1), b.Hq, 128), -7.0, dtype=out_type, device=DEV)
        b.layer(l, torch.from_numpy(x.reshape(T, x.shape[1] * 128)).to(DEV), out, n_tokens=T)
        q = m.layer(l, x)
        got_q = b.q[:T].double().cpu().numpy()
        mag = np.abs(q).max(-1, keepdims=True) if T else 0
        assert np.all(np.abs(got_q - q) <= 2.0 ** -8 * np.abs(q) + 2.0 ** -20 * mag + 1e-30)
        if T and b.bits == 8:
            o, a, e, big = paged8.attention(got_q, m.pools[l], b.page, m.table, m.kv_len, m.q_start, b.scale)
            # as for the attention alone: scores 2^-15 of sum |q k| (twice), p 2^-11, the output 2^-8; sums below 2^-12
            bound = 2.0 ** -8 * np.abs(o) + a * (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -14 * e[..., None]) + 2.0 ** -20 * big[..., None]
            err = np.abs(out[:T].double().cpu().numpy() - o)
            assert np.all(err <= bound + 1e-30), float(np.max(err / (bound + 1e-30)))
    m.same_pools()
    assert not b.bad.any()


@pytest.mark.parametrize("bits", [8, 4])
def test_steps_forks_and_compactions(bits):
    R, page = 6, 32
    g = np.random.default_rng(bits)
    inv = 1000.0 ** (-np.arange(64) / 64)
    b = pg.PagedBatch(R, 2, n_pages=40, page_size=page, max_len=160, max_window=40, n_q_heads=6, n_kv_heads=2, rope=svd.Rope(inv),
                      max_tokens=R * 40, bits=bits)
    m = Model(b, inv)
    step(b, m, g, np.array([37, 5, 20, 1, 16, 33]), None)
    # three answers to request 0's prompt, and two to request 5's
    parent = np.array([-1, 0, 0, 3, 5, 5])
    assert not b.fork(i32(parent)).any() and not m.fork(parent, None).any()
    m.same_state()
    m.same_pools()
    window = np.array([0, 0, 0, 0, 0, 0])
    for n in range(5):
        n_new = g.integers(0, 6, R)
        emitted = g.integers(np.minimum(1, window), window + 1)
        step(b, m, g, n_new, emitted)
        window = n_new
        if n == 1:  # a search goes on with request 2 alone, behind the tokens that it keeps
            emitted = g.integers(0, window + 1)
            parent = np.array([2, 2, 2, -1, -1, 9])
            got, want = b.fork(i32(parent), i32(emitted)), m.fork(parent, emitted)
            assert np.array_equal(got.cpu().numpy(), want) and want.tolist() == [0, 0, 0, 0, 0, paged8.BAD_REQUEST]
            m.same_state()
            window = np.where(m.window == 0, 0, window)
        if n == 2:  # two requests end; the rest moves to the start of the pools
            over = np.array([False, True, False, True, False, False])
            b.end(torch.tensor(over, device=DEV))
            m.window = np.where(over, -m.held, m.window).astype(np.int32)
            emitted = g.integers(0, window + 1)
            step(b, m, g, np.zeros(R, int), emitted)
            window = np.zeros(R, int)
            b.compact()
            m.compact()
            m.same_state()
            m.same_pools()
            used = b.table[b.now][b.table[b.now] >= 0]
            assert int(used.max()) < b.n_pages - int(b.n_free[b.now])


def test_fp32_outputs():
    g = np.random.default_rng(2)
    inv = 1000.0 ** (-np.arange(64) / 64)
    b = pg.PagedBatch(3, 1, n_pages=20, page_size=16, max_len=96, max_window=20, n_q_heads=4, n_kv_heads=2, rope=svd.Rope(inv), bits=8,
                      out_dtype=svd.SVD_F32)
    m = Model(b, inv)
    step(b, m, g, np.array([20, 3, 17]), None, torch.float32)
    step(b, m, g, np.array([1, 4, 2]), np.array([11, 3, 17]), torch.float32)


def test_a_fork_that_lacks_pages_leaves_its_request_alone():
    g = np.random.default_rng(3)
    inv = np.zeros(64)
    b = pg.PagedBatch(3, 1, n_pages=7, page_size=16, max_len=96, max_window=60, n_q_heads=2, n_kv_heads=1, rope=svd.Rope(inv), bits=8)
    m = Model(b, inv)
    step(b, m, g, np.array([60, 5, 1]), None)
    parent = np.array([-1, 0, 0])
    assert b.fork(i32(parent)).tolist() == [0, paged8.NO_PAGES, paged8.NO_PAGES]
    m.fork(parent, None)
    m.same_state()
    m.same_pools()
    step(b, m, g, np.array([0, 2, 3]), np.array([17, 5, 1]))  # the rejected tokens' pages serve the next fork
    parent = np.array([-1, 0, -1])
    assert b.fork(i32(parent)).tolist() == [0, 0, 0]
    m.fork(parent, None)
    m.same_state()
    m.same_pools()


def test_a_recorded_step_with_a_fork_replays():
    """begin, both layers, fork and compact in one graph on a stream of its own, replayed; beside it another batch on
    another stream."""
    def batch():
        return pg.PagedBatch(4, 2, n_pages=60, page_size=16, max_len=200, max_window=8, n_q_heads=4, n_kv_heads=2, bits=8,
                             rope=svd.Rope(100.0 ** (-np.arange(64) / 64)))
    T = 16
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    rows = torch.randn((2, T, 8 * 128), generator=g, device=DEV)
    n_new, emitted, parent = i32([4] * 4), i32([3, 4, 2, 1]), i32([-1, 0, -1, 2])

    def one(b, out, stream):
        b.begin(n_new, emitted, stream=stream)
        for l in range(2):
            b.layer(l, rows[l], out[l], n_tokens=T, stream=stream)
        b.fork(parent, emitted, stream=stream)
        b.compact(stream=stream)

    runs = []
    for recorded in (False, True):
        b, other = batch(), batch()
        out, o2 = (torch.zeros((2, T, 4, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        one(b, out, s)
        one(other, o2, s2)
        torch.cuda.synchronize()
        if recorded:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                one(b, out, None)
            for _ in range(4):
                graph.replay()
                one(other, o2, s2)
        else:
            for _ in range(4):
                one(b, out, s)
                one(other, o2, s2)
        torch.cuda.synchronize()
        for x, o in ((b, out), (other, o2)):
            used = x.n_pages - int(x.n_free[x.now])
            runs.append((o.clone(), x.table[x.now].clone(), x.held[x.now].clone(), [p[:used * (p.numel() // x.n_pages)].clone() for p in x.pools]))
    for r in runs[1:]:
        assert torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1]) and torch.equal(r[2], runs[0][2])
        assert all(torch.equal(a, c) for a, c in zip(r[3], runs[0][3]))


@pytest.mark.parametrize("bits,samples", [(8, 1), (8, 4), (4, 2)])
def test_demo(bits, samples):
    b, kept = pg.demo(requests=8, window=4, steps=3, prompt=50, layers=1, bits=bits, samples=samples)
    assert len(kept) == 4 and not b.status.any() and not b.bad.any() and not b.fork_status.any()
    assert all(np.all(np.diff([k[r] for k in kept]) >= 1) for r in range(8))
    assert int(b.attention_status) == 0


def test_attention_right_behind_kernels_that_hold_tensor_memory():
    """A product on the tensor cores, and another attention, directly ahead on the stream, launched and replayed: an attention takes its
    tensor memory once they have ended, and all results are as they are apart."""
    from speculative_decoding_verify_06_gb300 import stack
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    lin = stack.Linear(1024, 2048, 32, 3, torch.device(DEV))
    ws = torch.zeros(svd.svd_verify_linear_workspace_bytes(1024, 2048, 32), dtype=torch.uint8, device=DEV)
    Hq, Hkv, page, n_pages, R = 20, 4, 64, 64, 2
    pool = torch.randint(0, 0x70, (svd.svd_paged8_cache_bytes(Hkv, page, n_pages),), dtype=torch.uint8, generator=g, device=DEV)
    pool.view(-1, svd.SVD_PAGED8_UNIT_BYTES)[:, 4096:4104] = torch.tensor([0, 0, 0, 0x3A] * 2, dtype=torch.uint8, device=DEV)  # 2^-11
    table = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).reshape(R, -1)
    runs = []
    for new in (4, 40, 13):  # row tiles that leave room for the product's kernel beside them, and that take a whole SM
        T = R * new
        q = torch.randn((T, Hq, 128), generator=g, device=DEV).to(torch.bfloat16)
        out = torch.zeros((T, Hq, 128), dtype=torch.bfloat16, device=DEV)
        aw = torch.zeros(svd.svd_paged8_attention_workspace_bytes(Hq, Hkv, R, new), dtype=torch.uint8, device=DEV)
        runs.append((q, T, i32([2048, 1999]), i32([0, new, T]), new, out, aw))

    def product():
        svd.svd_verify_linear(lin.W, lin.X, 32, lin.Y, ws, flags=svd.SVD_F_PDL)

    def attend(q, T, kv_len, q_start, new, out, aw):
        svd.svd_paged8_attention(q, T, kv_len, q_start, R, new, table, table.shape[1], pool, page, n_pages, Hq, Hkv, 128 ** -0.5, out,
                                 svd.SVD_BF16, aw)

    product()
    torch.cuda.synchronize()
    want = [lin.Y.clone()]
    for r in runs:
        attend(*r)
        torch.cuda.synchronize()
        want.append(r[5].clone())

    def all_of_them():
        for r in runs:
            product()
            attend(*r)
            attend(*r)

    def same():
        torch.cuda.synchronize()
        assert torch.equal(lin.Y, want[0]) and all(torch.equal(r[5], w) for r, w in zip(runs, want[1:]))
        assert not any(r[6][:4].any() for r in runs)

    for _ in range(10):
        all_of_them()
    same()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            all_of_them()
        for r in runs:
            r[5].zero_()
        for _ in range(10):
            graph.replay()
    same()
