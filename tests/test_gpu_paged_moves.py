"""Forking requests, compacting pools and copying pages on the GPU against the reference, entry by entry."""
import numpy as np
import pytest
import torch

from oracle import paged8
from speculative_decoding_verify_06_gb300 import svd
from tests.gpu_helpers import DEV, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def i32(a):
    return None if a is None else torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def state(g, R, page, width, spare):
    """Lengths, and a table and a stack of free pages that hold every page once."""
    held = g.integers(0, width * page + 1, R)
    have = -(-held // page)
    ids = g.permutation(int(have.sum()) + spare).astype(np.int32)
    table = np.full((R, width), -1, np.int32)
    table[np.arange(width) < have[:, None]] = ids[:have.sum()]
    free = np.full(len(ids), -1, np.int32)
    free[:spare] = ids[have.sum():]
    return held, table, free


def gpu_fork(held, window, emitted, parent, page, table, free, n_free, stream=None):
    R, width = table.shape
    n = len(free)
    mk = lambda *s: torch.full(s, -77, dtype=torch.int32, device=DEV)  # noqa: E731
    o = dict(held=mk(R), window=mk(R), table=mk(R, width), free=mk(n), n_free=mk(1), src=mk(n), dst=mk(n), n=mk(1), status=mk(R))
    ins = [i32(a) for a in (held, window, emitted, parent, table, free, [n_free])]
    svd.svd_paged_fork(*ins[:4], R, page, ins[4], width, ins[5], ins[6], n, o["held"], o["window"], o["table"], o["free"],
                       o["n_free"], o["src"], o["dst"], o["n"], o["status"], stream=stream)
    torch.cuda.synchronize()
    return o


def moves(o):
    src, dst = o["src"].cpu().numpy(), o["dst"].cpu().numpy()
    n = int(o["n"][0])
    assert (src[n:] == -1).all() and (dst[n:] == -1).all()
    return list(zip(src[:n].tolist(), dst[:n].tolist()))


def same(o, want):
    for k in ("held", "window", "table", "free", "status"):
        if k in want:
            assert np.array_equal(o[k].cpu().numpy(), want[k]), k
    assert int(o["n_free"][0]) == want["n_free"] and moves(o) == want["moves"]


@pytest.mark.parametrize("R,page,width,spare", [(1, 16, 1, 0), (2, 16, 5, 9), (7, 32, 40, 60), (64, 64, 17, 200), (513, 16, 6, 300),
                                                (1025, 256, 5, 4000), (4096, 16, 3, 900)])
def test_fork(R, page, width, spare):
    g = np.random.default_rng(R + page)
    held, table, free = state(g, R, page, width, spare)
    window = np.minimum(held, g.integers(0, 9, R))
    emitted = g.integers(0, window + 1)
    parent = np.where(g.random(R) < 0.6, g.integers(0, R, R), -1)
    parent[g.random(R) < 0.7] = -1
    for r in g.integers(0, R, R // 8):  # contradictions
        [lambda: parent.__setitem__(r, R), lambda: emitted.__setitem__(r, window[r] + 1), lambda: window.__setitem__(r, held[r] + 1),
         lambda: held.__setitem__(r, -1), lambda: window.__setitem__(r, -held[r]), lambda: parent.__setitem__(r, r)][g.integers(0, 6)]()
    args = (held, window, emitted, parent, page, table, free, spare)
    want = paged8.fork(*args)
    same(gpu_fork(*args), want)
    if R > 500:
        assert {0, paged8.BAD_REQUEST} <= set(want["status"].tolist())


@pytest.mark.parametrize("R", [6, 600, 4096])
def test_fork_with_too_few_pages(R):
    """Children of long parents: the first ones are served, then none; those that give pages back always are."""
    g = np.random.default_rng(R)
    held = np.where(np.arange(R) % 3 == 0, 60, np.where(np.arange(R) % 3 == 1, 20, 90))
    have = -(-held // 16)
    ids = g.permutation(int(have.sum()) + 7).astype(np.int32)
    table = np.full((R, 6), -1, np.int32)
    table[np.arange(6) < have[:, None]] = ids[:have.sum()]
    free = np.full(len(ids), -1, np.int32)
    free[:7] = ids[have.sum():]
    parent = np.arange(R) // 3 * 3                      # every third one's: itself, one page more or less
    want = paged8.fork(held, None, None, parent, 16, table, free, 7)
    same(gpu_fork(held, None, None, parent, 16, table, free, 7), want)
    parent[2::3] = -1
    want = paged8.fork(held, None, None, parent, 16, table, free, 7)
    same(gpu_fork(held, None, None, parent, 16, table, free, 7), want)
    assert (paged8.NO_PAGES in want["status"].tolist()) == (R > 10) and want["status"][1] == 0


def test_fork_without_windows_or_counts():
    g = np.random.default_rng(5)
    held, table, free = state(g, 20, 32, 12, 100)
    parent = np.array([-1, 0, 0, 0, 4] * 4)
    parent[5:] = np.where(parent[5:] == 0, 5, -1)
    window = np.minimum(held, 3)
    for win, emi in ((None, None), (window, None), (-window, window)):
        same(gpu_fork(held, win, emi, parent, 32, table, free, 100), paged8.fork(held, win, emi, parent, 32, table, free, 100))


@pytest.mark.parametrize("R,page,width,spare", [(1, 16, 1, 0), (1, 16, 3000, 500), (3, 32, 40, 5000), (64, 64, 17, 200), (700, 16, 9, 900),
                                                (4096, 16, 20, 60000)])
def test_compact(R, page, width, spare):
    g = np.random.default_rng(R + width)
    held, table, free = state(g, R, page, width, spare)
    n = len(free)
    if R > 3:  # a page held twice, ids outside the pool, lengths out of range
        held[1], held[2] = max(held[1], 1), max(held[2], 1)
        table[1, 0] = table[2, 0] if table[2, 0] >= 0 else table[3, 0]
        held[3], table[0, 0] = -5, n + 3
    want = paged8.compact(held, page, table, n)
    mk = lambda *s: torch.full(s, -77, dtype=torch.int32, device=DEV)  # noqa: E731
    o = dict(table=mk(R, width), free=mk(n), n_free=mk(1), src=mk(n), dst=mk(n), n=mk(1))
    svd.svd_paged_compact(i32(held), R, page, i32(table), width, n, o["table"], o["free"], o["n_free"], o["src"], o["dst"], o["n"])
    torch.cuda.synchronize()
    same(o, want)


def test_compact_of_the_largest_pool():
    n = svd.SVD_PAGED_COMPACT_MAX_PAGES
    g = np.random.default_rng(6)
    held = np.array([16 * 3000, 16 * 999 - 3])
    table = np.full((2, 3001), -1, np.int32)
    ids = g.permutation(n)[:3999]
    ids[:2] = n - 1, 0
    ids = np.array(list(dict.fromkeys(ids.tolist() + g.permutation(n)[:10].tolist())))[:3999]
    table[0, :3000], table[1, :999] = ids[:3000], ids[3000:]
    want = paged8.compact(held, 16, table, n)
    mk = lambda *s: torch.full(s, -77, dtype=torch.int32, device=DEV)  # noqa: E731
    o = dict(table=mk(2, 3001), free=mk(n), n_free=mk(1), src=mk(n), dst=mk(n), n=mk(1))
    svd.svd_paged_compact(i32(held), 2, 16, i32(table), 3001, n, o["table"], o["free"], o["n_free"], o["src"], o["dst"], o["n"])
    torch.cuda.synchronize()
    same(o, want)


@pytest.mark.parametrize("page_bytes", [16, 2304, 4112, 16384, 16400, 131584, 147472])
@pytest.mark.parametrize("layers", [1, 3, 130])
def test_copy(page_bytes, layers):
    g = np.random.default_rng(page_bytes + layers)
    n_pages = 40 if page_bytes < 20000 else 14
    if layers > 100:
        n_pages = 8
    pools = [torch.from_numpy(g.integers(0, 256, n_pages * page_bytes + 32, dtype=np.uint8)).to(DEV) for _ in range(layers)]
    want = [p.clone() for p in pools]
    ids = g.permutation(n_pages)
    m = n_pages // 2
    src, dst = ids[:m].copy(), ids[m:2 * m].copy()
    src[1] = src[0]  # one page copied twice
    list_src, list_dst = np.full(m + 6, -1), np.full(m + 6, -1)
    list_src[:m], list_dst[:m] = src, dst
    list_src[m:m + 3], list_dst[m:m + 3] = (-1, n_pages, ids[0]), (dst[0], dst[1], 2 ** 31 - 1)  # passed over
    for p in want:
        v = p[:n_pages * page_bytes].view(n_pages, page_bytes)
        v[torch.tensor(dst, device=DEV)] = v[torch.tensor(src, device=DEV)]
    n = i32([m + 3])
    handle = svd.Pools(pools, page_bytes)
    svd.svd_paged_copy(handle, n_pages, i32(list_src), i32(list_dst), n, m + 6)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    # no more than max_copies, and a count below 0 is none
    svd.svd_paged_copy(handle, n_pages, i32(list_dst), i32(list_src), i32([m]), 0)
    svd.svd_paged_copy(handle, n_pages, i32(list_dst), i32(list_src), i32([-4]), m)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


def test_copy_past_32_bits():
    per = 64 * 4112 * 8
    n = 5 * 2 ** 30 // per
    pool = torch.empty(n * per, dtype=torch.uint8, device=DEV)
    pool[:per] = torch.randint(0, 256, (per,), dtype=torch.uint8, device=DEV)
    pool[(n - 1) * per:] = 0
    svd.svd_paged_copy(svd.Pools([pool], per), n, i32([0]), i32([n - 1]), i32([1]), 1)
    assert torch.equal(pool[:per], pool[(n - 1) * per:])
