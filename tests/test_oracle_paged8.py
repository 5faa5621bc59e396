"""The fp64 reference of the paged 8-bit cache and of moving pages, pinned by hand-worked values and invariants."""
import numpy as np
import pytest
import torch

from oracle import paged8


def test_values_of_the_codes():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged8.VALUE, t, equal_nan=True)
    assert paged8.VALUE[[0x01, 0x08, 0x38, 0x7E, 0xFE]].tolist() == [2.0 ** -9, 2.0 ** -6, 1.0, 448.0, -448.0]


def test_encode():
    x = np.array([0.0, -0.0, 1.0, 1.0625, 1.1875, 1.07, 2.0 ** -10, 3 * 2.0 ** -10, 447.0, 432.0, 431.9, -1e9, 2.0 ** -6 - 2.0 ** -10])
    assert paged8.encode(x).tolist() == [0, 0x80, 0x38, 0x38, 0x3A, 0x39, 0, 2, 0x7E, 0x7E, 0x7D, 0xFE, 0x08]
    g = np.random.default_rng(0)
    x = g.normal(0, 1, 20000) * 2.0 ** g.integers(-14, 9, 20000)
    x = np.clip(x, -448, 448).astype(np.float32)
    assert np.array_equal(paged8.encode(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert np.array_equal(paged8.encode(paged8.VALUE[:127]), np.arange(127))


@pytest.mark.parametrize("top,e", [(0.0, -64), (448.0, 0), (np.nextafter(448.0, 999), 1), (1.75, -8), (1.0, -8), (57344.0, 7), (1e9, 7)])
def test_exponent(top, e):
    assert paged8.exponent(top) == e


def test_every_byte_of_a_unit_has_its_place():
    at = np.concatenate([paged8.k_bytes(i) for i in range(16)] + [paged8.v_bytes(i) for i in range(16)])
    assert sorted(at) == list(range(4096))
    assert paged8.k_bytes(3)[[0, 16, 47, 127]].tolist() == [3 * 128 + 48, 3 * 128 + 32, 3 * 128 + 16 + 15, 3 * 128 + 64 + 15]


def test_append_and_get():
    pool = np.zeros((2, 1, 2, paged8.UNIT), np.uint8)
    table = np.array([[1, -1]])
    x = np.zeros((1, 1, 128))
    x[0, 0, :3] = 1.0, -0.3, 448.0
    assert paged8.append(pool, x, -x, [1], [0, 1], table, 32) == []
    k, v = paged8.get(pool, [32, 33, 64, -1], 32)
    assert k[0, 0, :3].tolist() == [1.0, -0.3125, 448.0] and v[0, 0, :3].tolist() == [-1.0, 0.3125, -448.0]
    assert not k[1:].any() and not v[1:].any()
    # a louder token: the scale grows by 8, and 0.3125 is held as 0.3125 / 8 = 20 steps of 2^-9
    x[0, 0, :3] = 3000.0, 0.0, 0.0
    assert paged8.append(pool, x, x, [2], [0, 1], table, 32) == []
    k, v = paged8.get(pool, [32, 33], 32)
    assert k[0, 0, :3].tolist() == [1.0, -0.3125, 448.0] and k[1, 0, 0] == 384.0 * 8
    x[0, 0, :3] = 50000.0, 0.0, 0.0
    paged8.append(pool, x, x, [3], [0, 1], table, 32)
    k, _ = paged8.get(pool, [32], 32)
    assert k[0, 0, :3].tolist() == [1.0, -0.25, 448.0]  # -0.3125 / 128 = -1.25 steps
    assert paged8.append(pool, x, x, [65], [0, 1], table, 32) == [0] and paged8.append(pool, x, x, [0], [0, 1], table, 32) == [0]


def test_attention_of_equal_scores_is_the_mean():
    pool = np.zeros((1, 1, 1, paged8.UNIT), np.uint8)
    v = np.arange(1, 6)[:, None, None] * np.ones((5, 1, 128))
    paged8.append(pool, np.zeros((5, 1, 128)), v, [5], [0, 5], np.array([[0]]), 16)
    o, a, e, big = paged8.attention(np.ones((2, 1, 128)), pool, 16, np.array([[0]]), [5], [0, 2], 1.0)
    assert np.allclose(o[:, 0, 0], [2.5, 3.0], atol=1e-15) and not e.any() and np.allclose(big[1, 0], 1.0)


def test_fork_by_hand():
    # pages of 16; request 0 holds 40 positions of which 3 of its window of 5 stay: 38, three pages
    table = np.array([[7, 2, 5, -1], [1, -1, -1, -1], [3, 4, 6, 8]])
    free = np.array([9, 0, -1, -1, -1, -1, -1, -1, -1, -1])
    o = paged8.fork([40, 10, 64], [5, 4, 0], [3, 9, 0], [-1, 0, -1], 16, table, free, 2)
    assert o["table"].tolist() == [[7, 2, 5, -1], [1, 0, 9, -1], [3, 4, 6, 8]] and o["n_free"] == 0
    assert o["moves"] == [(7, 1), (2, 0), (5, 9)] and o["held"].tolist() == [40, 38, 64] and o["window"].tolist() == [5, 0, 0]
    # a shorter parent: the surplus goes onto the stack
    o = paged8.fork([40, 10, 64], [5, 4, 0], [3, 1, 0], [-1, -1, 1], 16, table, free, 2)
    assert o["table"][2].tolist() == [3, -1, -1, -1] and o["free"][:5].tolist() == [9, 0, 4, 6, 8] and o["held"][2] == 7
    # no pages; a parent that is a child; one that does not exist; a count out of order
    o = paged8.fork([64, 0, 0], [0, 0, 0], [0, 0, 0], [-1, 0, 1], 16, table, free, 2)
    assert o["status"].tolist() == [0, paged8.NO_PAGES, paged8.BAD_REQUEST] and not o["moves"]
    assert paged8.fork([40, 10, 64], [5, 4, 0], [6, 1, 0], [-1, 0, 3], 16, table, free, 2)["status"].tolist() == [0, 32, 32]


def test_compact_by_hand():
    o = paged8.compact([20, 1, 0], 16, np.array([[7, 2, 9], [5, 5, 5], [1, 1, 1]]), 10)
    assert o["moves"] == [(5, 0), (7, 1)] and o["table"].tolist() == [[1, 2, -1], [0, -1, -1], [-1, -1, -1]]
    assert o["n_free"] == 7 and o["free"].tolist() == [9, 8, 7, 6, 5, 4, 3, -1, -1, -1]


def test_fork_and_compact_keep_every_page_in_one_place():
    g = np.random.default_rng(1)
    R, page, width, n = 12, 16, 9, 60
    held = np.zeros(R, int)
    table, free, n_free = np.full((R, width), -1), g.permutation(n), n
    for step in range(60):
        for r in range(R):  # grow, one by one
            want = min(int(held[r]) + int(g.integers(0, 12)), width * page)
            need = -(-want // page) - -(-int(held[r]) // page)
            if need <= n_free:
                for c in range(-(-int(held[r]) // page), -(-want // page)):
                    n_free -= 1
                    table[r, c] = free[n_free]
                held[r] = want
        parent = np.where(g.random(R) < 0.4, g.integers(0, R, R), -1)
        o = paged8.fork(held, None, None, parent, page, table, free, n_free)
        assert len({d for _, d in o["moves"]}) == len(o["moves"]) and not {d for _, d in o["moves"]} & {s for s, _ in o["moves"]}
        table, free, n_free, held = o["table"], o["free"], o["n_free"], o["held"].astype(int)
        if step % 3 == 2:
            o = paged8.compact(held, page, table, n)
            table, free, n_free = o["table"], o["free"], o["n_free"]
        ids = [int(x) for r in range(R) for x in table[r, :-(-held[r] // page)]] + [int(x) for x in free[:n_free]]
        assert sorted(ids) == list(range(n))
