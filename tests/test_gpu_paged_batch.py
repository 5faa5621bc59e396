"""Batched verify steps through PagedBatch: ragged windows, rejected drafts and new prompts over several
steps and layers, against a plain cache kept on the host; and the step recorded into a graph."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from speculative_decoding_verify_06_gb300 import paged, svd
from tests.gpu_helpers import DEV, lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def held_values(x):
    c, d = ref.quantise(x)
    return ((c.reshape(*x.shape[:-1], 4, 32).astype(float) - 8) * d[..., None]).reshape(x.shape)


def test_steps_match_a_plain_cache():
    R, layers, Hq, Hkv, page = 5, 2, 6, 2, 16
    g = np.random.default_rng(1)
    inv = 1000.0 ** (-np.arange(64) / 64)
    b = paged.PagedBatch(R, layers, n_pages=60, page_size=page, max_len=160, max_window=40, n_q_heads=Hq, n_kv_heads=Hkv,
                         rope=svd.Rope(inv), max_tokens=R * 40)
    cache = [[[np.zeros((0, Hkv, 128)), np.zeros((0, Hkv, 128))] for _ in range(R)] for _ in range(layers)]
    window = np.zeros(R, int)
    for step in range(7):
        emitted = g.integers(np.minimum(1, window), window + 1) if step else None
        n_new = g.integers(1, 38, R) if step == 0 else g.integers(0, 6, R)
        b.begin(i32(n_new), None if emitted is None else i32(emitted))
        if step:
            for l in range(layers):
                for r in range(R):
                    keep = len(cache[l][r][0]) - window[r] + emitted[r]
                    cache[l][r] = [a[:keep] for a in cache[l][r]]
        window = n_new
        T = int(n_new.sum())
        assert b.q_start.tolist() == np.concatenate([[0], np.cumsum(n_new)]).tolist() and not b.status.any()
        for l in range(layers):
            x = g.normal(0, 1, (T, Hq + 2 * Hkv, 128)).astype(np.float32)
            out = torch.full((max(T, 1), Hq, 128), -7.0, dtype=torch.bfloat16, device=DEV)
            b.layer(l, torch.from_numpy(x.reshape(T, -1)).to(DEV), out, n_tokens=T)
            q = b.q[:T].double().cpu().numpy()
            got, t = out.double().cpu().numpy(), 0
            for r in range(R):
                k, v = cache[l][r]
                base = len(k)
                pos = np.arange(base, base + n_new[r])
                xr = x[t:t + n_new[r]].astype(np.float64)
                y = ref.rotate(xr, pos[None], inv, [0] * 64, False)
                assert np.all(np.abs(q[t:t + n_new[r]] - y[:, :Hq]) <= 2.0 ** -8 * np.abs(y[:, :Hq]) + 2.0 ** -17)
                k = np.concatenate([k, held_values(y[:, Hq:Hq + Hkv])])
                v = np.concatenate([v, held_values(xr[:, Hq + Hkv:])])
                cache[l][r] = [k, v]
                for i in range(n_new[r]):
                    for h in range(Hq):
                        n = base + i + 1
                        s = k[:n, h // 3] @ q[t + i, h] * b.scale
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        want, a = p @ v[:n, h // 3], p @ np.abs(v[:n, h // 3])
                        # bf16 output 2^-8, p in fp16 2^-11, scores 2^-16 of sum |q k| (below 64 here), twice
                        assert np.all(np.abs(got[t + i, h] - want) <= 2.0 ** -8 * np.abs(want) + a * (2.0 ** -11 + 2.0 ** -9))
                t += n_new[r]
        assert b.kv_len.tolist() == [len(cache[0][r][0]) for r in range(R)]
    assert not b.bad.any()


def test_a_pool_that_is_full_refuses_and_recovers():
    b = paged.PagedBatch(2, 1, n_pages=3, page_size=16, max_len=64, max_window=40, n_q_heads=2, n_kv_heads=1)
    b.begin(i32([30, 30]))
    assert b.status.tolist() == [0, svd.SVD_ST_NO_PAGES] and b.kv_len.tolist() == [30, 0] and b.window.tolist() == [30, 0]
    b.begin(i32([0, 30]), i32([3, 0]))  # the first request keeps three tokens and gives a page back
    assert b.status.tolist() == [0, 0] and b.kv_len.tolist() == [3, 30] and int(b.n_free[b.now]) == 0
    b.begin(i32([0, 0]), i32([0, 0]))
    assert b.kv_len.tolist() == [3, 0] and int(b.n_free[b.now]) == 2


def test_two_steps_recorded_in_a_graph():
    """Both copies of the tables in turn: a graph of two steps can be replayed."""
    R, n = 3, 2

    def make():
        b = paged.PagedBatch(R, 1, n_pages=40, page_size=16, max_len=256, max_window=n, n_q_heads=4, n_kv_heads=2,
                             rope=svd.Rope(np.full(64, 0.3)))
        g = torch.Generator(device=DEV)
        g.manual_seed(3)
        x = torch.randn((2, R * n, 8 * 128), generator=g, device=DEV)
        return b, x, [torch.zeros((R * n, 4, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)], i32([1, 2, 1])

    new = i32([n] * R)
    b, x, outs, emitted = make()
    b.begin(new)
    for step in range(6):
        b.begin(new, emitted)
        b.layer(0, x[step % 2], outs[step % 2])
    torch.cuda.synchronize()
    b2, x2, outs2, emitted2 = make()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b2.begin(new)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for step in range(2):
                b2.begin(new, emitted2)
                b2.layer(0, x2[step % 2], outs2[step % 2])
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    assert b2.held[b2.now].tolist() == b.kv_len.tolist()
    for a, c in zip(outs, outs2):
        assert torch.equal(a, c)


def test_demo_runs():
    b, lengths = paged.demo(requests=8, window=4, steps=3, prompt=40)
    a = np.array(lengths)
    assert np.all(a[0] == 40) and np.all((np.diff(a, axis=0) >= 1) & (np.diff(a, axis=0) <= 4))
    assert not b.status.any() and not b.bad.any()
