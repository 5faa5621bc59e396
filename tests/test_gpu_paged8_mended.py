"""The paged 8-bit calls and the moves of pages on the GPU in cases that once went wrong or that nothing ordered, against the
fp64 reference: appends whose CTAs handle many runs one after the other; requests whose tokens do not begin at row 0;
numbers of requests whose sums just fill the shared memory that a launch gets unasked; queries near the largest that bf16 holds, and scales of scores far from 1."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged, paged8
from speculative_decoding_verify_06_gb300 import svd
from tests.gpu_helpers import DEV, lib, to_dev
from tests.test_gpu_paged import gpu_tables, same_tables
from tests.test_gpu_paged8 import BOTH, Case, as_type, check_q, gpu_append, layout, random_pool, same_zeros
from tests.test_gpu_paged_moves import gpu_fork, same, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib()


@pytest.mark.parametrize("dtype", [svd.SVD_F32, svd.SVD_BF16])
@pytest.mark.parametrize("most,Hkv,rotate", [(1, 4, False), (4, 3, True), (9, 2, True)])
def test_appends_of_many_runs_to_a_cta(dtype, most, Hkv, rotate):
    """Some 5000 tokens in windows of 1 to `most`, begun at every place of a unit: up to sixteen runs follow one another in a CTA, and
    each fills shared memory that all warps of a head read at the end of the run before.  Every byte, thirty times over."""
    g = np.random.default_rng(most + Hkv)
    R = min(4096, 10000 // (most + 1))
    new = g.integers(1, most + 1, R)
    lens = (new + g.integers(0, 40, R)).tolist()
    table, q_start, n_pages = layout(lens, new.tolist(), 32, g)
    pool = random_pool(g, n_pages, Hkv, 32, e_lo=-9, e_hi=-5)
    T = int(q_start[-1])
    x = g.normal(0, 1, (T, 2 * Hkv, 128)).astype(np.float32) * 2.0 ** g.integers(-3, 4, (T, 1, 1))
    x = as_type(x, dtype).float().numpy()
    pos = np.concatenate([np.arange(n - k, n) for n, k in zip(lens, new)])[None]
    inv = 1e4 ** (-np.arange(64) / 64)
    y = paged.rotate(x.astype(np.float64), pos, inv, [0] * 64, False) if rotate else x.astype(np.float64)
    want = pool.copy()
    assert not paged8.append(want, y[:, :Hkv], x[:, Hkv:], lens, q_start, table, 32)
    rows, start = as_type(x.reshape(T, -1), dtype).to(DEV), to_dev(pool.reshape(-1))
    lens_d, q_d, tab, pos_d = to_dev(np.array(lens, np.int32)), to_dev(q_start), to_dev(table), to_dev(pos.astype(np.int32))
    status = torch.zeros(T, dtype=torch.int32, device=DEV)
    first = None
    for _ in range(30):
        p = start.clone()
        svd.svd_paged8_append(rows, 2 * Hkv * 128, T, 0, Hkv, lens_d, q_d, R, tab, tab.shape[1], p, 32, n_pages, None,
                              rope=svd.Rope(inv) if rotate else None, positions=pos_d, positions_ld=T, dtype=dtype, status=status)
        if first is None:
            first = p
            assert np.array_equal(same_zeros(p.cpu().numpy().reshape(pool.shape)), same_zeros(want))
        assert torch.equal(p, first)
    assert not status.any()


@pytest.mark.parametrize("dtype", [svd.SVD_F32, svd.SVD_BF16])
@pytest.mark.parametrize("first", [1, 5, 15, 16, 37, 2000])
def test_append_for_the_second_of_two_groups(dtype, first):
    """q_start[0] = first: the rows before are another group's.  Whatever block of tokens the first request begins in, all of it is stored."""
    g = np.random.default_rng(first)
    new = [0, 3, 0, 40, 1, 16, 500]
    lens = [9, 3, 0, 77, 17, 16, 501]
    table, q_start, n_pages = layout(lens, new, 32, g)
    pool = random_pool(g, n_pages, 3, 32)
    q_start = (q_start + first).astype(np.int32)
    T = int(q_start[-1])
    x = as_type(g.normal(0, 1, (T, 8, 128)).astype(np.float32), dtype).float().numpy()
    pos = g.integers(0, 3000, (1, T))
    inv = 1e4 ** (-np.arange(64) / 64)
    q, got, st = gpu_append(x, dtype, 2, 3, lens, q_start, table, pool, 32, rope=svd.Rope(inv), positions=pos)
    y = paged.rotate(x.astype(np.float64), pos, inv, [0] * 64, False)
    want = pool.copy()
    assert not paged8.append(want, y[first:, 2:5], x[first:, 5:], lens, q_start - first, table, 32)
    assert np.array_equal(same_zeros(got), same_zeros(want)) and not st.any()
    check_q(q[first:], y[first:, :2])


@BOTH
@pytest.mark.parametrize("first", [3, 130])
def test_attention_for_the_second_of_two_groups(out_dtype, first):
    c = Case([70, 200, 15], [4, 1, 9], 6, 2, 32, seed=first)
    o, a, e, _ = c.reference()
    rows = np.full((first, 6, 128), np.nan)
    c.q = torch.cat([torch.ones(first, 6, 128, dtype=torch.bfloat16), c.q])
    c.q_start = (c.q_start + first).astype(np.int32)
    c.T += first
    c.check(out_dtype, c.run(out_dtype), (np.concatenate([rows, o]), np.concatenate([rows, a]), np.concatenate([rows[..., 0], e])))


def fork_once(R):
    g = np.random.default_rng(R)
    held, table, free = state(g, R, 16, 3, 500)
    window = np.minimum(held, g.integers(0, 9, R))
    parent = np.where(g.random(R) < 0.3, g.integers(0, R, R), -1)
    args = (held, window, g.integers(0, window + 1), parent, 16, table, free, 500)
    same(gpu_fork(*args), paged8.fork(*args))


@pytest.mark.parametrize("R", [1638, 1639, 1960, 1961, 1963, 1965, 1966])
def test_a_first_fork_of_any_number_of_requests(R):
    """In a process of its own: a call that asked for more shared memory before would let this one have it."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", f"import tests.test_gpu_paged8_mended as t; t.lib(); t.fork_once({R})"], cwd=root, check=True, timeout=300)


def tables_once(R):
    g = np.random.default_rng(R)
    held, table, free = state(g, R, 16, 3, 500)
    window = np.minimum(held, g.integers(0, 9, R))
    emitted, new = g.integers(0, window + 1), g.integers(0, 5, R)
    args = (held, window, emitted, new, 16, table, free, 500, 3 * R)
    same_tables(gpu_tables(*args), paged.tables(*args))


@pytest.mark.parametrize("R", [1638, 1639, 1960, 1961, 1963, 1965, 1966])
def test_first_tables_of_any_number_of_requests(R):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", f"import tests.test_gpu_paged8_mended as t; t.lib(); t.tables_once({R})"], cwd=root, check=True, timeout=300)


@pytest.mark.parametrize("new,out_dtype", [(1, svd.SVD_BF16), (1, svd.SVD_F32), (4, svd.SVD_BF16), (4, svd.SVD_F32), (12, svd.SVD_BF16),
                                           (60, svd.SVD_BF16)])
@pytest.mark.parametrize("q_exp,k_exp,scale_exp", [(120, -64, -64), (125, -64, -64), (126, -64, 0), (116, -30, -90), (100, 7, -110), (116, 7, -122),
                                                   (-40, -20, 63), (-44, -20, 64), (-100, -3, 100), (-60, -64, 124)])
def test_queries_and_scales_of_any_size(new, out_dtype, q_exp, k_exp, scale_exp):
    """Rows as large as bf16 holds against keys as small as the cache holds, and the other way round: scores that are no larger than
    usual, or finite at least, give what the formula says."""
    c = Case([300, 150], [new, min(new, 3)], 5, 1, 64, seed=new, k_exp=(k_exp, k_exp + 1))
    c.q = (c.q.double().clamp(-2.5, 2.5) * 2.0 ** q_exp).to(torch.bfloat16)
    c.q[0, 0] = torch.finfo(torch.bfloat16).max if q_exp > 110 else c.q[0, 0]
    assert torch.isfinite(c.q).all()
    c.scale = 128 ** -0.5 * 2.0 ** scale_exp
    c.check(out_dtype, c.run(out_dtype), c.reference())
