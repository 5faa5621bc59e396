"""Refusals of the 8-bit cache's and the page-moving entry points, without a GPU."""
import inspect

import pytest
import torch

from speculative_decoding_verify_06_gb300 import build, paged, svd


@pytest.fixture(scope="module")
def lib():
    build.build_library()
    return svd.load()


APPEND = dict(qkv=16, dtype=0, ld=768, T=2, Hq=2, Hkv=2, rope=None, positions=None, positions_ld=0, kv_len=32, q_start=48, R=1, table=64,
              width=4, pages=80, page=16, n_pages=8, q=96, status=None, stream=None)
ATTENTION = dict(q=16, T=2, kv_len=32, q_start=48, R=1, max_new=2, table=64, width=4, pages=80, page=16, n_pages=8, Hq=4, Hkv=2,
                 scale=1.0, out=96, out_dtype=0, ws=112, ws_bytes=1 << 30, stream=None)
FORK = dict(held=16, window=32, emitted=48, parent=64, R=2, page=16, table=80, width=4, free=96, n_free=112, n_pages=8, held_out=128,
            window_out=144, table_out=160, free_out=176, n_free_out=192, src=208, dst=224, n=240, status=256, stream=None)
COMPACT = dict(held=16, R=2, page=16, table=80, width=4, n_pages=8, table_out=160, free_out=176, n_free_out=192, src=208, dst=224, n=240,
               stream=None)


@pytest.mark.parametrize("change", [
    dict(qkv=None), dict(qkv=24), dict(dtype=2), dict(ld=767), dict(ld=770), dict(T=-1), dict(Hq=-1), dict(Hkv=0), dict(Hq=4097),
    dict(kv_len=None), dict(q_start=None), dict(R=0), dict(R=4097), dict(table=None), dict(width=0), dict(width=1 << 28), dict(pages=None),
    dict(pages=88), dict(page=24), dict(page=272), dict(n_pages=0), dict(n_pages=(1 << 30) + 1), dict(q=None), dict(q=100)])
def test_append_refusals(lib, change):
    assert lib.svd_paged8_append(*{**APPEND, **change}.values()) == svd.SVD_ERR_INVALID_ARG


@pytest.mark.parametrize("rope", [svd.Rope([0.1] * 3), svd.Rope([1e10] * 4), svd.Rope([0.1] * 4, [0, 1, 0, 0], 1), svd.Rope([0.1] * 4, n_axes=5),
                                  svd.Rope([float("nan")] * 4)])
def test_append_refuses_such_rotary_positions(lib, rope):
    assert lib.svd_paged8_append(*{**APPEND, "rope": rope._p, "positions": 16}.values()) == svd.SVD_ERR_INVALID_ARG
    good = svd.Rope([0.1] * 4)
    assert lib.svd_paged8_append(*{**APPEND, "rope": good._p}.values()) == svd.SVD_ERR_INVALID_ARG  # no positions


def test_nothing_to_do(lib):
    assert lib.svd_paged8_append(*{**APPEND, "T": 0}.values()) == svd.SVD_OK
    assert lib.svd_paged8_read(16, 0, 2, 16, 16, 8, 32, 48, None) == svd.SVD_OK
    a = (svd.ctypes.c_void_p * 1)(16)
    assert lib.svd_paged_copy(a, 1, 4112, 8, 32, 48, 64, 0, None) == svd.SVD_OK


@pytest.mark.parametrize("args", [(None, 2, 2, 16, 16, 8, 32, 48), (16, -1, 2, 16, 16, 8, 32, 48), (16, 2, 0, 16, 16, 8, 32, 48),
                                  (16, 2, 2, 20, 16, 8, 32, 48), (16, 2, 2, 16, 17, 8, 32, 48), (16, 2, 2, 16, 16, 0, 32, 48),
                                  (16, 2, 2, 16, 16, 8, 36, 48), (16, 2, 2, 16, 16, 8, 32, None)])
def test_read_refusals(lib, args):
    assert lib.svd_paged8_read(*args, None) == svd.SVD_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(q=None), dict(q=24), dict(T=-1), dict(kv_len=None), dict(q_start=None), dict(R=0), dict(R=4097), dict(max_new=0), dict(table=None),
    dict(width=0), dict(pages=None), dict(pages=72), dict(page=8), dict(n_pages=0), dict(Hq=3), dict(Hq=0), dict(Hkv=0), dict(scale=0.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(out=None), dict(out=100), dict(out_dtype=2), dict(ws=116)])
def test_attention_refusals(lib, change):
    assert lib.svd_paged8_attention(*{**ATTENTION, **change}.values()) == svd.SVD_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(held=None), dict(parent=None), dict(R=0), dict(R=4097), dict(page=24), dict(table=None), dict(width=0), dict(free=None), dict(n_free=None),
    dict(n_pages=0), dict(held_out=None), dict(window_out=None), dict(table_out=None), dict(free_out=None), dict(n_free_out=None), dict(src=None),
    dict(dst=None), dict(n=None), dict(status=None), dict(held_out=16), dict(window_out=32), dict(table_out=80), dict(free_out=96),
    dict(n_free_out=112), dict(dst=208)])
def test_fork_refusals(lib, change):
    assert lib.svd_paged_fork(*{**FORK, **change}.values()) == svd.SVD_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(held=None), dict(R=0), dict(R=4097), dict(page=24), dict(table=None), dict(width=0), dict(n_pages=0), dict(table_out=None),
    dict(table_out=80), dict(free_out=None), dict(n_free_out=None), dict(src=None), dict(dst=None), dict(dst=208), dict(n=None)])
def test_compact_refusals(lib, change):
    assert lib.svd_paged_compact(*{**COMPACT, **change}.values()) == svd.SVD_ERR_INVALID_ARG


def test_compact_of_a_pool_too_large_for_a_bit_map(lib):
    assert lib.svd_paged_compact(*{**COMPACT, "n_pages": svd.SVD_PAGED_COMPACT_MAX_PAGES + 1}.values()) == svd.SVD_ERR_UNSUPPORTED


@pytest.mark.parametrize("pools,change", [([16], dict(n_pools=0)), ([16], dict(page_bytes=0)), ([16], dict(page_bytes=4104)), ([16], dict(n_pages=0)),
                                          ([16], dict(src=None)), ([16], dict(dst=None)), ([16], dict(n=None)), ([16], dict(most=-1)),
                                          ([16, 24], dict(n_pools=2)), ([16, None], dict(n_pools=2))])
def test_copy_refusals(lib, pools, change):
    a = (svd.ctypes.c_void_p * len(pools))(*pools)
    args = dict(pools=a, n_pools=1, page_bytes=4112, n_pages=8, src=32, dst=48, n=64, most=4, stream=None)
    assert lib.svd_paged_copy(*{**args, **change}.values()) == svd.SVD_ERR_INVALID_ARG
    assert lib.svd_paged_copy(*{**args, "pools": None}.values()) == svd.SVD_ERR_INVALID_ARG


def test_sizes(lib):
    assert svd.svd_paged8_cache_bytes(8, 64, 3) == 3 * 8 * 4 * 4112
    assert svd.svd_paged8_cache_bytes(8, 24, 3) == 0 and svd.svd_paged8_cache_bytes(0, 16, 3) == 0


def test_pools_keep_what_they_are_given():
    p = svd.Pools([16, 32, 48], 4112)
    assert len(p) == 3 and list(p._a) == [16, 32, 48] and p.page_bytes == 4112


# ---- PagedBatch: what its calls are given -----------------------------------------------------------
@pytest.fixture
def calls(lib, monkeypatch):
    """Every call of the entry points, recorded instead of made."""
    made = []

    def record(name):
        f = inspect.signature(getattr(svd, name))

        def call(*a, **k):
            b = f.bind(*a, **k)
            b.apply_defaults()
            made.append((name, b.arguments))
        monkeypatch.setattr(svd, name, call)
    for name in ("svd_paged_append", "svd_paged_attention", "svd_paged8_append", "svd_paged8_attention", "svd_paged_fork", "svd_paged_copy",
                 "svd_paged_compact"):
        record(name)
    return made


def batch(**kw):
    a = dict(requests=3, layers=2, n_pages=12, page_size=16, max_len=64, max_window=4, n_q_heads=4, n_kv_heads=2, device="cpu", bits=8)
    return paged.PagedBatch(**{**a, **kw})


@pytest.mark.parametrize("bits", [0, 5, 16, "8", None])
def test_other_bits_are_refused(lib, bits):
    with pytest.raises(ValueError, match="bits"):
        batch(bits=bits)


@pytest.mark.parametrize("bits,names", [(4, ["svd_paged_append", "svd_paged_attention"]), (8, ["svd_paged8_append", "svd_paged8_attention"])])
def test_a_layer_goes_to_the_cache_of_its_bits(calls, bits, names):
    b = batch(bits=bits)
    assert b.pools[0].numel() == 12 * 2 * (4112 if bits == 8 else 2304)
    b.layer(1, torch.zeros((9, 8 * 128)), torch.zeros((9, 4, 128), dtype=torch.bfloat16), n_tokens=7)
    assert [n for n, _ in calls] == names
    for _, a in calls:
        assert a["n_tokens"] == 7 and a["pages"] is b.pools[1] and a["page_size"] == 16 and a["n_pages"] == 12
    if bits == 8:
        a = calls[0][1]
        assert a["kv_len"] is b.kv_len and a["q_start"] is b.q_start and a["table"] is b.table[b.now] and a["max_pages"] == b.width


@pytest.mark.parametrize("bits", [4, 8])
def test_fork_and_compact_copy_whole_pages_of_all_layers(calls, bits):
    b = batch(bits=bits)
    assert b.fork(torch.zeros(3, dtype=torch.int32), torch.ones(3, dtype=torch.int32)) is b.fork_status
    b.compact()
    assert [n for n, _ in calls] == ["svd_paged_fork", "svd_paged_copy", "svd_paged_compact", "svd_paged_copy"]
    for name, a in calls:
        if name == "svd_paged_copy":
            assert a["pools"].page_bytes == b.pools[0].numel() // 12 and a["pools"].pools == b.pools
            assert a["copy_from"] is b._copy_from and a["copy_to"] is b._copy_to and a["n_copies"] is b._n_copies


def test_copies_go_to_the_pools_that_the_layers_use(calls):
    """A pool that takes another's place in the list is the one that a fork and a compaction copy."""
    b = batch()
    b.pools[1] = torch.zeros_like(b.pools[1])
    b.fork(torch.zeros(3, dtype=torch.int32))
    b.compact()
    copies = [a["pools"] for n, a in calls if n == "svd_paged_copy"]
    assert len(copies) == 2 and all(c.pools[i] is b.pools[i] and c._a[i] == b.pools[i].data_ptr() for c in copies for i in (0, 1))


@pytest.mark.parametrize("pool", [torch.zeros(12 * 2 * 4112 - 1, dtype=torch.uint8), torch.zeros(12 * 2 * 4112),
                                  torch.zeros(2 * 12 * 2 * 4112, dtype=torch.uint8)[::2],
                                  torch.zeros(12 * 2 * 4112, dtype=torch.uint8, device="meta")])
def test_pools_of_another_form_are_not_copied(calls, pool):
    b = batch()
    b.pools[0] = pool
    with pytest.raises(ValueError, match="pools"):
        b.compact()
    assert "svd_paged_copy" not in [n for n, _ in calls]


@pytest.mark.parametrize("parent", [torch.ones(3, dtype=torch.int64), torch.ones(2, dtype=torch.int32), torch.ones(3),
                                    torch.ones(6, dtype=torch.int32)[::2], torch.ones((3, 1), dtype=torch.int32),
                                    torch.ones(3, dtype=torch.int32, device="meta")])
def test_parents_and_counts_of_another_form_are_refused(calls, parent):
    good = torch.zeros(3, dtype=torch.int32)
    for a in ((parent, None), (good, parent)):
        with pytest.raises(ValueError, match="parent|emitted"):
            batch().fork(*a)
    assert not calls


def test_compact_keeps_the_lengths(calls):
    """The other copy's lengths are older than the state's: only the table and the stack come from there."""
    b = batch()
    b._state[0][-6:], b._state[1][-6:] = 5, 9
    b._state[1][:-6] = 3
    b.compact()
    assert (b._state[0][-6:] == 5).all() and (b._state[0][:-6] == 3).all()
