"""What the binding and PagedBatch hand to the library, without a GPU."""
import enum
import inspect

import numpy as np
import pytest
import torch

from speculative_decoding_verify_06_gb300 import build, paged, svd


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return svd.load()


class Address(enum.IntEnum):
    A = 16


@pytest.mark.parametrize("size", [int, np.int32, np.int64, torch.tensor])
def test_wrappers_take_sizes_and_addresses_of_any_integer_type(size):
    """Sizes and addresses of any integer type reach the library, whose own
    refusal (a page of 17 positions) is what comes back."""
    a, n = Address.A, size(2)
    calls = [lambda: svd.svd_paged_read(a, n, n, a, size(17), n, a, a, stream=0),
             lambda: svd.svd_paged_append(a, size(768), n, n, n, a, a, size(17), n, a, dtype=size(0), stream=0),
             lambda: svd.svd_paged_tables(a, None, None, a, n, size(17), a, n, a, a, n, a, a, a, a, a, a, a, n, a, stream=0),
             lambda: svd.svd_paged_attention(a, n, a, a, n, n, a, n, a, size(17), n, n, n, size(1), a, size(0), a, n, stream=0),
             lambda: svd.svd_kv_unpack(a, size(-1), n, size(0), n, a, a, a, a, n, stream=0)]
    for call in calls:
        with pytest.raises(svd.SvdError, match="INVALID_ARG"):
            call()


# ---- PagedBatch: what its calls are given -----------------------------------------------------------
@pytest.fixture
def calls(monkeypatch):
    """Every call of the paged entry points, recorded instead of made."""
    made = []

    def record(name):
        f = inspect.signature(getattr(svd, name))

        def call(*a, **k):
            b = f.bind(*a, **k)
            b.apply_defaults()
            made.append((name, b.arguments))
        monkeypatch.setattr(svd, name, call)
    for name in ("svd_paged_tables", "svd_paged_advance", "svd_paged_append", "svd_paged_attention"):
        record(name)
    return made


def batch(**kw):
    a = dict(requests=3, layers=1, n_pages=12, page_size=16, max_len=64, max_window=4, n_q_heads=4, n_kv_heads=2, device="cpu")
    return paged.PagedBatch(**{**a, **kw})


def rows(T, heads=8, dtype=torch.float32):
    return torch.zeros((T, heads * 128), dtype=dtype), torch.zeros((T, 4, 128), dtype=torch.bfloat16)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("given", [None, "row", "axes", "wide", "expanded"])
def test_every_axis_has_its_positions(calls, axes, given):
    b = batch(rope=svd.Rope([0.1] * 8, [i % axes for i in range(8)], axes))
    T = 9
    pos = {None: None, "row": torch.zeros(T, dtype=torch.int32), "axes": torch.zeros((axes, T), dtype=torch.int32),
           "wide": torch.zeros((axes + 1, T + 5), dtype=torch.int32), "expanded": torch.zeros(T, dtype=torch.int32).expand(axes, T)}[given]
    qkv, out = rows(T)
    b.layer(0, qkv, out, n_tokens=T, positions=pos)
    a = dict(calls)["svd_paged_append"]
    held, ld = a["positions"], a["positions_ld"]
    end = held.untyped_storage().nbytes() // 4
    # the last position that the call reads lies in the tensor, and axes do not lie inside each other
    assert held.storage_offset() + (axes - 1) * ld + a["n_tokens"] <= end and (ld == 0 or ld >= T)
    if given in ("axes", "wide") and axes > 1:
        assert ld == pos.stride(0)


@pytest.mark.parametrize("pos", [torch.zeros(9), torch.zeros((2, 9), dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                                 torch.zeros((3, 9), dtype=torch.int64), torch.zeros((3, 18), dtype=torch.int32)[:, ::2],
                                 torch.zeros((1, 3, 9), dtype=torch.int32)])
def test_positions_of_another_form_are_refused(calls, pos):
    b = batch(rope=svd.Rope([0.1] * 9, [0, 1, 2] * 3, 3))
    qkv, out = rows(9)
    with pytest.raises(ValueError, match="positions"):
        b.layer(0, qkv, out, n_tokens=9, positions=pos)
    assert not calls


@pytest.mark.parametrize("given,tokens", [(5, None), (12, None), (20, None), (9, 7), (0, None), (4, 0)])
def test_as_many_tokens_as_there_are_rows(calls, given, tokens):
    b = batch()  # 12 tokens at most
    qkv, out = rows(given)
    b.layer(0, qkv, out, n_tokens=tokens)
    for name, a in calls:
        assert a["n_tokens"] == (min(given, 12) if tokens is None else tokens), name


@pytest.mark.parametrize("change", [
    dict(n_tokens=13), dict(n_tokens=-1), dict(n_tokens=8, rows=7), dict(n_tokens=8, out=7), dict(out=11), dict(heads=7),
    dict(strided=True), dict(loose=True), dict(flat=True)])
def test_rows_that_do_not_suffice_are_refused(calls, change):
    b = batch()
    qkv, _ = rows(change.get("rows", 20), change.get("heads", 8))
    out = torch.zeros((change.get("out", 20), 4, 128), dtype=torch.bfloat16)
    if "strided" in change:
        qkv = torch.zeros((1024, 20)).t()
    if "loose" in change:
        out = torch.zeros((20, 8, 128), dtype=torch.bfloat16)[:, :4]
    if "flat" in change:
        qkv = qkv.reshape(-1)
    with pytest.raises(ValueError, match="tokens|qkv|out"):
        b.layer(0, qkv, out, n_tokens=change.get("n_tokens"))
    assert not calls


@pytest.mark.parametrize("kind", [torch.float16, torch.float64, torch.int32])
def test_activations_of_another_type_are_refused(calls, kind):
    qkv, out = rows(4, dtype=kind)
    with pytest.raises(ValueError, match="qkv"):
        batch().layer(0, qkv, out)
    assert not calls


@pytest.mark.parametrize("made,given", [(svd.SVD_F32, torch.bfloat16), (svd.SVD_BF16, torch.float32), (svd.SVD_BF16, torch.float16)])
def test_outputs_have_the_type_the_batch_was_made_for(calls, made, given):
    qkv, out = rows(4)
    with pytest.raises(ValueError, match="out"):
        batch(out_dtype=made).layer(0, qkv, out.to(given))
    assert not calls


@pytest.mark.parametrize("n_new", [torch.ones(3, dtype=torch.int64), torch.ones(2, dtype=torch.int32), torch.ones(3),
                                   torch.ones(6, dtype=torch.int32)[::2], torch.ones((3, 1), dtype=torch.int32),
                                   torch.ones(3, dtype=torch.int32, device="meta")])
def test_counts_of_another_form_are_refused(calls, n_new):
    good = torch.ones(3, dtype=torch.int32)
    for a in ((n_new, None), (good, n_new)):
        with pytest.raises(ValueError, match="n_new|emitted"):
            batch().begin(*a)
    assert not calls


ADVANCE = dict(held=16, window=16, emitted=16, n_new=16, R=2, max_new=4, page=16, table=32, width=4, free_ids=48, n_free=64, n_pages=8,
               held_out=208, window_out=224, table_out=80, free_out=96, n_free_out=112, kv_len=128, q_start=144, slots=160,
               positions=176, tokens=8, status=192, stream=None)


@pytest.mark.parametrize("change", [
    dict(held=None), dict(window=None), dict(n_new=None), dict(table=None), dict(held_out=None), dict(window_out=None),
    dict(held_out=16), dict(window_out=16), dict(table_out=32), dict(free_out=48), dict(n_free_out=64), dict(R=0), dict(R=4097),
    dict(page=24), dict(width=0), dict(n_pages=0), dict(tokens=0), dict(kv_len=None), dict(status=None), dict(max_new=0)])
def test_advance_refusals(lib, change):
    assert lib.svd_paged_advance(*{**ADVANCE, **change}.values()) == svd.SVD_ERR_INVALID_ARG


@pytest.mark.parametrize("who", [torch.ones(3, dtype=torch.int32), torch.ones(2, dtype=torch.bool), torch.ones((3, 1), dtype=torch.bool)])
def test_ends_of_another_form_are_refused(who):
    with pytest.raises(ValueError, match="who"):
        batch().end(who)


def test_a_step_without_tokens():
    """Every request idle: no rows, for which torch has no address either."""
    qkv, out = rows(0)
    assert batch().layer(0, qkv, out) is out
    assert batch().layer(0, *rows(3), n_tokens=0).shape == (3, 4, 128)


def test_one_row_of_any_stride(calls):
    b = batch()
    qkv = torch.zeros((8 * 128, 1)).t()  # [1][1024], whose rows torch says lie one element apart
    b.layer(0, qkv, rows(1)[1])
    a = dict(calls)["svd_paged_append"]
    assert a["n_tokens"] == 1 and a["ld"] >= 8 * 128 and a["ld"] % 4 == 0
