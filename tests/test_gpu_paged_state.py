"""The state that PagedBatch carries from step to step: every page in one place, on any stream."""
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


def i32(*a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def batch(R, **kw):
    a = dict(layers=1, n_pages=8, page_size=16, max_len=64, max_window=64, n_q_heads=2, n_kv_heads=1)
    return paged.PagedBatch(R, **{**a, **kw})


def whole(b):
    """Every page is held by one request or free."""
    held, table = b.held[b.now].tolist(), b.table[b.now].cpu().numpy()
    have = [-(-h // b.page) for h in held]
    ids = np.concatenate([table[r, :n] for r, n in enumerate(have)] + [b.free[b.now].cpu().numpy()[:int(b.n_free[b.now])]])
    assert np.array_equal(np.sort(ids), np.arange(b.n_pages))
    assert all((table[r, n:] == -1).all() for r, n in enumerate(have))


def test_a_step_on_a_stream_that_is_not_the_current_one():
    s = torch.cuda.Stream()
    batch(2).begin(i32(1, 1), stream=s)  # (kernels are loaded at their first use, which waits for the device)
    b = batch(2)
    new, kept = [i32(10, 20), i32(3, 3), i32(2, 2)], [None, i32(4, 20), i32(1, 3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # the current stream is busy for a fifth of a second
    for n, k in zip(new, kept):
        b.begin(n, k, stream=s)
    s.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(s):
        assert b.status.tolist() == [0, 0] and b.kv_len.tolist() == [7, 25] and b.window.tolist() == [2, 2]
    torch.cuda.synchronize()
    whole(b)
