"""What the binding and PagedBatch hand to the library, without a GPU."""
import enum

import numpy as np
import pytest

from speculative_decoding_verify_06_gb300 import build, svd


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build_library()
    return svd.load()


class Address(enum.IntEnum):
    A = 16


@pytest.mark.parametrize("size", [int, np.int32, np.int64, float])
def test_wrappers_convert_sizes_and_addresses(size):
    """Sizes of any numeric type and addresses of any integer type reach the library, whose own
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
