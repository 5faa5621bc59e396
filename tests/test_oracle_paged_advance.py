"""Pins of the carried state's reference against hand-worked steps, and of its reading of bytes that are no numbers."""
import warnings

import numpy as np

from oracle import paged


def test_advance_by_hand():
    # pages of 16.  0: six of ten kept; 1: a count out of order; 2: no room for its tokens in the row; 3: more than
    # max_new; 4: nothing to count (what is said of it is passed over), ends; 5: all kept, takes a page
    table = np.array([[7, 3], [2, -1], [9, 4], [1, 0], [8, -1], [6, -1]], np.int32)
    free = np.array([5, 10, -1, -1, -1, -1, -1, -1, -1, -1, -1], np.int32)
    held, window = [20, 5, 30, 24, 12, 16], [10, 3, 4, 9, -12, 2]
    o = paged.advance(held, window, [6, 4, 1, 2, 3, 2], [2, 1, 6, 8, 0, 4], 7, 16, table, free, 2, 20)
    assert o["status"].tolist() == [0, paged.BAD_REQUEST, paged.BAD_REQUEST, paged.NO_TOKENS, 0, 0]
    assert o["kv_len"].tolist() == [18, 2, 27, 17, 0, 20]
    assert o["held"].tolist() == [18, 5, 30, 24, 0, 20]
    assert o["window"].tolist() == [2, 3, -3, -7, 0, 4]
    assert o["q_start"].tolist() == [0, 2, 2, 2, 2, 2, 6]
    # page 8 goes onto the stack and comes off it again
    assert o["table"].tolist() == [[7, 3], [2, -1], [9, 4], [1, 0], [-1, -1], [6, 8]] and o["n_free"] == 2
    assert o["slots"][:7].tolist() == [3 * 16, 3 * 16 + 1] + [8 * 16 + i for i in range(4)] + [-1]
    # the next step: what was settled is not asked again, what was not is
    o = paged.advance(o["held"], o["window"], [0, 1, 4, 9, 1, 4], [0, 0, 4, 0, 1, 0], 7, 16, o["table"], o["free"], 2, 20)
    assert o["status"].tolist() == [0] * 6 and o["kv_len"].tolist() == [16, 3, 31, 17, 1, 20]
    assert o["window"].tolist() == [0, 0, 4, 0, 1, 0] and o["held"].tolist() == o["kv_len"].tolist()
    assert o["table"][:, :].tolist() == [[7, -1], [2, -1], [9, 4], [1, 0], [3, -1], [6, 8]]


def test_every_count_kept_when_none_is_given():
    table = np.array([[0], [1]], np.int32)
    o = paged.advance([5, 6], [4, -2], None, [1, 1], 8, 16, table, np.full(2, -1, np.int32), 0, 4)
    assert o["kv_len"].tolist() == [6, 5] and o["positions"].tolist() == [5, 4, -1, -1]


def test_bytes_that_are_no_numbers_are_read_quietly():
    pages = np.full((1, 1, 1, paged.UNIT), 0xFF, np.uint8)
    pages.view(np.uint16)[..., 1024:] = 0x7D01  # signalling NaNs
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        k, v = paged.get(pages, [3], 16)
    assert np.isnan(k).all() and np.isnan(v).all()
