"""CPU tests of the search by which the cache read finds a packed row's request
(``request_search.h``, built into ``libdspark_hostcheck.so``): over lengths in
order it finds the request, over any words it ends inside the batch."""

import numpy as np
import pytest

from dspark_verify_scheduling_amd import _lib


def search(cu, rows):
    cu, rows = np.ascontiguousarray(cu, np.int32), np.ascontiguousarray(rows, np.int32)
    got = np.empty(len(rows), np.int32)
    _lib.hostcheck().dspark_hostcheck_request_search(cu.ctypes.data, len(cu) - 1, rows.ctypes.data,
                                                     got.ctypes.data, len(rows))
    return got


BATCHES = [1, 2, 4, 63, 64, 65, 300, 4096, 4097, 8192]


@pytest.mark.parametrize("B", BATCHES)
@pytest.mark.parametrize("first", [0, 17])
def test_rows_of_requests_in_order(B, first):
    """Requests of any length, none among them, and a first one that starts later."""
    rng = np.random.default_rng(B)
    cu = np.concatenate([[first], first + np.cumsum(rng.integers(0, 5, B))])
    rows = np.arange(first, cu[-1])
    assert np.array_equal(search(cu, rows), np.searchsorted(cu[:-1], rows, side="right") - 1)
    assert not search(cu, np.arange(first)).any()  # rows of no request


@pytest.mark.parametrize("B", BATCHES)
def test_words_out_of_order_stay_inside_the_batch(B):
    rng = np.random.default_rng(B)
    cu0 = np.concatenate([[0], np.cumsum(rng.integers(2, 5, B))])
    total = int(cu0[-1])
    rows = np.arange(0, total, 1 + total // 500)
    words = [10 ** 6, -5, total, 0, 2 ** 31 - 1, -2 ** 31]
    for at in {0, B // 2, B - 1}:
        for w in words:
            cu = cu0.copy()
            cu[at] = w
            got = search(cu, rows)
            assert got.min() >= 0 and got.max() < B, (at, w)
    for _ in range(8):
        cu = rng.permutation(cu0) if rng.random() < 0.5 else rng.integers(-2 ** 31, 2 ** 31, B + 1)
        got = search(cu, rows)
        assert got.min() >= 0 and got.max() < B
    for cu in (np.full(B + 1, 2 ** 31 - 1), np.full(B + 1, -2 ** 31), cu0[::-1]):
        got = search(cu, rows)
        assert got.min() >= 0 and got.max() < B
