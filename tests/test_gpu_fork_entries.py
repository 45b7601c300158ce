"""Forks over tables with entries that are no pages."""
import numpy as np
import pytest

from test_gpu_fork import run_fork

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def api():
    from block_sparse_gqa_causal_gb300 import api
    return api


@pytest.mark.parametrize("stale", [2, -1, 99])
@pytest.mark.parametrize("changes", [False, True])
def test_an_entry_that_is_no_page_is_taken_as_it_is(api, stale, changes):
    """The source's second entry is -1; the slot that goes on from it has one page and, behind it, what an earlier request left."""
    lens = np.array([3 * 128, 100, 128], np.int32)
    table = np.array([[0, -1, 3], [4, stale, 5], [2, 7, 7]], np.int32)
    ring, free, shares = np.array([5, 6, 7, 1, -1, -1, -1, -1], np.int32), np.array([0, 4], np.int32), np.zeros(8, np.int32)
    src = np.array([2 if changes else 0, 0, 2])
    ws, got = run_fork(api, src, None, (lens, None, table, ring, free, shares))
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    lens2, _, table2, ring2, free2, shares2, moves = got
    assert list(table2[1]) == [0, -1, 3] and list(lens2) == [128 if changes else 384, 384, 128]
    want = np.zeros(8, int)
    if changes:                                # slot 0 lets its pages go, slot 1 holds them; it takes slot 2's
        want[2] = 1
    else:
        want[[0, 3]] = 1
    assert np.array_equal(shares2, want)
    assert list(free2) == [0, 5] and list(ring2[:5]) == [5, 6, 7, 1, 4] and (moves == [-1, -1, 0]).all()
    assert list(table2[2]) == [2, 7, 7] and list(table2[0]) == ([2, -1, 3] if changes else [0, -1, 3])


def test_rows_that_both_end_in_no_page_at_the_same_block(api):
    """Both rows hold -1 at block 1: dropped and taken alike, and recorded."""
    lens = np.array([256, 256], np.int32)
    table = np.array([[0, -1], [1, -1]], np.int32)
    ws, got = run_fork(api, np.array([0, 0]), None, (lens, None, table, np.array([2, 3, -1, -1], np.int32), np.array([0, 2], np.int32), np.zeros(4, np.int32)))
    with pytest.raises(api.MsaError):
        api.check_device_status(ws)
    assert got[2].tolist() == [[0, -1], [0, -1]] and list(got[5]) == [1, 0, 0, 0] and list(got[4]) == [0, 3] and got[3][2] == 1
