"""Damaged tables and counts of the paged cache: what the page calls refuse."""

import pytest
import torch

import flashattention_backward_gb300 as fa
from test_gpu_cache_pages import Cache, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fa.load_library()
    assert fa.get_device_status() == 0


@pytest.mark.parametrize("column,page", [(0, 4), (1, 4), (2, 4), (1, 9), (2, 9), (2, 3)])
@pytest.mark.parametrize("count", [0, -3])
def test_fork_refuses_entries_of_free_pages(column, page, count):
    """A source's entry, of a full page or of the last, partly filled one, that names a free page: the lowest, which the
    same call would hand out as the new last page, or another.  Nothing changes."""
    c = Cache(10, 4, 4, 5)
    c.extend([9, 4, 0, 0])    # pages 0 1 2 and 3
    if page == 3:
        c.free([1])
    c.table[0, column] = page
    c.refs[page] = count
    before = [t.clone() for t in c.args()]
    moves = fa.pages_fork(*c.args(), ints([0]), ints([2]), 4)
    assert fa.get_device_status() == fa.FA_ERR_PAGES
    assert (moves == -1).all() and all(torch.equal(a, b) for a, b in zip(before, c.args()))
    if page != 3:  # beside a sound pair: that is refused too
        moves = fa.pages_fork(*c.args(), ints([1, 0]), ints([2, 3]), 4)
        assert fa.get_device_status() == fa.FA_ERR_PAGES
        assert (moves == -1).all() and all(torch.equal(a, b) for a, b in zip(before, c.args()))


def test_fork_follows_sound_rows_beside_a_damaged_one():
    """A damaged row of a sequence that is no source does not matter; entries behind a source's pages neither."""
    c = Cache(10, 4, 4, 5)
    c.extend([9, 4, 0, 0])
    c.table[0, 1] = 9
    c.table[1, 1] = 77
    moves = fa.pages_fork(*c.args(), ints([1]), ints([3]), 4)
    assert fa.get_device_status() == 0
    assert moves.tolist() == [[-1, -1, -1]] and c.table[3].tolist() == [3, -1, -1, -1, -1]
    assert c.refs.tolist() == [1, 1, 1, 2, 0, 0, 0, 0, 0, 0] and c.lengths.tolist() == [9, 4, 0, 4]
