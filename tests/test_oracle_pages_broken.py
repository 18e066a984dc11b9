"""The cache-page oracles on state that is broken already, by hand (no GPU)."""

import numpy as np

from oracle import pages as P


def test_a_fork_of_a_last_page_that_is_none_takes_no_page():
    for entry, error in ((9, "block"), (-1, "block"), (3, "pages")):
        refs, table, lens = np.array([1, 0, 0, 0]), np.full((4, 2), -1), np.array([100, 30, 0, 0])
        table[0], table[1, 0] = [0, entry], 0
        refs[0] = 2
        pool = np.arange(4 * 64).reshape(4, 64, 1)
        assert P.fork([pool], refs, table, lens, [0, 1], [2, 3]) == {error}
        # the first child has a hole where its parent has none, the second one gets the lowest page
        assert table[2:].tolist() == [[0, -1], [1, -1]] and lens.tolist() == [100, 30, 100, 30]
        assert refs.tolist() == [3, 1, 0, 0] and (pool[1, :30] == pool[0, :30]).all()
        assert pool[2:].ravel().tolist() == list(range(128, 256))


def test_a_page_that_nobody_holds_is_not_shared():
    refs, table, lens = np.array([0, 1, 0, -2]), np.full((4, 3), -1), np.array([192, 70, 0, 0])
    table[0], table[1, :2] = [0, 1, 3], [1, 2]
    refs[1] = 2
    assert P.fork([], refs, table, lens, [0, 1], [2, 3]) == {"pages"}
    assert table[2:].tolist() == [[-1, 1, -1], [1, -1, -1]] and refs.tolist() == [0, 4, 0, -2]


def test_forks_of_a_broken_last_page_leave_the_pages_to_the_others():
    refs, table, lens = np.array([2, 0]), np.array([[5], [0], [0], [-1], [-1]]), np.array([3, 7, 9, 0, 0])
    assert P.fork([np.zeros((2, 64, 1))], refs, table, lens, [0, 1], [3, 4]) == {"block"}
    assert table[:, 0].tolist() == [5, 0, 0, -1, 1] and refs.tolist() == [2, 1] and lens.tolist() == [3, 7, 9, 3, 7]


def test_compact_looks_at_entries_where_nothing_moves():
    refs = np.array([1, 1, 1, 0, 0])
    table, lens = np.array([[0, 1], [2, 9], [4, -1]]), np.array([128, 100, 64])
    assert P.compact([], refs, table, lens) == (3, {"block", "pages"})
    assert table.tolist() == [[0, 1], [2, 9], [4, -1]] and refs.tolist() == [1, 1, 1, 0, 0]
    assert P.compact([], refs, table, np.array([128, 64, 129])) == (3, {"len", "pages", "block"})
    assert P.compact([], refs, table, np.array([128, 64, 0])) == (3, set())
