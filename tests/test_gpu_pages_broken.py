"""The cache-page calls on state that is broken already: what they flag, what they
leave, and that it does not spread, bit for bit as their oracle."""

import numpy as np
import pytest

from tests.test_gpu_cache_pages import State, _i32, m  # noqa: F401

pytestmark = pytest.mark.gpu


def _load(s):
    for d, x in zip(s.d, (s.refs, s.table, s.lens)):
        d.copy_(_i32(x))


@pytest.mark.parametrize("shapes", ["bf16", "scaled", "rows"])
def test_fork_of_a_broken_last_page(m, shapes):
    s = State(shapes, 30, 12, 4, [100, 30, 70, 200, 130], seed=60)
    s.table[0, 1], s.table[1, 0] = 30, -1              # no pages
    s.refs[s.table[2, 1]] = 0                          # held, and free
    s.refs[s.table[4, 2]] = -1
    _load(s)
    s.fork(m, [0, 3, 1, 2, 3, 4], [5, 6, 7, 8, 9, 10])
    assert s.lens.tolist() == [100, 30, 70, 200, 130, 100, 200, 30, 70, 200, 130, 0]
    assert [s.table[b, k] for b, k in ((5, 1), (7, 0), (8, 1), (10, 2))] == [-1] * 4
    s.resize(m, [0] * 12)


def test_fork_of_broken_pages_leaves_the_last_pages_to_others(m):
    s = State("bf16", 6, 8, 2, [100, 64, 70], seed=61)      # five pages held, one free
    s.table[0, 1] = 2 ** 31 - 1
    _load(s)
    s.fork(m, [0, 0, 2, 2], [3, 4, 5, 6])
    assert s.lens[3:].tolist() == [100, 100, 70, 0, 0]


@pytest.mark.parametrize("nb", [2000, 20000, 140000])
@pytest.mark.parametrize("n", [1, 3, 100])
def test_a_free_page_goes_to_one_owner(m, nb, n):
    """Of parents' pages one in three is free: they are the lowest free ones, which
    the same call gives to the children that need one."""
    s = State("small", nb, 2 + n, 400, [300 * 64 + 5, 399 * 64 + 63], seed=nb + n)
    held = s.table[0, :301], s.table[1, :400]
    for row in held:
        row[:] = np.sort(row)
    every = np.sort(np.concatenate(held))
    s.refs[:] = 1
    s.refs[every[s.g.random(every.size) < 0.33]] = 0
    s.refs[s.table[0, 300]] = s.refs[s.table[1, 399]] = 1
    _load(s)
    s.fork(m, np.arange(n) % 2, 2 + np.arange(n))
    last = s.table[2:, [300, 399]][np.arange(n), np.arange(n) % 2]
    assert len(set(last.tolist())) == n and (s.refs[last] == 1).all()
    shared = s.table[2:, :300]
    assert not np.isin(last, shared).any()


@pytest.mark.parametrize("row,entry,error", [(0, -1, 1), (7, 40, 1), (40, 39, 16), (4999, 2 ** 31 - 1, 1), (4999, 38, 16)])
def test_compact_flags_entries_where_nothing_moves(m, row, entry, error):
    """Of few sequences and of many: whatever a warp has of the table."""
    for B in (row + 1, 5000):
        s = State("small", 40, B, 9, seed=row)
        s.lens[row], s.table[row, :9] = 9 * 64 - 5, np.arange(9)
        s.refs[:9] = 1
        _load(s)
        s.compact(m)
        s.table[row, 8] = entry
        _load(s)
        s.compact(m)
        s.table[row, 8], s.lens[row] = 8, 9 * 64 + 1
        _load(s)
        m.mla_cache_compact(s.pools, *s.d)
        assert m.mla_get_device_error() == 2
        s.lens[row], s.table[row, 3] = 2 ** 31 - 1, entry
        _load(s)
        s.compact(m)
        s.lens[row] = -2 ** 31
        _load(s)
        s.compact(m)


def test_compact_of_one_long_row(m):
    """More entries than the grid has lanes for at once."""
    nb, n = 400000, 300000
    s = State("small", nb, 1, nb, [64 * n - 1], seed=77)
    s.table[0, n - 1] = nb
    s.table[0, 7] = -1
    _load(s)
    s.compact(m)
    s.compact(m)


@pytest.mark.parametrize("seed", range(40))
def test_any_calls_on_any_state(m, seed):
    """Tables over any pages, counted, and then broken here and there."""
    g = np.random.default_rng(9000 + seed)
    nb, B, mb = (int(np.exp(g.uniform(0, np.log(n)))) for n in (20000, 700, 300))
    s = State("rows" if nb < 100 else "small", nb, B, mb, seed=seed)
    s.lens[:] = g.integers(0, mb * 64 + 1, B) * (g.random(B) < 0.6)
    s.lens[np.cumsum(-(-s.lens // 64)) > nb * g.uniform(0.2, 1.5)] = 0
    for b, n in enumerate(-(-s.lens // 64)):
        s.table[b, :n] = g.integers(0, nb, n)
        np.add.at(s.refs, s.table[b, :n], 1)
    for x, values in ((s.table, [-1, nb, nb - 1, 0, 2 ** 31 - 1, -2 ** 31]), (s.refs, [0, 0, 1, 5, -1, -7]),
                      (s.lens, [-1, mb * 64 + 1, 2 ** 31 - 1, -2 ** 31])):
        here = g.random(x.shape) < g.choice([0, 0.001, 0.02, 0.2])
        x[here] = g.choice(values, here.sum())
    _load(s)
    for _ in range(4):
        what = int(g.integers(0, 4))
        if what == 0:
            s.resize(m, np.where(g.random(B) < 0.5, s.lens, g.integers(0, mb * 64 + 1, B)))
        elif what < 3:
            n = int(np.exp(g.uniform(0, np.log(1500))))
            s.fork(m, g.integers(-1, B, n), g.integers(0, B + 1, n))
        else:
            s.compact(m)
