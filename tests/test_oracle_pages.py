"""Pins of the tree / cache-page oracles (no GPU): worked examples by hand, the
pinned decode, the pinned append, and what must hold whatever the calls do."""

import numpy as np
import pytest

import synth
from oracle import codecs, mla as O, pages as P, tree as T, window as W


def test_words_of_trees_and_chains():
    #      0
    #     / \
    #    1   2
    #    |  / \
    #    3 4   5
    assert T.words([-1, 0, 0, 1, 2, 2]).tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b100101]
    assert T.words([-1, 0, 1, 2]).tolist() == T.chain(4).tolist() == [1, 3, 7, 15]
    assert int(T.chain(64)[63]) == 2 ** 64 - 1


@pytest.mark.parametrize("length,n,word,want", [
    (5, 2, 0b01, [0, 1, 2, 3]), (5, 2, 0b10, [0, 1, 2, 4]), (5, 2, 0, [0, 1, 2]), (2, 2, 0, []),
    (2, 4, 0b1111, [0, 1]), (2, 4, 0b0110, [0]), (3, 1, 0b10, [0, 1])])
def test_visible(length, n, word, want):
    assert T.visible(length, n, word).tolist() == want


def test_a_chain_is_the_causal_decode():
    g = synth.generator(4)
    lens = np.array([70, 3, 2, 130], np.int32)
    bt, nb = synth.paged_layout(g, lens)
    cache, q = g.standard_normal((nb, 64, 576)), g.standard_normal((4, 3, 2, 576))
    a = T.tree_decode(q, cache, bt, lens, np.tile(T.chain(3), (4, 1)), None, 0.07)
    b = O.paged_decode(q, cache, bt, lens, 0.07)
    np.testing.assert_allclose(a[0], b[0], atol=1e-14)
    np.testing.assert_allclose(a[1], b[1], atol=1e-14)


def test_a_branch_is_the_chain_that_its_path_makes():
    """A node sees what the last of a chain of its path's rows would."""
    g = synth.generator(5)
    parents = [-1, 0, 0, 1, 2, 4, 1]
    bt = np.array([[1, 0]], np.int32)
    cache, q = g.standard_normal((2, 64, 576)), g.standard_normal((1, 7, 3, 576))
    out, lse = T.tree_decode(q, cache, bt, np.array([67]), T.words(parents)[None], None, 0.07)
    for i, path in ((5, [0, 2, 4, 5]), (6, [0, 1, 6])):
        flat = cache.reshape(-1, 576).copy()
        rows = [int(bt[0, (60 + t) // 64]) * 64 + (60 + t) % 64 for t in path]
        to = [int(bt[0, (60 + k) // 64]) * 64 + (60 + k) % 64 for k in range(len(path))]
        flat[to] = flat[rows]
        want = O.paged_decode(q[:, i:i + 1], flat.reshape(2, 64, 576), bt, np.array([60 + len(path)]), 0.07)
        np.testing.assert_allclose(out[0, i], want[0][0, 0], atol=1e-13)
        np.testing.assert_allclose(lse[0, i], want[1][0, 0], atol=1e-13)


def test_copy():
    pool = np.arange(8)[:, None] * np.ones((1, 3), int)
    assert P.copy([pool], [1, 2, -1, 5, 0], [4, 6, 3, 5, 4]) == set()
    assert pool[:, 0].tolist() == [0, 1, 2, 3, 0, 5, 2, 7]      # of the two to page 4 the last
    assert P.copy([pool], [1, 2, 9], [2, 7, 3]) == {"pages", "block"}
    assert pool[:, 0].tolist() == [0, 1, 2, 3, 0, 5, 2, 2]      # page 2 is read: not written


def test_resize():
    refs, table = np.array([1, 0, 0, 2, 1, 1]), np.array([[0, 3, -1], [3, -1, -1], [5, -1, -1]])
    lens = np.array([100, 64, 10])
    assert P.resize(refs, table, lens, np.array([30, 65, 64])) == set()
    assert table.tolist() == [[0, -1, -1], [3, 1, -1], [5, -1, -1]]
    assert refs.tolist() == [1, 1, 0, 1, 1, 1] and lens.tolist() == [30, 65, 64]
    # one free page and the one that the first releases: the last sequence does not get its own
    assert P.resize(refs, table, lens, np.array([0, 192, 191])) == {"pages"}
    assert table.tolist() == [[-1] * 3, [3, 1, 0], [5, -1, -1]] and lens.tolist() == [0, 192, 64]
    assert P.resize(refs, table, lens, np.array([-1, 193, 65])) == {"len"}
    assert table.tolist() == [[-1] * 3, [3, 1, 0], [5, 2, -1]] and lens.tolist() == [0, 192, 65]


def test_fork():
    refs, table = np.array([1, 1, 0, 0, 1]), np.full((4, 3), -1)
    table[0, :2], table[1, 0], lens = [4, 0], 1, np.array([100, 64, 0, 0])
    pool = np.arange(5 * 64 * 16).reshape(5, 64, 16)
    was = pool.copy()
    assert P.fork([pool], refs, table, lens, [0, 1], [3, 2]) == set()
    assert table.tolist() == [[4, 0, -1], [1, -1, -1], [1, -1, -1], [4, 2, -1]] and lens.tolist() == [100, 64, 64, 100]
    assert refs.tolist() == [1, 2, 1, 0, 2]
    assert (pool[2, :36] == was[0, :36]).all() and (pool[2, 36:] == was[2, 36:]).all()


def test_compact():
    refs, table = np.array([0, 2, 0, 0, 1, 0, 3]), np.array([[6, 1], [6, 4], [6, 1]])
    pool = np.arange(7)[:, None].copy()
    assert P.compact([pool], refs, table, np.array([128, 70, 100])) == (3, set())
    assert table.tolist() == [[2, 1], [2, 0], [2, 1]] and refs.tolist() == [1, 2, 3, 0, 0, 0, 0]
    assert pool[:3, 0].tolist() == [4, 1, 6]


def test_accept_moves_rows_in_their_order():
    cache = np.arange(128)[:, None].repeat(576, 1).reshape(2, 64, 576)
    new, err = P.accept([cache], None, np.array([[1, 0]]), np.array([68]), None, 8, np.array([[0, 2, 3, 6, -1]]),
                        np.array([4]))
    assert err == set() and new.tolist() == [64]
    # sequence positions 60 .. 67: page 1 from row 60 on, then page 0
    assert cache[1, 60:, 0].tolist() == [124, 126, 127, 2] and cache[0, :4, 0].tolist() == [0, 1, 2, 3]
    for path, k in (([1, 1], 2), ([2, 1], 2), ([-1, 3], 2), ([0, 8], 2), ([0, 1], 3)):
        assert P.accept([cache], None, np.array([[1, 0]]), np.array([68]), None, 8, np.array([path]),
                        np.array([k]))[1] == {"range"}


def test_accept_of_the_whole_tree_is_an_append_of_its_values():
    """Block-scaled: the accepted rows' values appended behind the context."""
    g = synth.generator(6)
    for sb, ctx, path in ((16, 20, [0, 3, 4, 9, 30]), (64, 100, [0, 1, 2, 7]), (32, 64, [2, 5]), (16, 30, [1, 19])):
        table = np.array([[2, 0, 1]], np.int64)
        codes = codecs.f32_to_e4m3(g.standard_normal((3, 64, 576)).astype(np.float32) * 30)
        scales = np.exp2(g.integers(-5, 4, (3, 64 // sb))).astype(np.float32)
        values = W.scaled_values(codes, scales).reshape(-1, 576)

        def slot(p):
            return int(table[0, p // 64]) * 64 + p % 64

        rows = np.stack([values[slot(ctx + i)] for i in path])
        want = W.append(codes, scales, rows, [slot(ctx + i) for i in range(len(path))])
        got, sc = codes.copy(), scales.copy()
        new, err = P.accept([got], [sc], table, np.array([ctx + 31]), None, 31, np.array([path]),
                            np.array([len(path)]))
        assert err == set() and new.tolist() == [ctx + len(path)]
        assert (got == want[0]).all() and (sc == want[1]).all()


def test_pages_are_held_as_often_as_counted():
    """Over many random calls: refs are the table's counts, and no page is lost."""
    g = synth.generator(7)
    nb, B, mb = 40, 9, 7
    refs, table, lens = np.zeros(nb, int), np.full((B, mb), -1), np.zeros(B, int)
    pool = g.integers(0, 99, (nb, 2))
    for step in range(300):
        what = g.integers(0, 4)
        if what < 2:
            P.resize(refs, table, lens, np.where(g.random(B) < 0.5, lens, g.integers(0, mb * 64 + 1, B)))
        elif what == 2:
            n = g.integers(1, 4)
            P.fork([pool], refs, table, lens, g.integers(0, B, n), g.integers(0, B, n), [False])
        else:
            n, err = P.compact([pool], refs, table, lens)
            assert err == set() and n == (refs > 0).sum() and not refs[n:].any()
        held = np.concatenate([table[b, :-(-lens[b] // 64)] for b in range(B)])
        assert (np.bincount(held, minlength=nb) == refs).all()
