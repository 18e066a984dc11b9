"""Forks in pools, and of as many sequences, as take 256, 512 and 1024 threads a
CTA of the bookkeeping kernel, and a pool of which a warp has more pages than it
keeps in registers."""

import numpy as np
import pytest

from tests.test_gpu_cache_pages import State, _i32, m  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nb", [16384, 16385, 20000, 131072, 131073, 600001])
def test_fork_in_a_large_pool(m, nb):
    """Free pages lie scattered; most last pages are not full; some forks find no page."""
    B, n = 40, 30
    lens = np.array([100, 64, 63, 1, 700, 0, 128, 129, 640, 65])
    s = State("small", nb, B, 11, lens, seed=nb)
    free = np.flatnonzero(s.refs == 0)
    some = s.g.permutation(free)[:17]
    s.refs[free] = 1                                    # held elsewhere
    s.refs[some] = 0
    s.d[0].copy_(_i32(s.refs))
    children = 10 + s.g.permutation(B - 10)[:n]
    s.fork(m, s.g.integers(0, 10, n), children)
    s.fork(m, s.g.integers(0, B, 12), s.g.integers(0, B, 12))
    s.resize(m, s.lens * (s.g.random(B) < 0.6))
    s.fork(m, s.g.integers(0, B, 20), s.g.integers(0, B, 20))


@pytest.mark.parametrize("B,n", [(512, 40), (513, 40), (700, 600), (1024, 1024), (1025, 30), (40, 512), (40, 513),
                                 (40, 1025)])
def test_fork_of_some(m, B, n):
    s = State("small", 2200, B, 5, [100, 64, 129, 300, 0, 1, 255], seed=B + n)
    s.fork(m, s.g.integers(0, 7, n), s.g.integers(0, B, n))
    s.resize(m, s.lens * (s.g.random(B) < 0.5))
    s.fork(m, s.g.integers(0, B, n), s.g.integers(0, B, n))
