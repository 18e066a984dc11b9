"""Which pools a fork copies by rows and which by pages: what is taken for rows, and
what the caller says."""

import numpy as np
import pytest
import torch

import synth
from oracle import pages as P
from tests.test_gpu_cache_pages import _i32, m, raw  # noqa: F401

pytestmark = pytest.mark.gpu

U8, BF, F32 = torch.uint8, torch.bfloat16, torch.float32
# a page's shape, its type, and whether it goes by rows if nothing is said
KINDS = [((64,), BF, False), ((64,), U8, False), ((64, 3), U8, False), ((64, 9), BF, False), ((64, 64), U8, True),
         ((64, 2), BF, True), ((64,), F32, True), ((64, 576), BF, True), ((4,), F32, False), ((32, 16), F32, False),
         ((64, 1022), U8, False), ((2, 64), F32, False)]


def _run(m, g, kinds, lens, parents, children, rows, **kw):
    nb = 24
    pools = [torch.from_numpy(g.integers(0, 256, (nb, int(np.prod(s)) * t.itemsize), dtype=np.uint8)).view(t)
             .view(nb, *s).cuda() for s, t, _ in kinds]
    B = len(lens)
    refs, table, lens = np.zeros(nb, np.int32), np.full((B, 4), -1, np.int32), np.array(lens, np.int32)
    perm = g.permutation(nb)
    for b in range(B):
        k = -(-int(lens[b]) // 64)
        table[b, :k], perm = perm[:k], perm[k:]
    refs[table[table >= 0]] = 1
    d, want = [_i32(x) for x in (refs, table, lens)], [raw(p) for p in pools]
    errors = P.fork(want, refs, table, lens, parents, children, rows)
    m.mla_cache_fork(pools, *d, _i32(parents), _i32(children), **kw)
    assert m.mla_get_device_error() == 0 and not errors
    for x, y in zip(d, (refs, table, lens)):
        np.testing.assert_array_equal(x.cpu().numpy(), y)
    for k, (x, y) in enumerate(zip(pools, want)):
        np.testing.assert_array_equal(raw(x), y, err_msg=f"pool {k}: {kinds[k]}")


ONE = dict(lens=[100, 64, 191, 0, 0, 0, 0, 1, 0], parents=[0, 1, 2, 2, 7], children=[3, 4, 5, 6, 8])


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_a_pool_of_its_own(m, kind):
    _run(m, synth.generator(51000 + kind), [KINDS[kind]], **ONE, rows=[KINDS[kind][2]])


def test_all_of_them(m):
    _run(m, synth.generator(51100), KINDS, **ONE, rows=[k[2] for k in KINDS])


def test_what_the_caller_says(m):
    can = [int(np.prod(s)) * t.itemsize % 256 == 0 for s, t, _ in KINDS]
    assert any(c and not k[2] for c, k in zip(can, KINDS))
    g = synth.generator(51200)
    for rows in (can, [False] * len(KINDS), [c and k % 2 == 0 for k, c in enumerate(can)]):
        _run(m, g, KINDS, **ONE, rows=rows, by_rows=rows)
        _run(m, g, KINDS, **ONE, rows=rows, by_rows=tuple(rows))


def test_refusals(m):
    refs, table, lens = _i32([1] * 3), _i32([[0], [-1]]), _i32([30, 0])
    pools = [torch.zeros((3, 64), dtype=BF, device="cuda"), torch.zeros((3, 64), device="cuda")]
    for bad, error in (([True, True], ValueError), ([False], ValueError), ([False] * 3, ValueError), (True, TypeError),
                       ([0, 1], TypeError), ("ab", TypeError), ([False, None], TypeError)):
        with pytest.raises(error, match="by_rows"):
            m.mla_cache_fork(pools, refs, table, lens, _i32([0]), _i32([1]), by_rows=bad)
    assert lens.tolist() == [30, 0] and refs.tolist() == [1] * 3 and m.mla_get_device_error() == 0
