"""What holds at the ends of the arguments' ranges for the windowed and
block-scaled decode holds for a tree that is a chain: those tests, through the
tree's entry."""

import pytest
import torch

from oracle import tree as T
from tests import test_gpu_window_extremes as X

pytestmark = pytest.mark.gpu


class AsTree:
    """The module, with the decode calls as decodes of chains."""

    def __init__(self, m):
        self._m = m

    def __getattr__(self, name):
        return getattr(self._m, name)

    def _chain(self, q):
        return torch.from_numpy(T.chain(q.shape[1]).view("i8")).cuda()

    def mla_decode_paged_window(self, q, cache, table, lens, *, window, sinks=0, **kw):
        assert window == 0
        return self._m.mla_decode_paged_tree(q, cache, table, lens, self._chain(q), **kw)

    def mla_decode_paged_scaled(self, q, cache, scales, table, lens, *, window=0, sinks=0, **kw):
        assert window == 0
        return self._m.mla_decode_paged_tree(q, cache, table, lens, self._chain(q), kv_scales=scales, **kw)


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    mod.mla_get_device_error()
    return AsTree(mod)


@pytest.mark.parametrize("fmt", ["e4m3", "s16", "s64"])
@pytest.mark.parametrize("q_scale", [1e-15, 1e-45])
def test_scores_that_vanish(m, fmt, q_scale):
    X.test_scores_that_vanish(m, fmt, q_scale)


@pytest.mark.parametrize("q_scale,k_scale", [(2.0 ** -100, 2.0 ** 100), (2.0 ** 126, 2.0 ** -100)])
def test_factors_that_only_together_are_in_range(m, q_scale, k_scale):
    X.test_factors_that_only_together_are_in_range(m, q_scale, k_scale)


@pytest.mark.parametrize("far", [2.0 ** 30, 2.0 ** 100])
@pytest.mark.parametrize("split", [0, 1])
def test_blocks_whose_scales_are_far_apart(m, far, split):
    X.test_blocks_whose_scales_are_far_apart(m, far, split)


@pytest.mark.parametrize("fmt", ["e4m3", "s16", "s64"])
@pytest.mark.parametrize("n,split,sink_value", [
    (4096, 0, 1.0), (4096, 64, 1.0), (4096, 64, 0.0), (16384, 1 << 20, 1.0), (16384, 1 << 20, 30.0),
    (65536, 1 << 20, 1.0), (65536, 0, 30.0)])
def test_one_key_far_above_many(m, fmt, n, split, sink_value):
    X.test_one_key_far_above_many(m, fmt, n, 0, 0, split, sink_value)


@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_far_keys_anywhere(m, place):
    X.test_far_keys_anywhere(m, place)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0, 2.0 ** 121])
def test_what_is_no_scale(m, bad):
    X.test_what_is_no_scale(m, bad, 0)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "s32"])
@pytest.mark.parametrize("split", [0, 2])
def test_a_query_that_is_nan(m, fmt, split):
    X.test_a_query_that_is_nan(m, fmt, split)
