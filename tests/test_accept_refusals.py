"""mla_cache_accept refuses new lengths that lie where it reads (no GPU needed: on
the host, before any launch)."""

import ctypes

import pytest

INVALID = 1
BASE = 1 << 20
P = ctypes.c_void_p


def _accept(m, new, **kw):
    """A call of 5 requests; each array 4 KB behind the last one."""
    at = {k: BASE + 4096 * i for i, k in enumerate(("table", "lens", "tree", "path", "count"))}
    at.update(kw)
    pool = (ctypes.c_void_p * 1)(1 << 30)
    return m.lib.mla_cache_accept(pool, 0, None, 0, 1, 9, P(at["table"]), P(at["lens"]), P(at["tree"]), 8,
                                  P(at["path"]), 6, P(at["count"]), 5, 7, P(new), P(0))


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


@pytest.mark.parametrize("which,words", [(0, 5 * 7), (1, 5), (2, 5), (3, 5 * 6), (4, 5)])
def test_new_lengths_in_what_is_read(m, which, words):
    at = BASE + 4096 * which
    for off in (0, 1, words - 1, -1, -4):
        assert _accept(m, at + 4 * off) == INVALID, off


@pytest.mark.gpu
def test_new_lengths_beside_what_is_read(m):
    """One buffer for all of them, end to end."""
    import torch
    pool = torch.zeros((9, 64, 576), dtype=torch.bfloat16, device="cuda")
    sizes = [5 * 7, 5, 5, 5 * 6, 5]
    for where in range(6):
        buf = torch.zeros(sum(sizes) + 5, dtype=torch.int32, device="cuda")
        parts = torch.split(buf, sizes[:where] + [5] + sizes[where:])
        table, lens, tree, path, count = parts[:where] + parts[where + 1:]
        lens.fill_(40)
        tree.fill_(8)
        path.view(5, 6).copy_(torch.arange(6))
        count.fill_(6)
        table.view(5, 7).copy_(torch.arange(5)[:, None])
        new = m.mla_cache_accept([pool], table.view(5, 7), lens, path.view(5, 6), count, 8, tree_lens=tree,
                                 new_lens=parts[where])
        assert new.data_ptr() == parts[where].data_ptr() and new.tolist() == [38] * 5
    for name, bad in (("path_lens", count), ("tree_lens", tree), ("seq_lens", lens)):
        with pytest.raises(m.MlaError) as e:
            m.mla_cache_accept([pool], table.view(5, 7), lens, path.view(5, 6), count, 8, tree_lens=tree, new_lens=bad)
        assert e.value.status == INVALID, name
    assert m.mla_get_device_error() == 0
