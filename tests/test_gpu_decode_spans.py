"""GPU parity of decodes of more jobs (128 rows of a request) than the device
has pairs of CTAs, whose merge goes by the spans of the plan: jobs uncut, cut
in two and over many spans, with no key at all, and none of any.

Bounds as in test_gpu_window_decode.py."""

import numpy as np
import pytest
import torch

from tests.test_gpu_tree_decode import Case as TreeCase
from tests.test_gpu_window_decode import Case as WindowCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def lengths(B, most, every=7):
    """Of all sizes, some of them 0, the longest last."""
    n = (np.arange(B) * 53 + 11) % most
    n[::every] = 0
    n[-1] = most
    return n.tolist()


def check(m, c, label, dtype):
    m.mla_get_device_error()
    out, lse = c.run(m, out_dtype=dtype)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, label, out_bf16=dtype == torch.bfloat16)
    again = c.run(m, out_dtype=dtype)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "s32"])
@pytest.mark.parametrize("lens,q_len,H,kind,tree_lens,width", [
    (lengths(90, 700), 4, 64, "tree", None, 0),                          # two row groups a request
    (lengths(90, 700), 4, 64, "any", None, 40),                          # bf16: two pages a tile
    (lengths(100, 500), 5, 40, "any", [b * 3 % 6 for b in range(100)], 0),
    ([0] * 79 + [9000], 3, 16, "tree", None, 0),                         # all spans but a few of one job
    ([0] * 100, 2, 16, "any", None, 9),                                  # nothing at all
    ([700] * 36 + [0, 660, 0, 0], 4, 128, "tree", None, 0),               # two whole jobs a pair
    ([0, 700, 690, 641] * 24, 3, 16, "any", None, 0),                    # one
])
def test_trees(m, fmt, dtype, lens, q_len, H, kind, tree_lens, width):
    c = TreeCase(fmt, lens, q_len, H, kind, tree_lens, seed=500 + len(lens) + width, width=width)
    check(m, c, f"{fmt} {len(lens)} trees of {q_len}", dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "s64"])
@pytest.mark.parametrize("lens,q_len,H,window,sinks", [
    (lengths(90, 700), 2, 80, 0, 0),
    (lengths(90, 1500), 2, 64, 500, 4),
    ([0] * 79 + [9000], 1, 16, 0, 0),
    ([0] * 79 + [9000] + [0] * 10 + [700], 1, 16, 2000, 65),
    ([0] * 100 + [1], 2, 16, 0, 0),
])
def test_windows(m, fmt, dtype, lens, q_len, H, window, sinks):
    c = WindowCase(fmt, lens, q_len, H, window, sinks, seed=500 + len(lens) + window)
    if c.bt.shape[1] < 9:                                                # (a table of so few pages is never cut)
        c.bt = np.concatenate([c.bt, np.full((len(lens), 9 - c.bt.shape[1]), -1, c.bt.dtype)], axis=1)
    check(m, c, f"{fmt} {len(lens)} requests of {q_len}", dtype)
