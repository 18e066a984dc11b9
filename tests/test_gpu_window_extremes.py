"""The windowed and block-scaled decode at the ends of its arguments' ranges,
against the fp64 oracle."""

import numpy as np
import pytest
import torch

import synth
from oracle import window as W
from tests._helpers import f64
from tests.test_gpu_window_decode import Case, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


@pytest.mark.parametrize("fmt", ["e4m3", "s16", "s64"])
@pytest.mark.parametrize("q_scale", [1e-15, 1e-30, 1e-45])
def test_scores_that_vanish(m, fmt, q_scale):
    """Queries of a tiny scale: every visible key has the same weight, and
    masked ones none, whatever the factor of their block rounds to."""
    c = Case(fmt, [37, 200, 65], 1, 16, 0, 0, seed=200)
    if c.scales is None:
        c.c64 *= 2.0 ** -100 / c.k_scale
        c.row_scale *= 2.0 ** -100 / c.k_scale
        c.k_scale = 2.0 ** -100
    else:
        c.scales[c.scales.isnan()] = 0.0          # as a cleared cache has them
    c.q_scale, c.q64 = q_scale, f64(c.q) * float(np.float32(q_scale))
    out, lse = c.run(m, out_dtype=torch.float32)
    assert m.mla_get_device_error() == 0
    # (values of 2^-100: compared as multiples of it)
    unit = c.k_scale if c.scales is None else 1.0
    ref, ref_l = W.window_decode(c.q64, c.c64, c.bt, c.lens, 1 / np.sqrt(192), 0, 0)
    most = np.abs(c.c64).max() / unit
    # probabilities off by 2^-8, sums of up to 200 in fp32
    assert np.abs(f64(out) / unit - ref / unit).max() <= 2.0 ** -7 * most
    assert np.abs(lse.cpu().numpy() - ref_l).max() <= 1e-4


@pytest.mark.parametrize("q_scale,k_scale", [(2.0 ** -100, 2.0 ** 100), (2.0 ** 100, 2.0 ** -100),
                                             (2.0 ** -120, 2.0 ** 119), (2.0 ** 126, 2.0 ** -100)])
def test_factors_that_only_together_are_in_range(m, q_scale, k_scale):
    """The product of the scales makes the scores, not either by itself."""
    c = Case("e4m3", [130, 300], 1, 16, 0, 0, seed=201)
    args = (c.q.cuda(), c.cache.cuda(), torch.from_numpy(c.bt).cuda(), torch.from_numpy(c.lens).cuda())
    kw = dict(window=0, out_dtype=torch.float32)
    sm = 2.0 ** -12                                   # (codes of a few hundred: scores of a few units)
    base, base_l = m.mla_decode_paged_window(*args, sm_scale=sm, q_scale=1.0, k_scale=1.0, **kw)
    sm = sm / (q_scale * k_scale)                     # (a power of two)
    out, lse = m.mla_decode_paged_window(*args, sm_scale=sm, q_scale=q_scale, k_scale=k_scale, **kw)
    assert m.mla_get_device_error() == 0
    # the same scores, but for the roundings of log2 of the scale and what adds up
    # to it: 2^-17 at 128, a few times, so 2^-14 of a probability, and one e4m3
    # part in lo whose rounding that may tip: 2^-7 of it
    assert float((lse - base_l).abs().max()) <= 2.0 ** -13
    most = float(base.abs().max())
    assert float((out.double() / k_scale - base.double()).abs().max()) <= 2.0 ** -6 * most


@pytest.mark.parametrize("far", [2.0 ** 30, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("split", [0, 1])
def test_blocks_whose_scales_are_far_apart(m, far, split):
    """Blocks of tiny rows (2^-100 a unit) beside blocks of `far`: equal scores,
    so equal weights, and the output is the mean."""
    g = synth.generator(210)
    n, H = 300, 16
    nb = 6
    bt = g.permutation(nb).astype(np.int32)[None, :5]
    scales = np.where(g.random((nb, 4)) < 0.5, far, 2.0 ** -100).astype(np.float32)
    codes = g.integers(0, 127, (nb, 64, 576)).astype(np.uint8)
    codes[..., 512:] = 0
    q = np.zeros((1, 1, H, 576), np.float32)
    q[..., 512:] = g.standard_normal((H, 64))         # (of scores 0: the keys' last columns are)
    q8 = synth.as_e4m3(q)
    c64 = W.scaled_values(codes, scales)
    out, lse = m.mla_decode_paged_scaled(
        q8.cuda(), torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda(),
        _i32(bt), _i32([n]), sm_scale=0.1, out_dtype=torch.float32, split_tiles=split)
    assert m.mla_get_device_error() == 0
    ref, ref_l = W.window_decode(f64(q8), c64, bt, np.array([n]), 0.1, 0, 0)
    assert np.abs(lse.cpu().numpy() - ref_l).max() <= 1e-4
    # probabilities off by 2^-8 of themselves
    assert np.abs(f64(out) - ref).max() <= 2.0 ** -7 * np.abs(ref).max()
