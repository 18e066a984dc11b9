"""Pins of the window / block-scaled-cache oracle (no GPU): against scalar
loops, the pinned unwindowed oracle, and properties of the definitions."""

import math

import numpy as np
import pytest
import torch

import synth
from oracle import codecs, mla as O, window as W


def _cache(seed, lens, **kw):
    g = synth.generator(seed)
    bt, nb = synth.paged_layout(g, lens)
    return g, bt, nb, g.standard_normal((nb, 64, 576))


@pytest.mark.parametrize("p,window,sinks,want", [
    (-1, 4, 2, []), (0, 1, 0, [0]), (5, 2, 0, [4, 5]), (5, 2, 1, [0, 4, 5]),
    (5, 2, 9, [0, 1, 2, 3, 4, 5]), (5, 0, 0, [0, 1, 2, 3, 4, 5]), (2, 10, 1, [0, 1, 2]),
    (6, 3, 4, [0, 1, 2, 3, 4, 5, 6])])
def test_visible(p, window, sinks, want):
    assert W.visible(p, window, sinks).tolist() == want


def test_window_decode_is_the_plain_decode_without_a_window():
    lens = np.array([70, 3, 0], np.int32)
    g, bt, nb, cache = _cache(1, lens)
    q = g.standard_normal((3, 2, 4, 576))
    a = W.window_decode(q, cache, bt, lens, 0.07, 0, 5)
    b = O.paged_decode(q, cache, bt, lens, 0.07)
    np.testing.assert_allclose(a[0], b[0], atol=1e-14)
    np.testing.assert_allclose(a[1], b[1], atol=1e-14)


def test_window_decode_is_a_merge_of_sinks_and_window():
    lens = np.array([200], np.int32)
    g, bt, nb, cache = _cache(2, lens)
    q = g.standard_normal((1, 1, 3, 576))
    out, lse = W.window_decode(q, cache, bt, lens, 0.07, 50, 7)
    parts = [O.paged_decode(q, cache, bt, lens, 0.07, kv_starts=[a], kv_ends=[z])
             for a, z in ((0, 7), (150, 200))]
    mo, ml = O.merge_states(np.stack([p[0][0] for p in parts]), np.stack([p[1][0] for p in parts]))
    np.testing.assert_allclose(out[0], mo, atol=1e-13)
    np.testing.assert_allclose(lse[0], ml, atol=1e-13)


def test_window_prefill_brute_force():
    g = synth.generator(3)
    nq, nk, window, sinks = [4, 2], [9, 2], 3, 2
    cu_q, cu_k = np.cumsum([0] + nq), np.cumsum([0] + nk)
    q, k, v = (g.standard_normal((n, 2, d)) for n, d in ((6, 192), (11, 192), (11, 128)))
    out, lse = W.window_prefill(q, k, v, cu_q, cu_k, 0.1, window, sinks)
    for b in range(2):
        for i in range(nq[b]):
            p, t = i + nk[b] - nq[b], cu_q[b] + i
            for h in range(2):
                num, den = np.zeros(128), 0.0
                for j in range(nk[b]):
                    if j <= p and (p - j < window or j < sinks):
                        w = math.exp(0.1 * float(q[t, h] @ k[cu_k[b] + j, h]))
                        den += w
                        num += w * v[cu_k[b] + j, h]
                # up to nine fp64 terms of at most 4: sums off by 9 * 4 * 2^-52 < 1e-14
                np.testing.assert_allclose(out[t, h], num / den, rtol=1e-12, atol=1e-14)
                assert lse[t, h] == pytest.approx(math.log(den), rel=1e-12)


def test_block_scale_is_the_smallest_power_that_fits():
    for a in (448.0, 448.0001, 1.0, 3.5, 3.5000001, 1e-30, 7e37, 0.875, 1.75, 1.7500002):
        s = W.block_scale(a)
        assert a <= 448.0 * s
        assert a > 448.0 * s / 2 or s == 2.0 ** -100
        assert math.frexp(s)[0] == 0.5
    assert W.block_scale(0.0) == 2.0 ** -100


def test_append_fresh_block_matches_torch_cast():
    g = synth.generator(4)
    x = g.standard_normal((64, 576)).astype(np.float32)
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    codes, sc = W.append(np.zeros((2, 64, 576), np.uint8), np.zeros((2, 1), np.float32), x,
                         np.arange(64) + 64)
    s = W.block_scale(np.abs(x).max())
    assert sc[1, 0] == s and sc[0, 0] == 0
    want = torch.from_numpy((x / s).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert np.array_equal(codes[1], want.numpy())
    assert not codes[0].any()


def test_append_growth_keeps_what_is_there():
    """A larger row makes the block's scale grow; the rows that were there
    stand for the same values to within the coarser step."""
    g = synth.generator(5)
    first = np.clip(g.standard_normal((20, 576)), -3, 3)
    big = 40.0 * g.standard_normal((1, 576))
    codes, sc = W.append(np.zeros((1, 64, 576), np.uint8), np.zeros((1, 1), np.float32), first,
                         np.arange(20))
    before = W.scaled_values(codes, sc)[0, :20]
    codes2, sc2 = W.append(codes, sc, big, [20])
    assert sc2[0, 0] > sc[0, 0]
    after = W.scaled_values(codes2, sc2)[0]
    assert np.all(np.abs(after[:20] - before) <= 2.0 ** -10 * sc2[0, 0])   # half a subnormal step
    assert np.all(np.abs(after[20] - big[0]) <= np.abs(big[0]) * 2.0 ** -4 + 2.0 ** -10 * sc2[0, 0])
    # a smaller row changes nothing that is there
    codes3, sc3 = W.append(codes2, sc2, 0.1 * first[:1], [21])
    assert sc3[0, 0] == sc2[0, 0] and np.array_equal(codes3[0, :21], codes2[0, :21])


def test_append_rules():
    rows = np.ones((3, 576))
    rows[1] *= 2
    rows[2] *= 3
    codes = np.full((1, 64, 576), 0x7E, np.uint8)                # stale rows: 448 each
    sc = np.full((1, 4), 2.0 ** 90, np.float32)
    # the block's first row begins it afresh: the stale scale goes, stale rows keep their bits
    c, s = W.append(codes, sc, rows, [16, 17, -1])
    assert s[0, 1] == W.block_scale(2.0) and np.all(c[0, 18:32] == 0x7E)
    assert np.array_equal(s[0, [0, 2, 3]], sc[0, [0, 2, 3]])
    # the later of two equal slots stays; out of range stores nothing
    c, s = W.append(codes * 0, sc * 0, rows, [3, 64, 3])
    assert np.all(codecs.e4m3_to_f64(c[0, 3]) * s[0, 0] == 3.0) and not c[0, :3].any()


def test_scaled_values_takes_the_scale_of_the_block():
    codes = np.full((2, 64, 576), codecs.f32_to_e4m3(np.float32(1.5)), np.uint8)
    sc = np.arange(8, dtype=np.float32).reshape(2, 4)
    v = W.scaled_values(codes, sc)
    assert v[1, 47, 5] == 1.5 * 6 and v[0, 15, 0] == 0.0 and v[0, 16, 575] == 1.5
