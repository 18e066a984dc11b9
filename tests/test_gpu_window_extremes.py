"""The windowed and block-scaled decode at the ends of its arguments' ranges,
against the fp64 oracle."""

import numpy as np
import pytest
import torch

import synth
from oracle import window as W
from tests._helpers import AttnTerms, check_attention, f64, row_terms
from tests.test_gpu_window_decode import Case, _i32
from tests.test_gpu_window_prefill import _check as check_prefill

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


def _scaled(g, values, scales, bt):
    """A block-scaled pool of `values` [n, 576] at positions 0.. of one request."""
    n, sb = len(values), 64 // scales.shape[1]
    pages = -(-n // 64)
    x = np.zeros((scales.shape[0] * 64, 576), np.float32)
    at = bt[0, np.arange(n) // 64] * 64 + np.arange(n) % 64
    s = scales.reshape(-1)[at // sb].astype(np.float64)
    x[at] = values / s[:, None]
    codes = synth.as_e4m3(x.reshape(-1, 64, 576))
    exact = W.scaled_values(codes.view(torch.uint8).numpy(), scales)
    assert pages <= bt.shape[1]
    return codes, exact


@pytest.mark.parametrize("fmt", ["e4m3", "s16", "s64"])
@pytest.mark.parametrize("n,window,sinks,split,sink_value", [
    (4096, 0, 0, 0, 1.0), (4096, 0, 0, 64, 1.0), (4096, 0, 0, 64, 0.0), (16384, 0, 0, 1 << 20, 1.0),
    (16384, 0, 0, 1 << 20, 30.0), (65536, 0, 0, 1 << 20, 1.0), (65536, 0, 0, 0, 30.0),
    (20000, 9000, 4, 1 << 20, 1.0)])
def test_one_key_far_above_many(m, fmt, n, window, sinks, split, sink_value):
    """What sinks are: the first key 8 to 15 nats above thousands of others,
    which together have a weight like its own and values with a common part.
    Half of the heads see the others at exactly the same score, so that their
    probabilities' roundings all go one way.

    Bound: 2^-7 of sum w |V| (tests/_helpers.py), of any number of keys.  A
    probability of 2^-6 or more, as the largest of its row and tile is, is off by
    2^-8 of itself, and by 2^-7 down to 2^-7 (scores that differ by up to 0.7
    nats).  Only the 127 keys beside the first are further below the largest of
    their tile: with 11 nats or less by at most 2^-3 of themselves, 127 of 4096
    keys or more, so 2^-8 of the others' weight; with more by all of it, 127 e^-11
    of sum w at most, where the first key's own value is of the others' size."""
    g = synth.generator(n + window)
    H = 16
    x = g.standard_normal((n, 576)) + 0.5
    x[0, :512] *= sink_value
    x[:, 512] = 0.0
    x[0, 512:] = 0.0
    x[0, 512] = 8.0
    sb = 64 if fmt == "e4m3" else int(fmt[1:])
    pages = -(-n // 64)
    bt = g.permutation(pages + 1).astype(np.int32)[None, :pages]
    if fmt == "e4m3":
        per = np.full((pages + 1, 1), np.float32(np.abs(x).max() / 448))
    else:
        per = np.ones((pages + 1, 64 // sb), np.float32)
        amax = np.abs(x).reshape(-1, sb, 576).max(axis=(1, 2)) if n % sb == 0 else \
            np.array([np.abs(x[i:i + sb]).max() for i in range(0, n, sb)])
        at = np.arange(0, n, sb)
        per[bt[0, at // 64], at % 64 // sb] = np.exp2(np.ceil(np.log2(amax / 448)))
    codes, c64 = _scaled(g, x, per, bt)
    q = np.zeros((1, 1, H, 576))
    gaps = 1.0 + 0.125 * (np.arange(H) // 2 if sink_value else np.arange(H) // 2 % 4)
    q[0, 0, :, 512] = gaps                            # 8 to 15 nats (11 where the first key has no value)
    q[0, 0, 1::2, 513:] = 0.03 * g.standard_normal((H // 2, 63))
    q8 = synth.as_e4m3(q.astype(np.float32))
    kw = dict(sm_scale=1.0, window=window, sinks=sinks, split_tiles=split)
    if fmt == "e4m3":
        out, lse = m.mla_decode_paged_window(q8.cuda(), codes.cuda(), _i32(bt), _i32([n]), k_scale=float(per[0, 0]),
                                             **kw)
    else:
        out, lse = m.mla_decode_paged_scaled(q8.cuda(), codes.cuda(), torch.from_numpy(per).cuda(), _i32(bt),
                                             _i32([n]), **kw)
    assert m.mla_get_device_error() == 0
    j = W.visible(n - 1, window, sinks)
    rows = c64[bt[0, j // 64], j % 64]
    q64 = f64(q8)[0, 0]
    abs_wv, smag, _ = row_terms(q64, rows, rows[:, :512], 1.0)
    s = q64 @ rows.T
    top = s.max(axis=1, keepdims=True)
    p = np.exp(s - top)
    ref = p @ rows[:, :512] / p.sum(axis=1, keepdims=True)
    ref_l = top[:, 0] + np.log(p.sum(axis=1))
    check_attention(f64(out)[0, 0], lse.cpu().numpy()[0, 0], ref, ref_l, AttnTerms(abs_wv, smag),
                    out_tol=np.inf, lse_tol=np.inf, label=f"{fmt} {n} keys, window {window}, split {split}")


@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_far_keys_anywhere(m, place):
    """The key above the others in the first, a middle or the last tile, and
    every tile with one of its own."""
    g = synth.generator(230)
    n, H = 8192, 16
    x = g.standard_normal((n, 576)) + 0.5
    x[:, 512] = 0.0
    hot = {"first": [5], "middle": [4000], "last": [n - 1]}[place]
    x[hot, 512:] = 0.0
    x[hot, 512] = 8.0
    pages = n // 64
    bt = g.permutation(pages).astype(np.int32)[None]
    per = np.full((pages, 4), 2.0 ** -6, np.float32)
    codes, c64 = _scaled(g, x, per, bt)
    q = np.zeros((1, 1, H, 576))
    q[0, 0, :, 512] = 1.0 + 0.125 * (np.arange(H) // 2)
    q[0, 0, 1::2, 513:] = 0.2 * g.standard_normal((H // 2, 63))
    q8 = synth.as_e4m3(q.astype(np.float32))
    for split in (0, 1 << 20):
        out, lse = m.mla_decode_paged_scaled(q8.cuda(), codes.cuda(), torch.from_numpy(per).cuda(), _i32(bt),
                                             _i32([n]), sm_scale=1.0, split_tiles=split)
        assert m.mla_get_device_error() == 0
        rows = c64[bt[0, np.arange(n) // 64], np.arange(n) % 64]
        q64 = f64(q8)[0, 0]
        abs_wv, smag, _ = row_terms(q64, rows, rows[:, :512], 1.0)
        s = q64 @ rows.T
        top = s.max(axis=1, keepdims=True)
        p = np.exp(s - top)
        ref = p @ rows[:, :512] / p.sum(axis=1, keepdims=True)
        check_attention(f64(out)[0, 0], lse.cpu().numpy()[0, 0], ref, top[:, 0] + np.log(p.sum(axis=1)),
                        AttnTerms(abs_wv, smag), out_tol=np.inf, lse_tol=np.inf, label=f"{place}, split {split}")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -1.0, 2.0 ** 121])
@pytest.mark.parametrize("window", [0, 90])
def test_what_is_no_scale(m, bad, window):
    """A scale that is none makes the rows that see its block NaN, in the decode
    as in the gather, and no others."""
    c = Case("s16", [298, 200], 2, 16, window, 0, seed=240)
    c.scales[c.scales.isnan()] = 1.0
    good = c.run(m)
    # the query at 296 sees 207, the last token of its block, and the one at 297
    # with the window does not
    c.scales[int(c.bt[0, 207 // 64]), 207 % 64 // 16] = bad
    out, lse = c.run(m)
    for i, sees in enumerate((True, window == 0)):
        for t in (out[0, i], lse[0, i]):
            assert bool(torch.isnan(t).all()) == sees and bool(torch.isnan(t).any()) == sees
    assert torch.equal(out[1], good[0][1]) and torch.equal(lse[1], good[1][1])
    row = m.mla_gather_cache_scaled(c.cache.cuda(), c.scales.cuda(), _i32(c.bt), _i32(c.lens), _i32([0, 1, 1]),
                                    1, seq_starts=_i32([207, 0]))
    assert bool(torch.isnan(row).all())
    assert m.mla_get_device_error() == 0


def test_append_over_what_is_no_scale(m):
    """A block whose scale is none begins afresh, whatever row is written."""
    kv = torch.ones((3, 576), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((1, 64, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.tensor([[2.0 ** 121, -3.0, float("nan"), 2.0 ** 120]], device="cuda")
    m.mla_rope_cache_append(None, kv[:, 512:], kv[:, :512], _i32([0, 0, 0]), _i32([5, 20, 40]), cache, scales)
    assert m.mla_get_device_error() == 0
    assert scales.tolist() == [[2.0 ** -8] * 3 + [2.0 ** 120]]          # 1 <= 448 * 2^-8


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "s32"])
@pytest.mark.parametrize("split", [0, 2])
def test_a_query_that_is_nan(m, fmt, split):
    """Its row and logarithm are NaN, cut or not; the other rows are right."""
    c = Case(fmt, [2000, 1500], 1, 16, 0, 0, seed=250)
    good = c.run(m, split_tiles=split)
    if fmt == "bf16":
        c.q.view(torch.int16)[0, 0, 3, 7] = synth.BF16_NAN_BITS
    else:
        c.q.view(torch.uint8)[0, 0, 3, 7] = synth.E4M3_NAN_BITS
    out, lse = c.run(m, split_tiles=split)
    assert m.mla_get_device_error() == 0
    assert torch.isnan(out[0, 0, 3]).all() and torch.isnan(lse[0, 0, 3])
    out[0, 0, 3], lse[0, 0, 3] = good[0][0, 0, 3], good[1][0, 0, 3]
    c.check(out, lse, f"{fmt} NaN query, split {split}")


def test_step_element_by_element(m):
    """A prompt's chunk and a decode step over a block-scaled cache as a server
    makes them (append, gather, expand, windowed prefill, append, windowed decode),
    each result within its own elements' bounds: a weight or a sink that is off by
    a few percent does not pass."""
    g = synth.generator(260)
    H, sb, window, sinks, scale = 4, 16, 90, 3, 1 / np.sqrt(192)
    old, new = [170, 33], [60, 41]
    lens = np.array([a + n for a, n in zip(old, new)], np.int32)
    bt, nb = synth.paged_layout(g, lens + 1)
    slots = [bt[b, p // 64] * 64 + p % 64 for b in range(2) for p in range(lens[b])]
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    cache = torch.zeros((nb, 64, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((nb, 64 // sb), device="cuda")
    kv = synth.as_bf16(g.standard_normal((len(slots), 576)) + 0.5).cuda()
    q = synth.as_bf16(g.standard_normal((len(slots), H, 192))).cuda()
    w = synth.as_bf16(g.standard_normal((H * 256, 512)) * 0.05).cuda()
    m.mla_get_device_error()
    m.mla_rope_cache_append(q[:, :, 128:], kv[:, 512:], kv[:, :512], _i32(pos), _i32(slots), cache, scales)
    cu_k = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    cu_q = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rows = m.mla_gather_cache_scaled(cache, scales, _i32(bt), _i32(lens), _i32(cu_k), len(slots))
    K, V = m.mla_expand_kv(rows, w, H)
    qn = q[torch.from_numpy(np.concatenate([cu_k[b] + old[b] + np.arange(new[b]) for b in range(2)])).cuda()]
    out, lse = m.mla_prefill_attn_window(qn, K, V, _i32(cu_q), _i32(cu_k), max(new), window=window, sinks=sinks,
                                         sm_scale=scale)
    check_prefill(out, lse, qn, K, V, cu_q, cu_k, window, sinks, "prefill stage")
    kv1 = synth.as_bf16(g.standard_normal((2, 576)) + 0.5).cuda()
    q1 = g.standard_normal((2, 1, H, 576)).astype(np.float32)
    qs = float(np.float32(np.abs(q1).max() / 448))
    q1 = synth.as_e4m3(q1 / np.float32(qs)).cuda()
    slots1 = [bt[b, lens[b] // 64] * 64 + lens[b] % 64 for b in range(2)]
    m.mla_rope_cache_append(None, kv1[:, 512:], kv1[:, :512], _i32(lens), _i32(slots1), cache, scales)
    out, lse = m.mla_decode_paged_scaled(q1, cache, scales, _i32(bt), _i32(lens + 1), sm_scale=scale, q_scale=qs,
                                         window=window, sinks=sinks)
    assert m.mla_get_device_error() == 0
    c64 = W.scaled_values(cache.view(torch.uint8).cpu().numpy(), scales.cpu().numpy())
    q64 = f64(q1) * qs
    ref, ref_l = W.window_decode(q64, c64, bt, lens + 1, scale, window, sinks)
    abs_wv, smag = np.zeros((2, 1, H, 512)), np.zeros((2, 1, H))
    for b in range(2):
        j = W.visible(int(lens[b]), window, sinks)
        r = c64[bt[b, j // 64], j % 64]
        abs_wv[b, 0], smag[b, 0], _ = row_terms(q64[b, 0], r, r[:, :512], scale)
    # probabilities of 2^-6 of the largest and more off by 2^-8, fewer by 2^-19 of the
    # largest (of 93 keys: 2^-12 of the weights): the bound of bf16 ones holds
    check_attention(f64(out), lse.cpu().numpy(), ref, ref_l, AttnTerms(abs_wv, smag), out_tol=np.inf,
                    lse_tol=np.inf, label="decode stage")
