"""GPU parity of the windowed prefill attention against the fp64 oracle, with
the bounds of tests/_helpers.py."""

import numpy as np
import pytest
import torch

import synth
from oracle import window as W
from tests._helpers import AttnTerms, check_attention, f64, row_terms

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(192)


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _inputs(seed, nq, nk, H):
    g = synth.generator(seed)
    cu_q = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(nk)]).astype(np.int32)
    q, k, v = (synth.as_bf16(g.standard_normal((n, H, d)))
               for n, d in ((cu_q[-1], 192), (cu_k[-1], 192), (cu_k[-1], 128)))
    return q, k, v, cu_q, cu_k


def _check(out, lse, q, k, v, cu_q, cu_k, window, sinks, label, rows=None):
    q, k, v = f64(q), f64(k), f64(v)
    ro, rl = W.window_prefill(q, k, v, cu_q, cu_k, SCALE, window, sinks)
    abs_wv, smag = np.zeros(ro.shape), np.zeros(rl.shape)
    for b in range(len(cu_q) - 1):
        nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
        for i in range(nq):
            keys = cu_k[b] + W.visible(i + nk - nq, window, sinks)
            for h in range(q.shape[1]):
                a, s, _ = row_terms(q[cu_q[b] + i, h][None], k[keys, h], v[keys, h], SCALE)
                abs_wv[cu_q[b] + i, h], smag[cu_q[b] + i, h] = a[0], s[0]
    o, e = f64(out), lse.cpu().numpy()
    if rows is not None:
        o, e, ro, rl, abs_wv, smag = (x[rows] for x in (o, e, ro, rl, abs_wv, smag))
    check_attention(o, e, ro, rl, AttnTerms(abs_wv, smag), out_tol=np.inf, lse_tol=np.inf, label=label)


@pytest.mark.parametrize("nq,nk,H,window,sinks", [
    ([1], [1], 1, 1, 0),
    ([5, 0, 3], [2, 4, 3], 2, 2, 1),                   # rows before the first key, an empty request
    ([130, 257], [130, 400], 2, 96, 4),                # window within a tile
    ([300], [700], 3, 128, 0),
    ([129], [900], 2, 300, 130),                       # sinks over more than a tile
    ([64, 1], [1000, 777], 2, 1, 5),                   # a window of one token
    ([200], [300], 2, 2 ** 31 - 1, 2 ** 31 - 1),       # beyond every length
    ([140], [640], 1, 200, 1000),                      # sinks beyond every length
    ([512], [1536], 1, 384, 256),                      # borders on tile borders
])
def test_against_oracle(m, nq, nk, H, window, sinks):
    q, k, v, cu_q, cu_k = _inputs(sum(nq) + sum(nk), nq, nk, H)
    m.mla_get_device_error()
    out, lse = m.mla_prefill_attn_window(q.cuda(), k.cuda(), v.cuda(), _i32(cu_q), _i32(cu_k), max(nq),
                                         window=window, sinks=sinks, sm_scale=SCALE)
    assert m.mla_get_device_error() == 0
    _check(out, lse, q, k, v, cu_q, cu_k, window, sinks, f"{nq} of {nk}, window {window}, sinks {sinks}")


def test_a_wide_window_is_the_causal_attention(m):
    q, k, v, cu_q, cu_k = _inputs(31, [200, 300], [500, 300], 3)
    a = (q.cuda(), k.cuda(), v.cuda(), _i32(cu_q), _i32(cu_k), 300)
    got = m.mla_prefill_attn_window(*a, window=4096, sinks=0, sm_scale=SCALE)
    want = m.mla_prefill_attn(*a, causal=True, sm_scale=SCALE)
    # the two add up to 500 probabilities in fp32 in orders of their own: each
    # sum is off by at most 500 * 2^-24 of itself, so the LSEs differ by at
    # most 2 * 500 * 2^-24 (and their own rounding, 2^-21 at 8), and the
    # outputs, whose products are the same, by that and one bf16 step (2^-7)
    assert float((got[1] - want[1]).abs().max()) <= 1000 * 2.0 ** -24 + 2.0 ** -20
    d = (got[0].float() - want[0].float()).abs()
    assert bool((d <= want[0].float().abs() * (2.0 ** -7 + 2.0 ** -13)).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_a_query_does_not_see_stays_away(m, bad):
    """NaN and infinities in the keys and values of one position, which
    shares its tile with others: rows that do not see it are right, rows that
    see it are not finite."""
    nq, nk, window, sinks, j = [150], [400], 60, 3, 330
    q, k, v, cu_q, cu_k = _inputs(77, nq, nk, 2)
    kb, vb = k.clone(), v.clone()
    kb[j], vb[j] = float("nan"), bad
    out, lse = m.mla_prefill_attn_window(q.cuda(), kb.cuda(), vb.cuda(), _i32(cu_q), _i32(cu_k), 150,
                                         window=window, sinks=sinks, sm_scale=SCALE)
    p = np.arange(150) + 250
    sees = (j <= p) & (p - j < window)
    assert not torch.isfinite(out[torch.from_numpy(sees)]).any()
    _check(out, lse, q, k, v, cu_q, cu_k, window, sinks, "NaN elsewhere", rows=~sees)
    # values alone, one column: only that column of the rows that see it
    vb = v.clone()
    vb[j, 1, 17] = bad
    out, lse = m.mla_prefill_attn_window(q.cuda(), k.cuda(), vb.cuda(), _i32(cu_q), _i32(cu_k), 150,
                                         window=window, sinks=sinks, sm_scale=SCALE)
    fin = torch.isfinite(out).cpu().numpy()
    want = np.ones_like(fin)
    want[sees, 1, 17] = False
    assert np.array_equal(fin, want)
    clean = torch.from_numpy(~sees)
    good = m.mla_prefill_attn_window(q.cuda(), k.cuda(), v.cuda(), _i32(cu_q), _i32(cu_k), 150,
                                     window=window, sinks=sinks, sm_scale=SCALE)
    # column 17's chunk of head 1 is computed anew from the definition, in fp32
    d = (out[clean].float() - good[0][clean].float()).abs()
    assert float(d.max()) <= 2.0 ** -6 * float(v.float().abs().max())
    d[:, 1, :32] = 0
    assert float(d.max()) == 0.0


def test_next_requests_nan_stays_away(m):
    """The tile behind a request's last key holds the next request's NaN rows."""
    q, k, v, cu_q, cu_k = _inputs(78, [60, 10], [90, 80], 1)
    kb, vb = k.clone(), v.clone()
    kb[90:], vb[90:] = float("nan"), float("nan")
    out, lse = m.mla_prefill_attn_window(q.cuda(), kb.cuda(), vb.cuda(), _i32(cu_q), _i32(cu_k), 60,
                                         window=40, sinks=2, sm_scale=SCALE)
    _check(out, lse, q, k, v, cu_q, cu_k, 40, 2, "next request NaN", rows=np.arange(70) < 60)
    assert torch.isnan(out[60:]).all()


def test_padding_behind_the_keys(m):
    """Rows behind the last request hold NaN, as a reused buffer may: the last
    tile's values of many keys, one query tile and two."""
    for nq, nk, window in ((300, 2999, 2500), (100, 1201, 40), (1, 77, 1000)):
        q, k, v, cu_q, cu_k = _inputs(80 + nq, [nq], [nk], 2)
        pad = torch.full((200, 2, 192), float("nan"), dtype=torch.bfloat16)
        kb, vb = torch.cat([k, pad]), torch.cat([v, pad[:, :, :128]])
        out, lse = m.mla_prefill_attn_window(q.cuda(), kb.cuda(), vb.cuda(), _i32(cu_q), _i32(cu_k), nq,
                                             window=window, sinks=5, sm_scale=SCALE)
        want = m.mla_prefill_attn_window(q.cuda(), k.cuda(), v.cuda(), _i32(cu_q), _i32(cu_k), nq,
                                         window=window, sinks=5, sm_scale=SCALE)
        assert m.mla_get_device_error() == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])   # (no row was computed anew)


def test_nan_of_a_later_token_in_a_long_window(m):
    """The last token's values are NaN: the rows before it, computed anew from
    their 5000 keys, are right, and so is the error word."""
    q, k, v, cu_q, cu_k = _inputs(81, [140], [6000], 2)
    vb = v.clone()
    vb[5999] = float("nan")
    out, lse = m.mla_prefill_attn_window(q.cuda(), k.cuda(), vb.cuda(), _i32(cu_q), _i32(cu_k), np.int64(140),
                                         window=np.int64(5000), sinks=7, sm_scale=np.float32(SCALE))
    assert m.mla_get_device_error() == 0
    assert torch.isnan(out[139]).all()
    _check(out, lse, q, k, v, cu_q, cu_k, 5000, 7, "NaN behind", rows=np.arange(140) < 139)


def test_a_window_beyond_32_bits(m):
    q, k, v, cu_q, cu_k = _inputs(82, [30], [90], 1)
    a = (q.cuda(), k.cuda(), v.cuda(), _i32(cu_q), _i32(cu_k), 30)
    far = m.mla_prefill_attn_window(*a, window=2 ** 32 + 5, sinks=0, sm_scale=SCALE)
    want = m.mla_prefill_attn_window(*a, window=90, sinks=0, sm_scale=SCALE)
    assert torch.equal(far[0], want[0]) and torch.equal(far[1], want[1])


def test_graph_replay(m):
    q, k, v, cu_q, cu_k = _inputs(79, [100, 40], [300, 40], 2)
    a = [q.cuda(), k.cuda(), v.cuda(), _i32(cu_q), _i32(cu_k), 100]
    kw = dict(window=70, sinks=1, sm_scale=SCALE)
    m.mla_prefill_attn_window(*a, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = m.mla_prefill_attn_window(*a, **kw)
    a[0].copy_(a[0].flip(0))
    graph.replay()
    want = m.mla_prefill_attn_window(*a, **kw)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
