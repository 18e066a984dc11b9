"""The windowed prefill over many items and at the edges of its inputs, against
itself on each request alone."""

import numpy as np
import pytest
import torch

import synth
from tests.test_gpu_window_prefill import SCALE, _i32, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def test_many_short_items(m):
    """Thousands of items of one key tile and less, tens to a CTA, some without a
    key: the sums that the two threads of a row hand each other at the end of one
    are not mistaken for those of the next.  Each request alone is the same."""
    g = synth.generator(83)
    nq = g.integers(1, 300, 60)
    nk = np.maximum(nq - g.integers(0, 2, 60) * g.integers(0, 300, 60), 0) + 3
    q, k, v, cu_q, cu_k = _inputs(84, nq.tolist(), nk.tolist(), 40)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    kw = dict(window=30, sinks=2, sm_scale=SCALE)
    out, lse = m.mla_prefill_attn_window(q, k, v, _i32(cu_q), _i32(cu_k), int(nq.max()), **kw)
    for b in range(60):
        a, z, x, y = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        o, e = m.mla_prefill_attn_window(q[a:z], k[x:y], v[x:y], _i32([0, z - a]), _i32([0, y - x]), int(z - a), **kw)
        assert torch.equal(out[a:z], o) and torch.equal(lse[a:z], e)
    for _ in range(10):
        again = m.mla_prefill_attn_window(q, k, v, _i32(cu_q), _i32(cu_k), int(nq.max()), **kw)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert m.mla_get_device_error() == 0


def test_requests_outside_the_tensors(m):
    """They set the error word and nothing of theirs is written, in the tensors
    or behind them; the other requests are right."""
    q, k, v, cu_q, cu_k = _inputs(85, [100, 300, 50], [100, 300, 50], 2)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    kw = dict(window=60, sinks=1, sm_scale=SCALE)
    want = m.mla_prefill_attn_window(q, k, v, _i32(cu_q), _i32(cu_k), 300, **kw)
    assert m.mla_get_device_error() == 0
    for which, bad, rows in (("q", [0, 100, 400, 451], (0, 400)), ("q", [0, 100, 400, 2 ** 31 - 1], (0, 400)),
                             ("q", [-5, 100, 400, 450], (100, 450)), ("q", [0, 100, 40, 450], (0, 40)),
                             ("k", [0, 100, 400, 451], (0, 400)), ("k", [-1, 100, 400, 450], (100, 450)),
                             ("k", [0, 100, 90, 450], (0, 100))):
        out = torch.full((600, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((600, 2), 7.0, device="cuda")
        cu = (bad, cu_k) if which == "q" else (cu_q, bad)
        m.mla_prefill_attn_window(q, k, v, _i32(cu[0]), _i32(cu[1]), 300, out=out[:450], lse=lse[:450], **kw)
        assert m.mla_get_device_error() == 4, (which, bad)
        a, b = rows
        assert bool((out[450:] == 7.0).all()) and bool((lse[450:] == 7.0).all())
        if bad[0] == 0 and bad[2] == 400 or bad[0] < 0:
            keep = torch.ones(600, dtype=torch.bool)
            keep[a:b] = False
            assert torch.equal(out[a:b], want[0][a:b]) and torch.equal(lse[a:b], want[1][a:b])
            assert bool((out[keep.cuda()] == 7.0).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "both"])
def test_values_that_are_not_finite(m, bad):
    """In tiles that queries see in part and as a whole, at the diagonal, the
    window's edge and among the sinks: the columns of the rows that see them are
    what the definition makes of them, all others bit for bit what they are without."""
    q, k, v, cu_q, cu_k = _inputs(86, [300, 40], [900, 700], 3)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    window, sinks = 200, 5
    kw = dict(window=window, sinks=sinks, sm_scale=SCALE)
    want, want_l = m.mla_prefill_attn_window(q, k, v, _i32(cu_q), _i32(cu_k), 300, **kw)
    vb = v.clone()
    put = {}                                     # (row of v, head, column) -> value
    for i, j in enumerate((0, 3, 5, 401, 500, 630, 760, 880, 899, 900 + 4, 900 + 480, 900 + 699)):
        for h, col in ((i % 3, 7 * i), (2, 100)):
            put[j, h, col] = {"both": float("inf") if i % 2 else -float("inf")}.get(bad, bad)
    for at, x in put.items():
        vb[at] = x
    out, lse = m.mla_prefill_attn_window(q, k, vb, _i32(cu_q), _i32(cu_k), 300, **kw)
    assert m.mla_get_device_error() == 0
    add = torch.zeros((340, 3, 128))
    for (j, h, col), x in put.items():
        b = int(j >= 900)
        for i in range(int(cu_q[b]), int(cu_q[b + 1])):
            p, jj = i - cu_q[b] + (cu_k[b + 1] - cu_k[b]) - (cu_q[b + 1] - cu_q[b]), j - cu_k[b]
            if jj <= p and (p - jj < window or jj < sinks):
                add[i, h, col] += x
    ref = (want.float().cpu() + add)
    got = out.float().cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.nan_to_num(nan=0.0, posinf=1e9, neginf=-1e9), ref.nan_to_num(nan=0.0, posinf=1e9, neginf=-1e9))
    assert torch.equal(lse, want_l)


def test_nan_at_the_end_of_long_windows(m):
    """The last token's values are NaN behind 30000 others, in more items than the
    device has SMs: each call ends within ten times what it takes without, the
    error word stays clear, and the rows before the last are bit for bit the same."""
    H, nk, nq = 160, 30000, 256
    g = torch.Generator(device="cuda").manual_seed(87)
    q, k, v = (torch.randn((n, H, d), generator=g, device="cuda", dtype=torch.bfloat16)
               for n, d in ((nq, 192), (nk, 192), (nk, 128)))
    a = (_i32([0, nq]), _i32([0, nk]), nq)
    kw = dict(window=2 ** 31 - 1, sm_scale=SCALE)
    m.mla_prefill_attn_window(q, k, v, *a, **kw)

    def timed(values):
        t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        torch.cuda.synchronize()
        t[0].record()
        got = m.mla_prefill_attn_window(q, k, values, *a, **kw)
        t[1].record()
        torch.cuda.synchronize()
        return got, t[0].elapsed_time(t[1])

    want, plain = timed(v)
    vb = v.clone()
    vb[-1] = float("nan")
    got, slow = timed(vb)
    assert m.mla_get_device_error() == 0
    assert torch.equal(got[0][:-1], want[0][:-1]) and torch.equal(got[1], want[1])
    assert torch.isnan(got[0][-1]).all()
    assert slow <= 10 * plain
    vb[:] = float("nan")                         # and where every value is
    got, slow = timed(vb)
    assert m.mla_get_device_error() == 0
    assert torch.isnan(got[0]).all() and torch.equal(got[1], want[1])
    assert slow <= 100 * plain
