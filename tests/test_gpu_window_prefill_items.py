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
