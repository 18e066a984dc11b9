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
