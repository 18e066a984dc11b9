"""GPU parity of the append to a block-scaled e4m3 cache and of its gather.

The rotation is held to |gpu - ref| <= 2^-8 |ref| + 2^-20 |(a, b)| (one bf16
rounding; the fp32 sine, cosine and products are off by a few 2^-24).  Codes
and scales are compared bit for bit with the oracle's append, which is given
the kernel's own rotated k_pe."""

import numpy as np
import pytest
import torch

import synth
from oracle import mla as O, window as W
from tests._helpers import bits, check_attention, f64, prefill_terms
from tests.test_gpu_rope_cache import _check_rot

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def _pool(g, nb, sb):
    """A pool of random codes without NaN, random power-of-two scales, some 0."""
    codes = g.integers(0, 255, (nb, 64, 576)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 3
    s = np.exp2(g.integers(-12, 3, (nb, 64 // sb))).astype(np.float32)
    s[g.random(s.shape) < 0.2] = 0.0
    return codes, s


def _append(m, codes, scales, slots, pos, q, kv, layout="interleaved", **kw):
    d_c = torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn)
    d_s = torch.from_numpy(scales).cuda()
    m.mla_get_device_error()
    qo, ko = m.mla_rope_cache_append(q, kv[:, 512:], kv[:, :512], _i32(pos), _i32(slots),
                                     d_c, d_s, layout=layout, **kw)
    err = m.mla_get_device_error()
    return qo, ko, bits(d_c), d_s.cpu().numpy(), err


def _rows(kv_c, k):
    return np.concatenate([f64(kv_c), f64(k)], axis=1)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("sb", [16, 32, 64])
@pytest.mark.parametrize("T,H,kind", [(1, 1, "one"), (40, 33, "scattered"), (300, 4, "runs"),
                                      (513, 65, "interleaved"), (70, 128, "fresh")])
def test_append(m, layout, sb, T, H, kind):
    g = synth.generator(7000 + T + sb)
    nb = 12
    codes, scales = _pool(g, nb, sb)
    if kind == "runs":                      # three requests' runs, from anywhere in a page
        slots = np.concatenate([100 + np.arange(150), 333 + np.arange(100), 5 + np.arange(50)])
    elif kind == "interleaved":             # tokens of two runs in turn
        slots = np.where(np.arange(T) % 2 == 0, np.arange(T) // 2, 384 + np.arange(T) // 2)
    elif kind == "fresh":
        slots = 128 + np.arange(T)
    else:
        slots = g.choice(nb * 64, T, replace=False)
    slots = slots.astype(np.int32)
    if T > 10:
        slots[[3, T - 1]] = -1              # padding
    pos = g.integers(0, 200000, T).astype(np.int32)
    pos[0] = 0
    kv = synth.as_bf16(g.standard_normal((T, 576)) * np.exp2(g.integers(-6, 5, (T, 1)))).cuda()
    qfull = synth.as_bf16(g.standard_normal((T, H, 192))).cuda()
    q = qfull[:, :, 128:]                   # strided, as the projection leaves it
    before_q, before_kv = qfull.clone(), kv.clone()
    q_out = torch.empty((T, H, 64), dtype=torch.bfloat16, device="cuda")
    k_out = torch.empty((T, 64), dtype=torch.bfloat16, device="cuda")
    qo, ko, got_c, got_s, err = _append(m, codes, scales, slots, pos, q, kv, layout, q_out=q_out, k_out=k_out)
    assert err == 0 and qo is q_out and ko is k_out
    assert torch.equal(qfull, before_q) and torch.equal(kv, before_kv)
    inter = layout == "interleaved"
    _check_rot(qo, f64(q.contiguous()), pos, inter, f"q {layout}")
    _check_rot(ko, f64(kv[:, 512:].contiguous()), pos, inter, f"k {layout}")
    want_c, want_s = W.append(codes, scales, _rows(kv[:, :512], ko), slots)
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)
    # in place: the same values, the rest of the rows untouched
    qi, ki, got_c, got_s, err = _append(m, codes, scales, slots, pos, q, kv, layout)
    assert torch.equal(qi, q_out) and torch.equal(ki, k_out)
    assert torch.equal(qfull[:, :, :128], before_q[:, :, :128]) and torch.equal(kv[:, :512], before_kv[:, :512])
    assert np.array_equal(got_c, want_c) and np.array_equal(got_s, want_s)


def test_append_far_positions(m):
    """Positions up to 2^31 - 1: the angle's fraction of a turn keeps fp32
    precision (the reference's own fp64 angle is off by 2^31 * 2^-53)."""
    g = synth.generator(7100)
    T = 16
    kv = synth.as_bf16(g.standard_normal((T, 576))).cuda()
    pos = np.concatenate([2 ** 31 - 1 - np.arange(8), g.integers(10 ** 6, 2 ** 31 - 1, 8)]).astype(np.int32)
    x = f64(kv[:, 512:].contiguous())
    _, ko, _, _, _ = _append(m, *_pool(g, 2, 64), np.arange(T), pos, None, kv,
                             k_out=torch.empty((T, 64), dtype=torch.bfloat16, device="cuda"))
    _check_rot(ko, x, pos, True, "far positions")


def test_append_duplicates_out_of_range_and_special_values(m):
    g = synth.generator(7200)
    nb, sb = 3, 32
    codes, scales = _pool(g, nb, sb)
    scales[1, 0] = np.nan                   # not a scale: the block begins afresh
    scales[2, 1] = np.inf
    codes[0, 5, :3] = 0x7F                  # a NaN that is there stays NaN when the scale grows
    slots = np.array([7, 9, 7, 40, nb * 64, 2 ** 31 - 1, -5, 7, 70, 171, 100], np.int32)
    T = len(slots)
    x = g.standard_normal((T, 576)).astype(np.float32)
    x[0] *= 1e6                             # loses its slot to token 7: does not count for the scale
    x[7] *= 3000.0
    x[3, 10], x[3, 11], x[3, 12] = np.inf, -np.inf, np.nan
    x[8] = 0.0
    kv = synth.as_bf16(x).cuda()
    kv[9, :512] = 3.3e38                    # near bf16's largest value
    kv[10, :] = 1e-38                       # below the smallest scale's reach
    pos = np.arange(T, dtype=np.int32)
    k0 = f64(kv[:, 512:].contiguous())
    _, ko, got_c, got_s, err = _append(m, codes, scales, slots, pos, None, kv,
                                       k_out=torch.empty((T, 64), dtype=torch.bfloat16, device="cuda"))
    assert err == 1
    _check_rot(ko, k0, pos, True, "k")      # rotated whatever their slots
    with np.errstate(invalid="ignore"):
        want_c, want_s = W.append(codes, scales, _rows(kv[:, :512], ko), slots)
    assert np.array_equal(got_s, want_s, equal_nan=True)
    nan = (want_c & 0x7F) == 0x7F
    assert np.array_equal((got_c & 0x7F) == 0x7F, nan)
    assert np.array_equal(got_c[~nan], want_c[~nan])


@pytest.mark.parametrize("sb", [16, 32, 64])
@pytest.mark.parametrize("kind", ["random", "runs", "apart"])
def test_append_many_tokens(m, sb, kind):
    """Thousands of tokens: several to a CTA, slots taken twice, padding and
    slots out of range among them, old scales that are no powers of two."""
    g = synth.generator(7300 + sb)
    nb, T = 90, 5000
    codes, scales = _pool(g, nb, sb)
    scales *= g.uniform(1.0, 2.0, scales.shape).astype(np.float32)
    if kind == "random":
        slots = g.integers(-40, nb * 64 + 40, T)
    elif kind == "runs":                    # ten requests' runs, from anywhere in a page
        slots = np.concatenate([576 * r + g.integers(0, 70) + np.arange(500) for r in range(10)])
    else:                                   # neighbours in different blocks, every page twice
        slots = (np.arange(T) * 64 + np.arange(T) // nb // 2) % (nb * 64)
    slots = slots.astype(np.int32)
    pos = g.integers(0, 10 ** 6, T).astype(np.int32)
    kv = synth.as_bf16(g.standard_normal((T, 576)) * np.exp2(g.integers(-6, 5, (T, 1)))).cuda()
    k0 = f64(kv[:, 512:].contiguous())
    _, ko, got_c, got_s, err = _append(m, codes, scales, slots, pos, None, kv, "half")
    assert err == (1 if kind == "random" else 0)
    _check_rot(ko, k0, pos, False, "k")
    want_c, want_s = W.append(codes, scales, _rows(kv[:, :512], ko), slots)
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H", [(9, 1), (33, 16), (17, 17), (5, 64), (3, 129), (2, 300)])
def test_append_query_heads(m, layout, T, H):
    """Head counts on both sides of the groups that a CTA takes; queries whose
    heads are apart and whose tokens are closer than their heads."""
    g = synth.generator(7400 + H)
    kv = synth.as_bf16(g.standard_normal((T, 576))).cuda()
    pos = g.integers(0, 5000, T).astype(np.int32)
    for order in ("token", "head"):
        base = synth.as_bf16(g.standard_normal((T, H, 72) if order == "token" else (H, T, 72))).cuda()
        view = base if order == "token" else base.transpose(0, 1)
        q, before = view[:, :, :64], view.clone()
        want = f64(q.contiguous())
        qo, _, _, _, err = _append(m, *_pool(g, 2, 64), np.full(T, -1), pos, q, kv.clone(), layout)
        assert err == 0 and qo is q
        _check_rot(q, want, pos, layout == "interleaved", f"q {order}")
        assert torch.equal(view[:, :, 64:], before[:, :, 64:])


def test_append_token_by_token_then_read(m):
    """Tokens appended one call at a time, then gathered: every value within
    half an e4m3 step at the block's final scale, plus the half subnormal
    step that each growth of the scale may add."""
    g = synth.generator(7300)
    n, sb = 100, 16
    kv = synth.as_bf16(g.standard_normal((n, 576)) * np.exp2(g.integers(-3, 6, (n, 1)))).cuda()
    cache = torch.zeros((2, 64, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((2, 4), device="cuda")
    k_out = torch.empty((1, 64), dtype=torch.bfloat16, device="cuda")
    rows, bt = [], np.array([[1, 0]], np.int32)
    for t in range(n):
        slot = bt[0, t // 64] * 64 + t % 64
        m.mla_rope_cache_append(None, kv[t:t + 1, 512:], kv[t:t + 1, :512], _i32([t]), _i32([slot]),
                                cache, scales, k_out=k_out)
        rows.append(np.concatenate([f64(kv[t, :512]), f64(k_out[0])]))
    rows = np.stack(rows)
    out = m.mla_gather_cache_scaled(cache, scales, _i32(bt), _i32([n]), _i32([0, n]), n)
    assert m.mla_get_device_error() == 0
    s = scales.cpu().numpy().astype(np.float64)
    per_row = s[bt[0]].reshape(-1).repeat(sb)[:n, None]
    bound = np.abs(rows) * (2.0 ** -4 + 2.0 ** -8) + 2 * 2.0 ** -10 * per_row
    assert np.all(np.abs(f64(out) - rows) <= bound)


@pytest.mark.parametrize("sb", [16, 32, 64])
def test_gather_scaled(m, sb):
    g = synth.generator(7400 + sb)
    lens = np.array([300, 1, 64, 130], np.int32)
    bt, nb = synth.paged_layout(g, lens)
    codes = g.integers(0, 256, (nb, 64, 576)).astype(np.uint8)
    s = np.exp2(g.uniform(-20, 20, (nb, 64 // sb))).astype(np.float32)
    starts = np.array([37, 0, 10, 130], np.int32)
    n = np.array([250, 1, 54, 0])
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    total = int(cu[-1]) + 3
    out = torch.full((total, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    m.mla_get_device_error()
    m.mla_gather_cache_scaled(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(s).cuda(),
                              _i32(bt), _i32(lens), _i32(cu), total, seq_starts=_i32(starts), out=out)
    assert m.mla_get_device_error() == 0
    v = torch.from_numpy(W.scaled_values(codes, s).astype(np.float32)).to(torch.bfloat16)   # one rounding
    want = torch.cat([torch.stack([v[bt[b, p // 64], p % 64] for p in range(starts[b], starts[b] + n[b])])
                      for b in range(4) if n[b]])
    assert torch.equal(out[:int(cu[-1])].cpu().nan_to_num(nan=1234.0), want.nan_to_num(nan=1234.0))
    assert torch.all(out[int(cu[-1]):] == 7.0)          # rows behind the last sequence
    # a range beyond the sequence is flagged and gives zeros
    m.mla_gather_cache_scaled(torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(s).cuda(),
                              _i32(bt), _i32(lens - 60), _i32(cu), total, seq_starts=_i32(starts), out=out)
    assert m.mla_get_device_error() & 4
    assert not out[249].any()


def test_captured_step(m):
    """A decode step (append, then attention over the cache) captured on a
    stream of its own and replayed for the next tokens gives what eager calls
    give, scales and all."""
    g = synth.generator(7700)
    B, H, nb, sb = 3, 32, 40, 32
    bt = _i32(g.permutation(nb - 1)[:B * 12].reshape(B, 12))
    codes, scales = _pool(g, nb, sb)
    base = np.array([500, 63, 130], np.int32)
    steps = [(synth.as_bf16(g.standard_normal((B, 576)) * 2.0 ** i).cuda(),
              synth.as_bf16(g.standard_normal((B, H, 64))).cuda(),
              synth.as_e4m3(g.standard_normal((B, 1, H, 576)).astype(np.float32)).cuda()) for i in range(4)]

    def state():
        return (torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda(),
                steps[0][0].clone(), steps[0][1].clone(), steps[0][2].clone(), _i32(base))

    def step(cache, sc, kv, q_pe, q, pos):
        p = pos.long()
        slots = (bt.long().gather(1, (p // 64)[:, None])[:, 0] * 64 + p % 64).int()
        m.mla_rope_cache_append(q_pe, kv[:, 512:], kv[:, :512], pos, slots, cache, sc)
        return m.mla_decode_paged_scaled(q, cache, sc, bt, pos + 1, sm_scale=0.05, window=200, sinks=3)

    eager, got = state(), state()
    want = []
    for i, (kv, q_pe, q) in enumerate(steps):
        for t, x in zip(eager[2:5], (kv, q_pe, q)):
            t.copy_(x)
        eager[5].copy_(_i32(base + i))
        want.append([t.clone() for t in step(*eager)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*state())                      # warm-up on tensors of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = step(*got)
        for i, (kv, q_pe, q) in enumerate(steps):
            for t, x in zip(got[2:5], (kv, q_pe, q)):
                t.copy_(x)
            got[5].copy_(_i32(base + i))
            graph.replay()
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0].view(torch.uint8), eager[0].view(torch.uint8)) and torch.equal(got[1], eager[1])
    assert m.mla_get_device_error() == 0


def test_calls_close_behind_one_another(m):
    """Append, gather, prefill and decode on the same cache, twenty times over
    without a wait between them (each starts while the one before drains), give
    bit for bit what they give with a wait behind each call."""
    g = synth.generator(7800)
    B, H, sb, window, sinks, nb, new = 4, 16, 16, 150, 3, 60, 37
    bt = g.permutation(nb - 1)[:B * 14].reshape(B, 14).astype(np.int32)
    w = synth.as_bf16(g.standard_normal((H * 256, 512)) * 0.05).cuda()
    steps = []
    for i in range(20):
        lens = np.full(B, (i + 1) * new) + np.arange(B)
        slots = np.concatenate([bt[b, np.arange(n - new, n) // 64] * 64 + np.arange(n - new, n) % 64
                                for b, n in enumerate(lens)])
        kv = synth.as_bf16(g.standard_normal((B * new, 576)) * 2.0 ** (i % 5)).cuda()
        q = synth.as_bf16(g.standard_normal((B * new, H, 192))).cuda()
        q1 = synth.as_e4m3(g.standard_normal((B, 1, H, 576)).astype(np.float32)).cuda()
        steps.append((kv, q, q1, _i32(lens), _i32(slots), _i32(np.arange(B * new)),
                      _i32(np.concatenate([[0], np.cumsum(lens)])), int(lens.sum()),
                      _i32(np.arange(B + 1) * new)))
    table = _i32(bt)

    def run(wait):
        cache = torch.zeros((nb, 64, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        sc = torch.zeros((nb, 64 // sb), device="cuda")
        got = []
        for kv0, q0, q1, lens, slots, pos, cu_k, total, cu_q in steps:
            kv, q = kv0.clone(), q0.clone()
            torch.cuda.synchronize()
            m.mla_rope_cache_append(q[:, :, 128:], kv[:, 512:], kv[:, :512], pos, slots, cache, sc)
            wait()
            rows = m.mla_gather_cache_scaled(cache, sc, table, lens, cu_k, total)
            wait()
            K, V = m.mla_expand_kv(rows, w, H)
            wait()
            a = m.mla_prefill_attn_window(q, K, V, cu_q, cu_k, new, window=window, sinks=sinks, sm_scale=0.07)
            wait()
            b = m.mla_decode_paged_scaled(q1, cache, sc, table, lens, sm_scale=0.01, window=0)
            wait()
            c = m.mla_decode_paged_scaled(q1, cache, sc, table, lens, sm_scale=0.01, window=window, sinks=sinks)
            wait()
            got += [rows, q, *a, *b, *c]
        torch.cuda.synchronize()
        return got + [cache.view(torch.uint8), sc]

    want, got = run(torch.cuda.synchronize), run(lambda: None)
    assert m.mla_get_device_error() == 0
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_step_over_a_scaled_cache(m):
    """One serving step as it is used: a prompt's chunk is appended, its
    context gathered, expanded and attended to with a window; then a decode
    step appends one token and attends over the cache; each stage against the
    oracle on the stage's own inputs."""
    g = synth.generator(7500)
    H, sb, window, sinks, scale = 4, 32, 100, 4, 1 / np.sqrt(192)
    old, new = [150, 20], [70, 33]
    lens = np.array([a + n for a, n in zip(old, new)], np.int32)
    bt, nb = synth.paged_layout(g, lens + 1)
    slots = [bt[b, p // 64] * 64 + p % 64 for b in range(2) for p in range(lens[b])]
    pos = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    T = len(slots)
    cache = torch.zeros((nb, 64, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.zeros((nb, 64 // sb), device="cuda")
    kv = synth.as_bf16(g.standard_normal((T, 576))).cuda()
    q = synth.as_bf16(g.standard_normal((T, H, 192))).cuda()
    w = synth.as_bf16(g.standard_normal((H * 256, 512)) * 0.05).cuda()
    m.mla_get_device_error()
    m.mla_rope_cache_append(q[:, :, 128:], kv[:, 512:], kv[:, :512], _i32(pos), _i32(slots), cache, scales)
    cu_k = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = m.mla_gather_cache_scaled(cache, scales, _i32(bt), _i32(lens), _i32(cu_k), T)
    want = W.scaled_values(bits(cache), scales.cpu().numpy()).reshape(-1, 576)[slots]
    assert np.array_equal(f64(rows), want)              # scales are powers of two: exact in bf16
    K, V = m.mla_expand_kv(rows, w, H)
    new_rows = np.concatenate([cu_k[b] + old[b] + np.arange(new[b]) for b in range(2)])
    qn = q[torch.from_numpy(new_rows).cuda()].contiguous()
    cu_q = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out, lse = m.mla_prefill_attn_window(qn, K, V, _i32(cu_q), _i32(cu_k), max(new), window=window,
                                         sinks=sinks, sm_scale=scale)
    ro, rl = W.window_prefill(f64(qn), f64(K), f64(V), cu_q, cu_k, scale, window, sinks)
    # the terms of the unwindowed rows bound those of the window's keys in smag;
    # sum w |V| <= max |V| over all keys
    t = prefill_terms(f64(qn), f64(K), f64(V), cu_q, cu_k, True, scale)
    t.abs_wv = np.maximum(t.abs_wv, np.abs(f64(V)).max())
    check_attention(f64(out), lse.cpu().numpy(), ro, rl, t, out_tol=np.inf, lse_tol=np.inf, label="prefill stage")
    # decode step
    kv1 = synth.as_bf16(g.standard_normal((2, 576))).cuda()
    q1 = g.standard_normal((2, 1, H, 576)).astype(np.float32)
    qs = float(np.abs(q1).max() / 448)
    q1 = synth.as_e4m3(q1 / np.float32(qs)).cuda()
    slots1 = [bt[b, lens[b] // 64] * 64 + lens[b] % 64 for b in range(2)]
    m.mla_rope_cache_append(None, kv1[:, 512:], kv1[:, :512], _i32(lens), _i32(slots1), cache, scales)
    out, lse = m.mla_decode_paged_scaled(q1, cache, scales, _i32(bt), _i32(lens + 1), sm_scale=scale,
                                         q_scale=qs, window=window, sinks=sinks)
    assert m.mla_get_device_error() == 0
    c64 = W.scaled_values(bits(cache), scales.cpu().numpy())
    ro, rl = W.window_decode(f64(q1) * qs, c64, bt, lens + 1, scale, window, sinks)
    # 8-bit probabilities held in two parts, the output in bf16: 2^-7 of sum w |V|
    err = np.abs(f64(out) - ro)
    assert np.all(err <= 2.0 ** -7 * np.abs(c64).max() + 2.0 ** -8 * np.abs(ro))
    assert np.abs(lse.cpu().numpy() - rl).max() <= 1e-3
