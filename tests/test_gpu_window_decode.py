"""GPU parity of the windowed and the block-scaled decode against the fp64
oracle, at the sizes and masks where they can go wrong.

Bounds (per element; w_j the exact weights): probabilities rounded to 8
significant bits, partial results of a split and the output to bf16 (2^-8
each, relative to half a step), scores off by their fp32 accumulation: the
bound of tests/_helpers.py.  Over an e4m3 cache a probability is held as the
sum of two e4m3 values: off by at most 2^-8 of itself or, when it is small,
half a subnormal step, 2^-10, where the row's largest probability times scale
is at least 2^5 - so 2^-15 of the largest w_j scale_j, times the codes that
it multiplies."""

import numpy as np
import pytest
import torch

import synth
from oracle import codecs, window as W
from tests._helpers import AttnTerms, check_attention, f64, row_terms

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(192)


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Case:
    """fmt: bf16, e4m3, or s16 / s32 / s64 (block-scaled).  Rows that no
    query sees hold NaN, their scales NaN, unseen pages bad block ids."""

    def __init__(self, fmt, lens, q_len, H, window, sinks, seed=0):
        g = synth.generator(9000 + seed)
        self.fmt, self.window, self.sinks = fmt, window, sinks
        self.lens = np.asarray(lens, np.int32)
        B = len(lens)
        self.bt, self.nb = synth.paged_layout(g, np.maximum(self.lens, 1))
        x = g.standard_normal((self.nb, 64, 576), dtype=np.float32)
        x *= np.exp2(g.uniform(-1, 1, (self.nb, 4, 1, 1)).astype(np.float32)).repeat(16, 1).reshape(self.nb, 64, 1)
        q = g.standard_normal((B, q_len, H, 576), dtype=np.float32)
        seen = np.zeros((self.nb, 64), bool)
        for b in range(B):
            for i in range(q_len):
                j = W.visible(int(lens[b]) - q_len + i, window, sinks)
                seen[self.bt[b, j // 64], j % 64] = True
        self.seen = seen
        self.q_scale = self.k_scale = 1.0
        self.scales = None
        if fmt == "bf16":
            self.cache, self.q = synth.as_bf16(x), synth.as_bf16(q)
            self.cache.view(torch.int16)[torch.from_numpy(~seen)] = synth.BF16_NAN_BITS
            self.c64 = f64(self.cache)
        else:
            self.q_scale = float(np.float32(np.abs(q).max() / 448))
            self.q = synth.as_e4m3(q / np.float32(self.q_scale))
            if fmt == "e4m3":
                self.k_scale = float(np.float32(np.abs(x).max() / 448))
                self.cache = synth.as_e4m3(x / np.float32(self.k_scale))
                per_row = np.full((self.nb, 64), self.k_scale)
            else:
                sb = int(fmt[1:])
                blocks = x.reshape(self.nb, 64 // sb, sb * 576)
                s = np.exp2(np.ceil(np.log2(np.abs(blocks).max(axis=2) / 448))).astype(np.float32)
                self.cache = synth.as_e4m3((blocks / s[..., None]).reshape(self.nb, 64, 576))
                per_row = s.repeat(sb, axis=1).astype(np.float64)
                s[~seen.reshape(self.nb, 64 // sb, sb).any(axis=2)] = np.nan
                self.scales = torch.from_numpy(s)
            self.cache.view(torch.uint8)[torch.from_numpy(~seen)] = synth.E4M3_NAN_BITS
            self.row_scale = per_row
            self.c64 = codecs.e4m3_to_f64(self.cache.view(torch.uint8).numpy()) * per_row[..., None]
        page_seen = seen.any(axis=1)
        for b in range(B):
            for k in range(self.bt.shape[1]):
                if self.bt[b, k] >= 0 and not page_seen[self.bt[b, k]]:
                    self.bt[b, k] = -7 if (b + k) % 2 else 1 << 30
        self.c64[~seen] = 0.0
        self.q64 = f64(self.q) * self.q_scale

    def run(self, m, **kw):
        a = (self.q.cuda(), self.cache.cuda())
        b = (_i32(self.bt), _i32(self.lens))
        kw = dict(sm_scale=SCALE, q_scale=self.q_scale, window=self.window, sinks=self.sinks, **kw)
        if self.scales is not None:
            return m.mla_decode_paged_scaled(*a, self.scales.cuda(), *b, **kw)
        return m.mla_decode_paged_window(*a, *b, k_scale=self.k_scale, **kw)

    def check(self, out, lse, label="", out_bf16=True):
        q, bt = self.q64, self.bt
        B, q_len, H, _ = q.shape
        abs_wv, smag = np.zeros((B, q_len, H, 512)), np.zeros((B, q_len, H))
        extra = np.zeros((B, q_len, H, 512))
        ref, ref_l = W.window_decode(q, self.c64, bt, self.lens, SCALE, self.window, self.sinks)
        for b in range(B):
            for i in range(q_len):
                j = W.visible(int(self.lens[b]) - q_len + i, self.window, self.sinks)
                rows = self.c64[bt[b, j // 64], j % 64]
                abs_wv[b, i], smag[b, i], _ = row_terms(q[b, i], rows, rows[:, :512], SCALE)
                if self.fmt != "bf16" and len(j):
                    s = self.row_scale[bt[b, j // 64], j % 64]
                    w = np.exp(SCALE * (q[b, i] @ rows.T) - ref_l[b, i][:, None])
                    top = (w * s).max(axis=1, keepdims=True)
                    extra[b, i] = 2.0 ** -15 * top * np.abs(rows[:, :512] / s[:, None]).sum(axis=0)
        check_attention(f64(out), lse.cpu().numpy(), ref, ref_l, AttnTerms(abs_wv, smag, extra),
                        out_tol=np.inf, lse_tol=np.inf, out_bf16=out_bf16, label=label)


FMTS = ["bf16", "e4m3", "s16", "s32", "s64"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,q_len,H,window,sinks", [
    ([37, 130], 1, 16, 0, 0),                 # ragged, every earlier key
    ([1, 64, 65, 127, 128, 129, 300], 1, 16, 64, 4),      # page and tile borders
    ([0, 2, 1, 5], 3, 5, 2, 1),               # fewer keys than query tokens, rows without a key
    ([700], 1, 16, 128, 4),
    ([500, 90], 2, 20, 1, 0),                 # a window of one token
    ([500, 90], 2, 20, 1, 70),                # sinks over more than a page
    ([400, 260], 4, 16, 100, 1000),           # sinks beyond every length
    ([321], 1, 128, 2 ** 31 - 1, 3),           # a window beyond every length
    ([650, 1000], 1, 200, 192, 64),           # more heads than one group, sinks a whole page
])
def test_against_oracle(m, fmt, lens, q_len, H, window, sinks):
    c = Case(fmt, lens, q_len, H, window, sinks, seed=len(lens) + q_len)
    m.mla_get_device_error()
    out, lse = c.run(m)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} {lens} window {window} sinks {sinks}")


@pytest.mark.parametrize("fmt", ["bf16", "s32"])
@pytest.mark.parametrize("split", [1, 2, 5])
def test_forced_splits_and_fp32_output(m, fmt, split):
    c = Case(fmt, [1500, 3, 700, 0], 2, 24, 600, 130, seed=split)
    out, lse = c.run(m, split_tiles=split, out_dtype=torch.float32)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} split {split}", out_bf16=True)
    again = c.run(m, split_tiles=split, out_dtype=torch.float32)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "s64"])
def test_long_rows_split_over_the_device(m, fmt):
    """Long requests next to short ones: the automatic split cuts them."""
    c = Case(fmt, [9000, 64, 4100], 1, 128, 0, 0, seed=50)
    out, lse = c.run(m)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} long")


@pytest.mark.parametrize("fmt", ["bf16", "s32"])
@pytest.mark.parametrize("lens,q_len,H,window,sinks,split", [
    ([900, 3, 0, 1700, 650, 64, 2, 1100, 40, 500, 777, 1300], 3, 128, 700, 5, 0),   # three row groups
    ([2600, 1, 333], 4, 160, 0, 0, 0),                                          # five
    ([2600, 1, 333], 4, 160, 0, 0, 4),
    ([700, 60], 20, 256, 300, 4, 0),          # forty: too many to plan each apart
])
def test_row_groups(m, fmt, lens, q_len, H, window, sinks, split):
    """More query rows than a pair takes at once, cut and uncut."""
    c = Case(fmt, lens, q_len, H, window, sinks, seed=40 + q_len)
    out, lse = c.run(m, split_tiles=split)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} {lens} x {q_len * H} rows")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_even_parts(m, fmt):
    """Fewer requests than CTA pairs, of lengths alike and not: cut into even
    parts or end to end, the same rows."""
    for n, lens in enumerate(([1100] * 20, [1100 + 7 * i for i in range(30)], [640] * 70,
                              [5000, 0, 1, 64] + [390] * 30)):
        c = Case(fmt, lens, 1, 16, 0, 0, seed=30 + n)
        out, lse = c.run(m)
        assert m.mla_get_device_error() == 0
        c.check(out, lse, f"{fmt} {n}")


def test_partials_of_any_magnitude(m):
    """Values from 2^-90 to 2^90 by runs of 64 columns, cut, rounded to 16 bits
    and merged: every column as good as its own values allow."""
    c = Case("bf16", [1300], 1, 16, 0, 0, seed=65)
    e = np.repeat([-90, 60, 0, 20, -30, -20, -60, 5, 0], 64).astype(np.float64)
    c.cache = (c.cache.double() * torch.from_numpy(np.exp2(e))).bfloat16()
    c.q[..., :512] = 0                      # (scores by the last 64 columns)
    rows = f64(c.cache)[c.bt[0, np.arange(1300) // 64], np.arange(1300) % 64][:, :512]
    most = torch.from_numpy(np.abs(rows).max(axis=0)).cuda()
    run = most.view(4, 128).amax(dim=1, keepdim=True).expand(4, 128).reshape(512)
    want, want_l = c.run(m, out_dtype=torch.float32)
    assert bool((want.abs() > 0).all())
    for kw in (dict(), dict(split_tiles=3)):
        out, lse = c.run(m, **kw)
        # the output's rounding 2^-8; with weights that sum to 1, the bf16
        # probabilities of either call 2^-8 of the column's largest value, the
        # fp16 partials 2^-11 of it or 2^-39 of the largest of 128 columns
        bound = want.double().abs() * 2.0 ** -8 + most * (2.0 ** -7 + 2.0 ** -10) + run * 2.0 ** -38
        assert bool(((out.double() - want.double()).abs() <= bound).all())
        assert float((lse - want_l).abs().max()) <= 1e-4


@pytest.mark.parametrize("fmt", ["bf16", "s16"])
def test_many_requests(m, fmt):
    lens = (np.arange(300) * 37) % 180
    c = Case(fmt, lens, 1, 8, 40, 3, seed=60)
    out, lse = c.run(m)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} 300 requests")


@pytest.mark.parametrize("fmt", ["bf16", "s64"])
def test_nan_of_a_later_token_stays_away_from_earlier_queries(m, fmt):
    """The last of three draft tokens is NaN: only its own query sees it."""
    c = Case(fmt, [200, 77], 3, 16, 50, 2, seed=70)
    last = c.bt[0, 199 // 64], 199 % 64
    if fmt == "bf16":
        c.cache.view(torch.int16)[last] = synth.BF16_NAN_BITS
    else:
        c.cache.view(torch.uint8)[last] = synth.E4M3_NAN_BITS
    out, lse = c.run(m)
    assert torch.isnan(out[0, 2]).all() and torch.isnan(lse[0, 2]).all()
    out[0, 2], lse[0, 2] = 0, 0
    c.lens[0] = 199                     # the first two queries, as the last two of a shorter request
    got_o, got_l = out.clone(), lse.clone()
    got_o[0, 1:], got_l[0, 1:] = out[0, :2], lse[0, :2]
    c.q64[0, 1:] = c.q64[0, :2].copy()
    got_o, got_l = got_o[:, 1:], got_l[:, 1:]
    c.q64 = c.q64[:, 1:]
    c.check(got_o, got_l, f"{fmt} NaN draft token")


@pytest.mark.parametrize("fmt", ["bf16", "s64"])
def test_bad_ids_and_lengths_are_flagged(m, fmt):
    """A seen page with a bad id and a length beyond the table set the error
    word; the other request's rows are right all the same."""
    c = Case(fmt, [300, 200], 1, 16, 0, 0, seed=80)
    good = c.run(m)
    assert m.mla_get_device_error() == 0
    keep = c.bt.copy()
    c.bt[0, 1] = c.nb
    out, lse = c.run(m)
    assert m.mla_get_device_error() == 1
    assert torch.equal(out[1], good[0][1]) and torch.equal(lse[1], good[1][1])
    c.bt = keep
    c.lens[0] = c.bt.shape[1] * 64 + 1
    out, lse = c.run(m)
    assert m.mla_get_device_error() & 2
    assert torch.equal(out[1], good[0][1])


def test_offsets_beyond_32_bits(m):
    """Pages behind the first 4 GiB of a bf16 cache."""
    nb = 60000                                            # 60000 * 73728 B = 4.4 GB
    cache = torch.zeros((nb, 64, 576), dtype=torch.bfloat16, device="cuda")
    c = Case("bf16", [200, 300], 1, 16, 0, 0, seed=90)
    small = c.cache.cuda()
    at = torch.arange(nb - c.nb, nb, device="cuda")
    cache[at] = small
    bt = np.where((c.bt >= 0) & (c.bt < c.nb), c.bt + nb - c.nb, c.bt)
    out, lse = m.mla_decode_paged_window(c.q.cuda(), cache, _i32(bt), _i32(c.lens), sm_scale=SCALE,
                                         window=0)
    want = c.run(m)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("fmt", ["bf16", "s32"])
def test_streams_and_graphs(m, fmt):
    """Two calls at once on streams and workspaces of their own, and a
    captured call replayed on new inputs."""
    a = Case(fmt, [900, 40, 333], 1, 32, 0, 0, seed=100)    # (no window: shorter lengths see seen rows)
    b = Case(fmt, [64, 700], 2, 16, 128, 0, seed=101)
    want = [c.run(m) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, c in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(c.run(m))
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
    q, cache, bt, lens = a.q.cuda(), a.cache.cuda(), _i32(a.bt), _i32(a.lens)
    kw = dict(sm_scale=SCALE, q_scale=a.q_scale, window=a.window, sinks=a.sinks)

    def call():
        if a.scales is not None:
            return m.mla_decode_paged_scaled(q, cache, sc, bt, lens, **kw)
        return m.mla_decode_paged_window(q, cache, bt, lens, k_scale=a.k_scale, **kw)

    sc = None if a.scales is None else a.scales.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    graph.replay()
    assert torch.equal(out, want[0][0])
    lens.copy_(_i32([500, 40, 9]))
    graph.replay()
    fresh = call()
    assert torch.equal(out, fresh[0]) and torch.equal(lse, fresh[1])


def test_the_error_word_stays_clear(m):
    assert m.mla_get_device_error() == 0
