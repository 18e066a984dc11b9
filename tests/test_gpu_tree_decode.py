"""GPU parity of the decode of drafted trees against the fp64 oracle, at the
sizes and masks where it can go wrong.

Bounds as in test_gpu_window_decode.py, whose kernel this is: that of
tests/_helpers.py and, over an e4m3 cache, 2^-15 of the largest weight times
scale for every code that it multiplies."""

import numpy as np
import pytest
import torch

import synth
from oracle import codecs, tree as T
from tests._helpers import AttnTerms, check_attention, f64, row_terms

pytestmark = pytest.mark.gpu

SCALE = 1 / np.sqrt(192)
FMTS = ["bf16", "e4m3", "s16", "s32", "s64"]


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def tree_words(g, q_len):
    """A random tree, every node below one of the few in front of it."""
    return T.words([-1] + [max(0, i - 1 - int(g.integers(0, 4))) for i in range(1, q_len)])


class Case:
    """fmt: bf16, e4m3, or s16 / s32 / s64 (block-scaled).  kind of masks: tree,
    chain, any (random words, some of them 0) or one (a tree for all).  Rows
    that nobody sees hold NaN, their scales NaN; queries behind a tree's last
    token are NaN; pages behind a sequence, up to `width`, have bad ids."""

    def __init__(self, fmt, lens, q_len, H, kind="tree", tree_lens=None, seed=0, width=0):
        g = synth.generator(12000 + seed)
        self.fmt, self.kind = fmt, kind
        self.lens, B = np.asarray(lens, np.int32), len(lens)
        self.tree_lens = None if tree_lens is None else np.asarray(tree_lens, np.int32)
        self.n = [q_len] * B if tree_lens is None else list(tree_lens)
        if kind == "any":
            words = g.integers(0, 1 << 64, (B, q_len), dtype=np.uint64)
            words[g.random((B, q_len)) < 0.2] = 0
        elif kind == "chain":
            words = np.tile(T.chain(q_len), (B, 1))
        elif kind == "one":
            words = np.tile(tree_words(g, q_len), (B, 1))
        else:
            words = np.stack([tree_words(g, q_len) for _ in range(B)])
        self.words = words
        self.bt, self.nb = synth.paged_layout(g, np.maximum(self.lens, 1))
        more = max(0, width - self.bt.shape[1])
        self.bt = np.concatenate([self.bt, np.full((B, more), -1, self.bt.dtype)], axis=1)
        x = g.standard_normal((self.nb, 64, 576), dtype=np.float32)
        x *= np.exp2(g.uniform(-1, 1, (self.nb, 4, 1, 1)).astype(np.float32)).repeat(16, 1).reshape(self.nb, 64, 1)
        q = g.standard_normal((B, q_len, H, 576), dtype=np.float32)
        seen = np.zeros((self.nb, 64), bool)
        for b in range(B):
            for i in range(self.n[b]):
                j = T.visible(int(lens[b]), self.n[b], words[b, i])
                seen[self.bt[b, j // 64], j % 64] = True
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
        for b in range(B):
            used = -(-int(lens[b]) // 64)
            self.bt[b, used:] = np.where(np.arange(used, self.bt.shape[1]) % 2, -7, 1 << 30)
            if self.n[b] < q_len:
                bits = self.q[b, self.n[b]:].view(torch.int16 if fmt == "bf16" else torch.uint8)
                bits.fill_(synth.BF16_NAN_BITS if fmt == "bf16" else synth.E4M3_NAN_BITS)
        self.c64[~seen] = 0.0
        self.q64 = f64(self.q) * self.q_scale

    def mask(self):
        w = self.words[0] if self.kind == "one" else self.words
        return torch.from_numpy(np.ascontiguousarray(w).view(np.int64)).cuda()

    def run(self, m, **kw):
        return m.mla_decode_paged_tree(
            self.q.cuda(), self.cache.cuda(), _i32(self.bt), _i32(self.lens), self.mask(), sm_scale=SCALE,
            q_scale=self.q_scale, k_scale=self.k_scale, kv_scales=None if self.scales is None else self.scales.cuda(),
            tree_lens=None if self.tree_lens is None else _i32(self.tree_lens), **kw)

    def check(self, out, lse, label="", out_bf16=True):
        q, bt = self.q64, self.bt
        B, q_len, H, _ = q.shape
        ref, ref_l = T.tree_decode(q, self.c64, bt, self.lens, self.words, self.tree_lens, SCALE)
        abs_wv, smag = np.zeros((B, q_len, H, 512)), np.zeros((B, q_len, H))
        extra = np.zeros((B, q_len, H, 512))
        for b in range(B):
            for i in range(self.n[b]):
                j = T.visible(int(self.lens[b]), self.n[b], self.words[b, i])
                rows = self.c64[bt[b, j // 64], j % 64]
                abs_wv[b, i], smag[b, i], _ = row_terms(q[b, i], rows, rows[:, :512], SCALE)
                if self.fmt != "bf16" and len(j):
                    s = self.row_scale[bt[b, j // 64], j % 64]
                    w = np.exp(SCALE * (q[b, i] @ rows.T) - ref_l[b, i][:, None])
                    top = (w * s).max(axis=1, keepdims=True)
                    extra[b, i] = 2.0 ** -15 * top * np.abs(rows[:, :512] / s[:, None]).sum(axis=0)
        empty = np.isneginf(ref_l)
        assert not f64(out)[empty].any() and np.isneginf(lse.cpu().numpy()[empty]).all()
        check_attention(f64(out), lse.cpu().numpy(), ref, ref_l, AttnTerms(abs_wv, smag, extra),
                        out_tol=np.inf, lse_tol=np.inf, out_bf16=out_bf16, label=label)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,q_len,H,kind,tree_lens", [
    ([37, 130], 4, 16, "tree", None),
    ([64, 65, 67, 128, 129, 132, 1000], 5, 16, "tree", None),        # trees over page and tile borders
    ([5, 5, 9, 3, 0, 1], 5, 5, "any", None),                         # no context, fewer keys than tokens, none
    ([300, 64], 1, 16, "tree", None),                                # one token
    ([300, 64], 1, 16, "any", None),
    ([200, 90, 64], 64, 2, "any", None),                             # the widest tree, every bit
    ([700], 64, 16, "tree", None),                                   # eight row groups
    ([333, 40, 7, 90], 33, 20, "tree", [33, 7, 0, 20]),              # ragged, one without a tree
    ([333, 40, 7, 90], 33, 20, "any", [1, 33, 7, 32]),
    ([150, 20, 64], 6, 24, "one", [6, 2, 5]),                        # one tree for all, cut
    ([650, 130], 3, 200, "tree", None),                              # rows that end inside a group
])
def test_against_oracle(m, fmt, lens, q_len, H, kind, tree_lens):
    c = Case(fmt, lens, q_len, H, kind, tree_lens, seed=len(lens) + q_len)
    m.mla_get_device_error()
    out, lse = c.run(m)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} {lens} {kind}")


WIDE = 5000       # pages of a table with which bf16 keys are taken 128 at a time


@pytest.mark.parametrize("lens,q_len,H,kind,tree_lens,split", [
    ([37, 130], 4, 16, "tree", None, 0),
    ([64, 65, 67, 128, 129, 132, 1000], 5, 16, "tree", None, 0),
    ([5, 5, 9, 3, 0, 1], 5, 5, "any", None, 0),
    ([300, 192, 256, 257], 1, 16, "any", None, 1),
    ([200, 90, 64], 64, 2, "any", None, 0),
    ([700], 64, 16, "tree", None, 0),
    ([333, 40, 7, 90], 33, 20, "tree", [33, 7, 0, 20], 0),
    ([333, 40, 7, 90, 1500], 33, 20, "any", [1, 33, 7, 32, 33], 2),
    ([150, 20, 64], 6, 24, "one", [6, 2, 5], 0),
    ([650, 130, 1300], 3, 200, "tree", None, 0),
    ([2300, 3, 700, 0, 1500], 9, 32, "any", [9, 3, 5, 0, 9], 1),
    ([2300, 3, 700, 0, 1500], 9, 32, "any", [9, 3, 5, 0, 9], 5),
    ([130] * 12, 20, 128, "tree", None, 0),
])
def test_wide_tiles(m, lens, q_len, H, kind, tree_lens, split):
    """The tiles of two pages that many pages of a bf16 cache are taken by."""
    c = Case("bf16", lens, q_len, H, kind, tree_lens, seed=300 + len(lens) + q_len, width=WIDE)
    m.mla_get_device_error()
    out, lse = c.run(m, split_tiles=split)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"wide {lens} {kind} split {split}")
    again = c.run(m, split_tiles=split)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_wide_tiles_of_uncut_jobs(m):
    """Many jobs of so few pages that none is cut."""
    c = Case("bf16", [(37 * b) % 200 for b in range(210)], 8, 60, "tree", seed=320, width=6)
    out, lse = c.run(m)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, "wide, uncut")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "s32"])
@pytest.mark.parametrize("split", [0, 1, 2, 5])
def test_splits_and_fp32_output(m, fmt, split):
    c = Case(fmt, [1500, 3, 700, 0, 2300], 9, 32, "any", [9, 3, 5, 0, 9], seed=split)
    out, lse = c.run(m, split_tiles=split, out_dtype=torch.float32)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} split {split}")
    again = c.run(m, split_tiles=split, out_dtype=torch.float32)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", ["bf16", "s64"])
@pytest.mark.parametrize("lens,q_len,H", [([900, 300, 64], 3, 128), ([1100], 4, 128), ([130] * 12, 20, 128),
                                          ([5000], 2, 128), ([640] * 50, 2, 64)])
def test_row_groups(m, fmt, lens, q_len, H):
    """Row groups planned apart, by request, and cut."""
    c = Case(fmt, lens, q_len, H, "tree", seed=40 + q_len)
    out, lse = c.run(m)
    assert m.mla_get_device_error() == 0
    c.check(out, lse, f"{fmt} {lens} x {q_len * H} rows")


@pytest.mark.parametrize("fmt", FMTS)
def test_a_chain_is_the_causal_decode(m, fmt):
    """The same definition: the same oracle values hold for both."""
    c = Case(fmt, [900, 64, 33, 2, 1], 4, 16, "chain", seed=7)
    out, lse = c.run(m)
    a = (c.q.cuda(), c.cache.cuda())
    b = (_i32(c.bt), _i32(c.lens))
    if c.scales is not None:
        want = m.mla_decode_paged_scaled(*a, c.scales.cuda(), *b, sm_scale=SCALE, q_scale=c.q_scale)
    else:
        want = m.mla_decode_paged_window(*a, *b, sm_scale=SCALE, window=0, q_scale=c.q_scale, k_scale=c.k_scale)
    c.check(out, lse, f"{fmt} chain")
    c.check(*want, "causal")


@pytest.mark.parametrize("fmt,width", [("bf16", 0), ("bf16", WIDE), ("s64", 0)])
def test_nan_of_a_drafted_token_stays_with_those_that_see_it(m, fmt, width):
    """And NaN in the context makes the tree's rows NaN, but no row behind it."""
    c = Case(fmt, [200, 77], 6, 16, "tree", [6, 4], seed=70, width=width)
    out, lse = c.run(m)
    at = c.bt[0, 197 // 64], 197 % 64                     # node 3 of 6
    bits = (lambda t: t.view(torch.int16)) if fmt == "bf16" else (lambda t: t.view(torch.uint8))
    nan = synth.BF16_NAN_BITS if fmt == "bf16" else synth.E4M3_NAN_BITS
    sees = torch.tensor([int(w) >> 3 & 1 for w in c.words[0]], dtype=torch.bool)
    bits(c.cache)[at] = nan
    got, got_l = c.run(m)
    assert torch.isnan(got[0][sees]).all() and torch.isnan(got_l[0][sees]).all()
    assert torch.equal(got[0][~sees], out[0][~sees]) and torch.equal(got[1], out[1])
    bits(c.cache)[c.bt[1, 0], 5] = nan
    got, got_l = c.run(m)
    assert torch.isnan(got[1, :4]).all() and not got[1, 4:].any() and torch.isneginf(got_l[1, 4:]).all()


@pytest.mark.parametrize("fmt", ["bf16", "s64"])
def test_bad_ids_and_lengths_are_flagged(m, fmt):
    """And the other request's rows are right all the same."""
    c = Case(fmt, [300, 200], 4, 16, "tree", [4, 3], seed=80)
    good = c.run(m)
    assert m.mla_get_device_error() == 0
    keep, lens, nodes = c.bt.copy(), c.lens.copy(), c.tree_lens.copy()
    c.bt[0, 1] = c.nb
    got = c.run(m)
    assert m.mla_get_device_error() == 1
    assert torch.equal(got[0][1], good[0][1]) and torch.equal(got[1][1], good[1][1])
    c.bt = keep
    c.lens[0] = c.bt.shape[1] * 64 + 1
    got = c.run(m)
    assert m.mla_get_device_error() & 2 and torch.equal(got[0][1], good[0][1])
    c.lens = lens
    for bad in (-1, 5, -2 ** 31):
        c.tree_lens[0] = bad
        for split in (0, 2):
            got = c.run(m, split_tiles=split)
            assert m.mla_get_device_error() == 2
            assert not got[0][0].any() and torch.isneginf(got[1][0]).all()
            torch.testing.assert_close(got[0][1], good[0][1], rtol=2 ** -6, atol=2 ** -6)
    c.tree_lens = nodes


def test_offsets_beyond_32_bits(m):
    """Pages behind the first 4 GiB of a bf16 cache."""
    nb = 60000
    cache = torch.zeros((nb, 64, 576), dtype=torch.bfloat16, device="cuda")
    c = Case("bf16", [200, 300], 5, 16, "tree", seed=90)
    cache[nb - c.nb:] = c.cache.cuda()
    bt = np.where((c.bt >= 0) & (c.bt < c.nb), c.bt + nb - c.nb, c.bt)
    got = m.mla_decode_paged_tree(c.q.cuda(), cache, _i32(bt), _i32(c.lens), c.mask(), sm_scale=SCALE)
    want = c.run(m)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("fmt,width", [("bf16", 0), ("bf16", WIDE), ("s32", 0)])
def test_streams_and_graphs(m, fmt, width):
    """Two calls at once on streams and workspaces of their own, and a captured
    call replayed on new lengths and masks."""
    a = Case(fmt, [900, 40, 333], 6, 32, "chain", [6, 6, 4], seed=100, width=width)
    b = Case(fmt, [64, 700], 20, 16, "tree", seed=101, width=width)
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
    q, cache, bt, lens, mask = a.q.cuda(), a.cache.cuda(), _i32(a.bt), _i32(a.lens), a.mask()
    nodes, sc = _i32(a.tree_lens), None if a.scales is None else a.scales.cuda()

    def call():
        return m.mla_decode_paged_tree(q, cache, bt, lens, mask, sm_scale=SCALE, q_scale=a.q_scale, kv_scales=sc,
                                       k_scale=a.k_scale, tree_lens=nodes)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    graph.replay()
    assert torch.equal(out, want[0][0])
    lens.copy_(_i32([500, 40, 9]))
    nodes.copy_(_i32([2, 6, 0]))
    mask[0] = torch.tensor([1, 2, 0, 0, 0, 0])
    graph.replay()
    fresh = call()
    assert torch.equal(out, fresh[0]) and torch.equal(lse, fresh[1])


def test_the_error_word_stays_clear(m):
    assert m.mla_get_device_error() == 0
