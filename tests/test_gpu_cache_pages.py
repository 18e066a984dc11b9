"""The cache-page calls against their oracle, bit for bit: the whole state and
every byte of every pool after each call."""

import numpy as np
import pytest
import torch

import synth
from oracle import pages as P, tree as T

pytestmark = pytest.mark.gpu

BITS = {"block": 1, "len": 2, "range": 4, "pages": 16}


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    mod.mla_get_device_error()
    return mod


def code(errors):
    return sum(BITS[e] for e in errors)


def _i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def raw(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy().reshape(t.shape[0], -1)


SHAPES = {
    "bf16": [((64, 576), torch.bfloat16)],
    "scaled": [((64, 576), torch.uint8), ((64, 576), torch.uint8), ((4,), torch.float32), ((1,), torch.float32)],
    # pages of 4, 20, 1020, 1024, 1040, 36880 and 81920 bytes
    "odd": [((n,), torch.int32) for n in (1, 5, 255, 256, 260, 9220, 20480)],
    "small": [((2,), torch.float32), ((3,), torch.int32)],
    # rows of 4, 20, 16, 48 and 1152 bytes, and pages of as many that are no rows
    "rows": [((64, n), torch.int32) for n in (1, 5, 4, 12, 288)] + [((32, 2 * n), torch.int32) for n in (1, 5, 4)],
}


class State:
    """Sequences over a pool of nb pages, on the device and for the oracle."""

    def __init__(self, shapes, nb, B, mb, lens=None, seed=0):
        g = self.g = synth.generator(21000 + seed)
        self.pools = [torch.from_numpy(g.integers(0, 256, (nb, int(np.prod(s)) * t.itemsize), dtype=np.uint8))
                      .view(t).view(nb, *s).cuda() for s, t in SHAPES[shapes]]
        self.by_rows = [s[0] == 64 for s, _ in SHAPES[shapes]]
        self.refs = np.zeros(nb, np.int32)
        self.table = np.full((B, mb), -1, np.int32)
        self.lens = np.zeros(B, np.int32)
        if lens is not None:
            perm = g.permutation(nb).astype(np.int32)
            self.lens[:len(lens)] = lens
            for b, n in enumerate(lens):
                k = -(-int(n) // 64)
                self.table[b, :k], perm = perm[:k], perm[k:]
                self.refs[self.table[b, :k]] = 1
        self.d = [_i32(self.refs), _i32(self.table), _i32(self.lens)]
        self.bytes = [raw(p) for p in self.pools]

    def check(self, m, errors=()):
        assert m.mla_get_device_error() == code(errors)
        for name, want, got in zip(("refs", "table", "lens"), (self.refs, self.table, self.lens), self.d):
            np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)
        for k, (want, got) in enumerate(zip(self.bytes, self.pools)):
            np.testing.assert_array_equal(raw(got), want, err_msg=f"pool {k}")

    def resize(self, m, new):
        m.mla_cache_resize(*self.d, _i32(new))
        self.check(m, P.resize(self.refs, self.table, self.lens, np.asarray(new)))

    def fork(self, m, parents, children, **kw):
        m.mla_cache_fork(self.pools, *self.d, _i32(parents), _i32(children), **kw)
        self.check(m, P.fork(self.bytes, self.refs, self.table, self.lens, parents, children, self.by_rows))

    def compact(self, m, **kw):
        live = m.mla_cache_compact(self.pools, *self.d, **kw)
        n, errors = P.compact(self.bytes, self.refs, self.table, self.lens)
        self.check(m, errors)
        assert live.tolist() == [n]

    def copy(self, m, src, dst):
        m.mla_cache_copy(self.pools, _i32(src), _i32(dst))
        self.check(m, P.copy(self.bytes, src, dst))


# ------------------------------------------------------------------- copy
@pytest.mark.parametrize("shapes", list(SHAPES))
@pytest.mark.parametrize("n", [1, 2, 7, 60, 333])
def test_copy(m, shapes, n):
    s = State(shapes, 700 if n > 60 else 130, 1, 1, seed=n)
    perm = s.g.permutation(s.refs.size)
    s.copy(m, perm[:n], perm[n:2 * n])


@pytest.mark.parametrize("shapes", ["bf16", "scaled"])
def test_copy_padding_and_refusals(m, shapes):
    s = State(shapes, 20, 1, 1)
    s.copy(m, [-1, 3, 4, -2 ** 31, 5], [2, -1, 4, -7, 6])       # padding, a page onto itself
    s.copy(m, [0, 1, 2, 1], [9, 9, 9, 8])                       # the last of equal destinations
    s.copy(m, [0, 1, 2, 3], [1, 2, 3, 4])                       # a chain: only its end
    s.copy(m, [0, 1], [1, 0])                                   # a swap: neither
    s.copy(m, [20, 3, 5, 2 ** 31 - 1], [1, 20, 6, 7])           # no pages
    s.copy(m, [5, 5, 7], [5, 6, 5])                             # one onto itself reads nothing
    s.copy(m, [3, 4, 3], [9, 3, 3])
    m.mla_cache_copy(s.pools, _i32([]), _i32([]))
    s.check(m)


def test_copy_without_large_pools_and_one_tensor(m):
    s = State("small", 40, 1, 1)
    s.copy(m, np.arange(20), np.arange(20, 40))
    p = torch.arange(6 * 64 * 576, device="cuda", dtype=torch.int32).view(6, 64, 576)
    want = p.clone()
    want[4] = want[1]
    m.mla_cache_copy(p, _i32([1]), _i32([4]))
    assert torch.equal(p, want)


def test_copy_of_the_longest_list(m):
    n = 1 << 16
    g = torch.Generator(device="cuda").manual_seed(3)
    pools = [torch.randint(1 << 30, (2 * n + 9, w), dtype=torch.int32, device="cuda", generator=g) for w in (4, 256)]
    order = torch.randperm(2 * n + 9, device="cuda", generator=g, dtype=torch.int64).int()
    src, dst = order[:n].contiguous(), order[n:2 * n].contiguous()
    want = [p.clone() for p in pools]
    for w in want:
        w[dst.long()] = w[src.long()]
    m.mla_cache_copy(pools, src, dst)
    assert m.mla_get_device_error() == 0
    assert all(torch.equal(p, w) for p, w in zip(pools, want))


def test_copy_beyond_32_bits(m):
    pool = torch.zeros((60000, 64, 576), dtype=torch.bfloat16, device="cuda")
    pool[59990] = 3.0
    pool[2] = 5.0
    m.mla_cache_copy([pool], _i32([59990, 2]), _i32([1, 59999]))
    assert bool((pool[1] == 3).all()) and bool((pool[59999] == 5).all()) and not pool[59991:59999].any()
    assert m.mla_get_device_error() == 0


# ----------------------------------------------------------------- resize
def test_resize(m):
    s = State("small", 40, 6, 9, [100, 0, 64, 65, 1, 576], seed=1)
    s.resize(m, [100, 0, 64, 65, 1, 576])             # nothing
    s.resize(m, [128, 64, 1, 200, 0, 0])              # all kinds at once
    s.resize(m, [0, 576, 576, 576, 576, 1])           # into the pages that the first gives back
    s.resize(m, [576, 576, 576, 576, 576, 576])       # more than there are: from the first that lacks some on
    s.resize(m, [576] * 6)                            # and again
    s.resize(m, [-1, 577, 2 ** 31 - 1, 0, -2 ** 31, 64])
    s.resize(m, [0] * 6)
    assert not s.refs.any()


def test_resize_of_its_own_lengths_changes_nothing(m):
    s = State("small", 40, 3, 9, [100, 0, 64], seed=2)
    m.mla_cache_resize(*s.d, s.d[2])
    s.check(m)


@pytest.mark.parametrize("nb", [1, 3, 127, 128, 129, 4097, 40003])
def test_resize_takes_the_lowest_pages(m, nb):
    """Pools of any size, some pages held elsewhere."""
    s = State("small", nb, 3, max(1, nb), seed=nb)
    s.refs[:] = s.g.integers(0, 3, nb) * (s.g.random(nb) < 0.7)
    s.d[0].copy_(_i32(s.refs))
    free = int((s.refs == 0).sum())
    s.resize(m, [64 * (free // 3), 64 * (free // 4) + 1 if free >= 4 else 0, 0])
    s.resize(m, [0, s.lens[1], 64 * int((s.refs == 0).sum()) + (64 * (free // 3))])


def test_resize_many_sequences(m):
    for B in (1, 31, 1024, 1025, 4097, 8192):
        s = State("small", 9000, B, 2, seed=B)
        s.resize(m, s.g.integers(0, 129, B) * (s.g.random(B) < 0.6))
        s.resize(m, s.g.integers(0, 129, B))
        s.resize(m, np.zeros(B, int))


def test_a_large_pool(m):
    """More pages than the kernel keeps the counts of in registers."""
    nb = 700001
    refs = torch.ones(nb, dtype=torch.int32, device="cuda")
    free = torch.tensor([5, 77, 524287, 524288, 600000, 699999, 700000], device="cuda")
    refs[free] = 0
    table, lens = torch.full((2, 8), -1, dtype=torch.int32, device="cuda"), _i32([0, 0])
    m.mla_cache_resize(refs, table, lens, _i32([5 * 64, 2 * 64]))
    assert table.tolist() == [free[:5].tolist() + [-1] * 3, free[5:].tolist() + [-1] * 6]
    assert int(refs.sum()) == nb and m.mla_get_device_error() == 0
    pool = torch.arange(nb, device="cuda", dtype=torch.int32).view(nb, 1)
    refs[:] = 0
    refs[table[0, :5].long()] = 1
    refs[table[1, :2].long()] = 2
    live = m.mla_cache_compact([pool], refs, table, lens)
    # page 5 stays, the others go to 0 .. 4 and 6
    assert live.tolist() == [7] and m.mla_get_device_error() == 0
    assert refs[:7].tolist() == [1, 1, 1, 1, 2, 1, 2] and not refs[7:].any()
    assert table[0, :5].tolist() == [5, 0, 1, 2, 3] and table[1, :2].tolist() == [4, 6]
    assert pool[:7, 0].tolist() == [77, 524287, 524288, 600000, 699999, 5, 700000]


def test_broken_tables_are_flagged(m):
    s = State("small", 12, 2, 4, [130, 70], seed=3)
    s.table[0, 1], s.table[1, 0] = 12, -3
    s.refs[s.table[1, 1]] = 0                          # held, and free
    for k, x in enumerate((s.refs, s.table)):
        s.d[k].copy_(_i32(x))
    s.resize(m, [0, 0])


# ------------------------------------------------------------------- fork
@pytest.mark.parametrize("shapes", ["bf16", "scaled", "odd", "rows"])
def test_fork(m, shapes):
    s = State(shapes, 60, 10, 6, [100, 64, 1, 320, 0, 383], seed=4)
    s.fork(m, [0, 1, 2, 4], [6, 7, 8, 9])              # partial, whole, one token, none
    s.resize(m, [100, 0, 1, 320, 0, 383, 150, 64, 0, 0])
    s.fork(m, [6, 7, 5], [1, 4, 9])                    # a fork of forks
    s.resize(m, [0] * 10)
    assert not s.refs.any()


def test_fork_refusals(m):
    s = State("scaled", 12, 8, 4, [100, 64, 30], seed=5)
    s.fork(m, [0, 2, 0, 0, 1], [1, 3, 3, 3, 4])        # a child that has tokens, one twice
    s.fork(m, [-1, 0, 8, 0, 2 ** 31 - 1], [5, -1, 5, 8, 6])
    s.fork(m, [5, 5], [6, 5])                          # empty ones
    s.fork(m, [0, 0, 0], [5, 6, 7])
    s.lens[0] = 4 * 64 + 1
    s.d[2].copy_(_i32(s.lens))
    s.resize(m, [257, 0, 30, 0, 64, 0, 0, 0])
    s.fork(m, [0], [1])
    s.lens[0] = 100
    s.d[2].copy_(_i32(s.lens))
    s.table[0, 0], s.table[2, 0] = 99, -5
    s.d[1].copy_(_i32(s.table))
    s.fork(m, [0, 2], [1, 3])


def test_fork_runs_out_of_pages(m):
    s = State("bf16", 8, 9, 3, [100, 64, 70], seed=6)
    s.fork(m, [0, 1, 2, 0, 1, 2], [3, 4, 5, 6, 7, 8])  # three pages for four: whole ones need none
    s.resize(m, [100, 64, 70, 0, 0, 0, 0, 0, 0])


def test_fork_of_many(m):
    s = State("small", 3000, 2100, 3, [100, 64, 129], seed=7)
    n = 2000
    s.fork(m, s.g.integers(0, 3, n), 3 + s.g.permutation(2097)[:n])
    s.fork(m, s.g.integers(0, 2100, 8192), s.g.integers(0, 2100, 8192))


# ---------------------------------------------------------------- compact
@pytest.mark.parametrize("shapes", list(SHAPES))
def test_compact(m, shapes):
    s = State(shapes, 150, 12, 8, [100, 64, 1, 512, 0, 383, 200, 77], seed=8)
    s.fork(m, [0, 3, 5], [8, 9, 10])
    s.compact(m)
    s.compact(m)                                       # (nothing to do)
    s.resize(m, [0, 64, 0, 512, 100, 0, 0, 77, 100, 0, 383, 1])
    s.compact(m)
    s.resize(m, [0] * 12)
    s.compact(m)                                       # nothing in use


@pytest.mark.parametrize("nb,live", [(1, 0), (1, 1), (2, 1), (5, 5), (128, 1), (129, 128), (4100, 2050),
                                     (40003, 20001)])
def test_compact_of_any_size(m, nb, live):
    s = State("small", nb, 1, max(1, nb), [64 * live], seed=nb + live)
    s.compact(m)


def test_compact_leaves_what_it_cannot_move(m):
    s = State("small", 30, 3, 6, [300, 200, 100], seed=9)
    s.refs[s.table[2, 0]] = 0                          # held, and free
    s.table[1, 1] = 30
    s.lens[0] = 400
    for k, x in enumerate((s.refs, s.table, s.lens)):
        s.d[k].copy_(_i32(x))
    s.compact(m)


@pytest.mark.parametrize("seed", range(5))
def test_any_order_of_calls(m, seed):
    s = State(["scaled", "bf16", "odd", "small", "rows"][seed], 60, 9, 7, seed=50 + seed)
    for _ in range(25):
        what = s.g.integers(0, 5)
        if what < 2:
            s.resize(m, np.where(s.g.random(9) < 0.5, s.lens, s.g.integers(0, 449, 9)))
        elif what < 4:
            n = int(s.g.integers(1, 5))
            s.fork(m, s.g.integers(0, 9, n), s.g.integers(0, 9, n))
        else:
            s.compact(m)
        held = np.concatenate([s.table[b, :-(-s.lens[b] // 64)] for b in range(9)])
        assert (np.bincount(held, minlength=60) == s.refs).all()


# ----------------------------------------------------------------- accept
def _tree_cache(g, fmt, ctx, n, layers, spare=2):
    """Caches (bits) of sequences of ctx + n tokens, scales, table and lengths."""
    lens = np.asarray(ctx, np.int32) + np.asarray(n, np.int32)
    table, nb = synth.paged_layout(g, np.maximum(lens, 1))
    caches, scales = [], None
    if fmt == "bf16":
        caches = [torch.from_numpy(g.integers(-2 ** 15, 2 ** 15, (nb, 64, 576), dtype=np.int16)).view(torch.bfloat16)
                  for _ in range(layers)]
    else:
        caches = [torch.from_numpy(g.integers(0, 256, (nb, 64, 576), dtype=np.uint8)).view(torch.float8_e4m3fn)
                  for _ in range(layers)]
        if fmt != "e4m3":
            # rows of different sizes, so that scales grow, shrink and stay
            for c in caches:
                u = c.view(torch.uint8)
                small = torch.from_numpy(g.random((nb, 64)) < 0.5)
                u[small] = (u[small] & 0x9F).where((u[small] & 0x7F) != 0x7F, 0)
            scales = [torch.from_numpy(np.exp2(g.integers(-6, 7, (nb, 64 // int(fmt[1:])))).astype(np.float32))
                      for _ in range(layers)]
    return [c.cuda() for c in caches], None if scales is None else [s.cuda() for s in scales], table, lens


def _same_codes(got, want):
    nan = (want & 0x7F) == 0x7F
    np.testing.assert_array_equal((got & 0x7F) == 0x7F, nan)
    np.testing.assert_array_equal(got[~nan], want[~nan])


def _accept(m, caches, scales, table, lens, tree_lens, q_len, path, count):
    want = [c.cpu().view(torch.int16 if c.dtype == torch.bfloat16 else torch.uint8).numpy().copy() for c in caches]
    want_s = None if scales is None else [s.cpu().numpy().copy() for s in scales]
    new, errors = P.accept(want, want_s, table, lens, tree_lens, q_len, np.asarray(path), np.asarray(count))
    got = m.mla_cache_accept(caches, _i32(table), _i32(lens), _i32(path), _i32(count), q_len,
                             tree_lens=None if tree_lens is None else _i32(tree_lens), kv_scales=scales)
    assert m.mla_get_device_error() == code(errors)
    np.testing.assert_array_equal(got.cpu().numpy(), new)
    for k, c in enumerate(caches):
        g = c.cpu().view(torch.int16 if c.dtype == torch.bfloat16 else torch.uint8).numpy()
        if scales is None:
            np.testing.assert_array_equal(g, want[k])
        else:
            np.testing.assert_array_equal(scales[k].cpu().numpy(), want_s[k])
            _same_codes(g, want[k])
    return new


FMTS = ["bf16", "e4m3", "s16", "s32", "s64"]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("layers", [1, 5])
def test_accept(m, fmt, layers):
    g = synth.generator(31000 + layers)
    q_len = 64
    ctx = [0, 1, 15, 16, 60, 63, 64, 100, 127, 128, 300]
    n = [64, 1, 64, 40, 64, 33, 64, 5, 64, 17, 64]
    caches, scales, table, lens = _tree_cache(g, fmt, ctx, n, layers)
    path, count = np.full((len(n), 64), -9), np.zeros(len(n), int)
    for b, size in enumerate(n):
        k = [64, 1, 20, 0, 3, 33, 30, 2, 64, 9, 11][b]
        path[b, :k] = np.sort(g.permutation(size)[:k])
        count[b] = k
    _accept(m, caches, scales, table, lens, n, q_len, path, count)


@pytest.mark.parametrize("fmt", ["bf16", "s16"])
def test_accept_refuses(m, fmt):
    g = synth.generator(31100)
    ctx, n = [100] * 9 + [0], [8] * 9 + [3]
    caches, scales, table, lens = _tree_cache(g, fmt, ctx, n, 2)
    path = np.array([[0, 3, 5]] * 10)
    path[0] = [3, 3, 5]
    path[1] = [3, 5, 4]
    path[2] = [-1, 3, 5]
    path[3] = [0, 3, 8]
    count = np.array([3, 3, 3, 3, 4, -1, 3, 2, 3, 1])
    nodes = np.array([8, 8, 8, 8, 8, 8, 9, 8, 8, 4])       # over q_len, before the sequence's start
    table[8, 1] = -4
    _accept(m, caches, scales, table, lens, nodes, 8, path, count)
    lens[7], count[9], nodes[9] = table.shape[1] * 64 + 1, 0, 4
    table[8, 1] = caches[0].shape[0]
    _accept(m, caches, scales, table, lens, nodes, 8, path, count)


def test_accept_of_far_scales_and_of_no_scales(m):
    """Scales at both ends of the range, zero, and what is none."""
    g = synth.generator(31200)
    caches, scales, table, lens = _tree_cache(g, "s16", [20, 33, 5, 16], [30] * 4, 1)
    s = scales[0].view(-1)
    vals = [0.0, 2.0 ** -100, 2.0 ** 120, float("nan"), -1.0, float("inf"), 2.0 ** -126, 3.0, 1.0]
    s.copy_(torch.tensor([vals[int(i)] for i in g.integers(0, len(vals), s.numel())]))
    path = np.stack([np.sort(g.permutation(30)[:12]) for _ in range(4)])
    _accept(m, caches, scales, table, lens, None, 30, path, np.full(4, 12))


@pytest.mark.parametrize("fmt", ["bf16", "s32"])
def test_accept_many_layers_and_requests(m, fmt):
    g = synth.generator(31300)
    B, q_len = 90, 12
    caches, scales, table, lens = _tree_cache(g, fmt, g.integers(0, 200, B), [q_len] * B, 40)
    path, count = np.zeros((B, 7), int), g.integers(0, 8, B)
    for b in range(B):
        path[b, :count[b]] = np.sort(g.permutation(q_len)[:count[b]])
    _accept(m, caches, scales, table, lens, None, q_len, path, count)


def test_no_pools(m):
    s = State("small", 20, 4, 3, [100, 64], seed=11)
    s.pools, s.bytes = [], []
    s.fork(m, [0, 1], [2, 3])
    s.resize(m, [0, 64, 100, 64])
    s.compact(m)
    new = m.mla_cache_accept([], s.d[1], s.d[2], _i32([[1]] * 4), _i32([1, 1, 1, 0]), 2)
    assert m.mla_get_device_error() == 4 and new.tolist() == [0, 63, 99, 64 - 2]


# ------------------------------------------------- streams, graphs, a step
def test_captured_calls_on_a_stream(m):
    """A captured resize, fork, compact and accept, replayed on new state."""
    s = State("scaled", 60, 6, 6, [100, 64, 200], seed=12)
    new, parents, children = _i32([150, 64, 200, 0, 0, 0]), _i32([0, 2]), _i32([3, 4])
    ws = [torch.zeros(4096, dtype=torch.uint8, device="cuda") for _ in range(2)]
    live = _i32([0])

    def calls():
        m.mla_cache_resize(*s.d, new)
        m.mla_cache_fork(s.pools, *s.d, parents, children, workspace=ws[0])
        m.mla_cache_compact(s.pools, *s.d, n_live=live, workspace=ws[1])

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            calls()
        for step in range(4):
            want = [300, 64, 10, 0, 0, 0] if step else [150, 64, 200, 0, 0, 0]
            new.copy_(_i32(want))
            graph.replay()
            stream.synchronize()
            errors = P.resize(s.refs, s.table, s.lens, np.array(want))
            errors |= P.fork(s.bytes, s.refs, s.table, s.lens, [0, 2], [3, 4], s.by_rows)
            n, more = P.compact(s.bytes, s.refs, s.table, s.lens)
            s.check(m, errors | more)
            assert live.tolist() == [n]


@pytest.mark.parametrize("fmt", ["bf16", "s32"])
def test_speculative_steps(m, fmt):
    """Serving steps: prompts forked, room for a tree made, the drafted rows
    appended, attended to, the accepted ones kept, the rest released, the pool
    compacted; a chain's decode over what is left equals one over a cache
    where those rows were appended at once."""
    g = synth.generator(41000)
    layers, nb, B, mb, H, q_len = 2, 40, 4, 6, 16, 7
    bf = torch.bfloat16

    def fresh():
        if fmt == "bf16":
            return [torch.zeros((nb, 64, 576), dtype=bf, device="cuda") for _ in range(layers)], None
        return ([torch.zeros((nb, 64, 576), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                 for _ in range(layers)], [torch.zeros((nb, 2), device="cuda") for _ in range(layers)])

    def append(pools, scales, rows, pos, slots):
        for layer in range(layers):
            kv = rows[layer]
            k = kv[:, 512:].clone()
            if fmt == "bf16":
                m.mla_rope_cache_write(None, k, kv[:, :512].contiguous(), pos, slots, pools[layer])
            else:
                m.mla_rope_cache_append(None, k, kv[:, :512], pos, slots, pools[layer], scales[layer])

    def slots_of(table, b, pos):
        return [int(table[b, p // 64]) * 64 + p % 64 for p in pos]

    def some(n):
        return [torch.from_numpy(g.standard_normal((n, 576), dtype=np.float32)).to(bf).cuda() for _ in range(layers)]

    pools, scales = fresh()
    every = pools + (scales or [])
    refs, table, lens = _i32(np.zeros(nb)), _i32(np.full((B, mb), -1)), _i32(np.zeros(B))
    seqs = (refs, table, lens)
    kept = [[] for _ in range(B)]                # (position, row of each layer) of every sequence's tokens
    ctx = [70, 128, 0, 0]
    m.mla_cache_resize(*seqs, _i32(ctx))
    t = table.cpu().numpy()
    for b in (0, 1):
        rows = some(ctx[b])
        append(pools, scales, rows, _i32(np.arange(ctx[b])), _i32(slots_of(t, b, range(ctx[b]))))
        kept[b] = [(p, [r[p] for r in rows]) for p in range(ctx[b])]
    m.mla_cache_fork(every, *seqs, _i32([0, 1]), _i32([2, 3]))
    kept[2], kept[3] = list(kept[0]), list(kept[1])
    ctx[2:] = ctx[:2]
    parents = [-1, 0, 0, 1, 1, 2, 4]
    depth = [0, 1, 1, 2, 2, 2, 3]
    path = np.array([[0, 1, 4, 6], [0, 2, 5, -1], [0, -1, -1, -1], [0, 1, 3, -1]])
    count = np.array([4, 3, 1, 3])
    words = torch.from_numpy(T.words(parents).view(np.int64)).cuda()
    for step in range(3):
        m.mla_cache_resize(*seqs, _i32([c + q_len for c in ctx]))
        t = table.cpu().numpy()
        rows = some(B * q_len)
        pos = [ctx[b] + d for b in range(B) for d in depth]
        slots = [x for b in range(B) for x in slots_of(t, b, range(ctx[b], ctx[b] + q_len))]
        append(pools, scales, rows, _i32(pos), _i32(slots))
        q = torch.from_numpy(g.standard_normal((B, q_len, H, 576), dtype=np.float32)).cuda()
        q = q.to(bf) if fmt == "bf16" else (q / 0.02).to(torch.float8_e4m3fn)      # (far from 448)
        kw = dict(sm_scale=0.05, q_scale=0.02)
        out = [m.mla_decode_paged_tree(q, pools[n], table, lens, words, kv_scales=scales and scales[n], **kw)
               for n in range(layers)]
        new = m.mla_cache_accept(pools, table, lens, _i32(path), _i32(count), q_len, kv_scales=scales)
        m.mla_cache_resize(*seqs, new)
        live = m.mla_cache_compact(every, *seqs)
        # the same tokens, appended at once to a cache of its own
        for b in range(B):
            kept[b] += [(ctx[b] + depth[i], [r[b * q_len + i] for r in rows]) for i in path[b, :count[b]]]
            ctx[b] += int(count[b])
        assert lens.tolist() == ctx
        t = table.cpu().numpy()
        assert live.item() == len({int(x) for b in range(B) for x in t[b, :-(-ctx[b] // 64)]})
        plain, plain_s = fresh()
        for b in range(B):
            slots = [mb * 64 * b + p for p in range(ctx[b])]
            append(plain, plain_s, [torch.stack([r[n] for _, r in kept[b]]) for n in range(layers)],
                   _i32([p for p, _ in kept[b]]), _i32(slots))
        straight = _i32(np.arange(B * mb).reshape(B, mb))
        last = torch.as_tensor(path[np.arange(B), count - 1], device="cuda")
        every_b = torch.arange(B, device="cuda")
        one = q[every_b, last][:, None].contiguous()      # the queries of the paths' last nodes
        for n in range(layers):
            node = out[n][0][every_b, last].float()
            if fmt == "bf16":
                got = m.mla_decode_paged_window(one, pools[n], table, lens, sm_scale=0.05, window=0)
                want = m.mla_decode_paged_window(one, plain[n], straight, lens, sm_scale=0.05, window=0)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
                far = 2.0 ** -6           # (2^-7 of the values from either's probabilities, and both roundings)
            else:
                got = m.mla_decode_paged_scaled(one, pools[n], scales[n], table, lens, **kw)
                want = m.mla_decode_paged_scaled(one, plain[n], plain_s[n], straight, lens, **kw)
                # a code that took another scale on the way is off by a second rounding of at most 2^-4
                far = 2.0 ** -3
                assert float((got[0].float() - want[0].float()).abs().max()) <= far * 5
            # the tree's row of that node saw the same tokens (values of up to 5)
            assert float((got[0][:, 0].float() - node).abs().max()) <= far * 5
            assert float((got[1][:, 0] - out[n][1][every_b, last]).abs().max()) <= far
    assert m.mla_get_device_error() == 0
    m.mla_cache_resize(*seqs, _i32([0] * B))
    assert not refs.any()
