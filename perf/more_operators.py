"""Cases of the tree-attention and cache-page operators, with their plain forms.

What a serving loop with speculative trees and shared sequences does around and over the paged
latent cache:

tree      absorbed decode attention of a tree of drafted tokens, over a bf16, an e4m3 or a
          block-scaled e4m3 cache
accept    the rows of the drafted tokens that were accepted, moved together behind the context,
          in every layer's cache
copy      pages copied in every layer's cache
fork      sequences that go on from others': shared pages are counted, the last one is copied;
          the sequences of the step before are freed first
compact   finished sequences are freed, the pages in use move to the front of the pool in every
          layer's cache, and new sequences take the pages behind them

``own`` selects the library's calls; otherwise ``run`` computes the same with elementary torch
operations.  ``exact`` states the attention again, in 64 bits, request by request; the others move
bits, but for the block-scaled accept, which it states row by row.
"""

import math

import numpy as np
import torch

own = False

PAGE, LAT, DQK = 64, 512, 576
SM_SCALE = 1.0 / math.sqrt(192.0)
E4M3_MAX = 448.0
MIN_EXP = -100           # the smallest scale is 2^-100


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one chat on one shard of the heads, a small tree: latency counts
        dict(name="tree tiny", op="tree", requests=1, q_len=8, heads=16, shape="even", context=300,
             kv="bf16", ragged=False, lengths=1),
        # a serving batch: a tree of 16 tokens for each of 16 requests
        dict(name="tree batch", op="tree", requests=16, q_len=16, heads=128, shape="even",
             context=4096, kv="bf16", ragged=False, lengths=2),
        # trees of different sizes at mixed lengths, an odd number of heads, an e4m3 cache
        dict(name="tree ragged", op="tree", requests=8, q_len=33, heads=20, shape="uniform",
             context=8192, kv="e4m3", ragged=True, lengths=3),
        # a wide tree behind one long document, block scales
        dict(name="tree long", op="tree", requests=1, q_len=64, heads=128, shape="even",
             context=16384, kv="s64", ragged=False, lengths=4),
        # the accepted path of one chat's tree, one layer's cache
        dict(name="accept one", op="accept", requests=1, q_len=8, context=300, kv="bf16", layers=1,
             lengths=5),
        # every request of a batch, all layers of a model part at once
        dict(name="accept layers", op="accept", requests=32, q_len=16, context=700, kv="bf16",
             layers=30, lengths=6),
        # the same over a block-scaled cache: rows change their scales
        dict(name="accept scaled", op="accept", requests=16, q_len=33, context=500, kv="s16",
             layers=8, lengths=7),
        # a few pages in a few layers
        dict(name="copy few", op="copy", pages=6, kv="bf16", layers=4, pool=96, lengths=8),
        # a long document's pages, e4m3
        dict(name="copy document", op="copy", pages=500, kv="e4m3", layers=12, pool=1200, lengths=9),
        # beams of one request
        dict(name="fork beams", op="fork", parents=2, children=5, context=1000, kv="e4m3", layers=2,
             pool=80, lengths=10),
        # parallel samples of several requests, many layers
        dict(name="fork samples", op="fork", parents=8, children=64, context=8192, kv="bf16",
             layers=10, pool=1500, lengths=11),
        # half of a batch has finished
        dict(name="compact batch", op="compact", requests=48, context=2048, kv="bf16", layers=4,
             spare=40, lengths=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "accept", "accept", "copy", "fork", "compact"])
    c = dict(op=op, lengths=rng.randrange(1, 1 << 20))
    if op == "tree":
        c["q_len"] = _log(rng, 1, 64)
        c["heads"] = rng.choice([8, 16, 20, 64, 128])
        c["context"] = _log(rng, 16, 32768)
        most = (1 << 27) // (c["q_len"] * c["heads"] * (c["context"] + c["q_len"]))
        if most < 1:
            c["context"], most = (1 << 27) // (c["q_len"] * c["heads"]) - c["q_len"], 1
        c["requests"] = _log(rng, 1, min(64, most, max(1, 262144 // c["context"])))
        c["shape"] = rng.choice(["even", "uniform", "lognormal"])
        c["kv"] = rng.choice(["bf16", "bf16", "e4m3", "s16", "s32", "s64"])
        c["ragged"] = rng.random() < 0.5
    elif op == "accept":
        c["q_len"] = _log(rng, 2, 64)
        c["layers"] = _log(rng, 1, 32)
        c["context"] = _log(rng, 16, 900)
        c["requests"] = _log(rng, 1, max(1, min(64, 16384 // (c["layers"] * (c["context"] // PAGE + 2)))))
        c["kv"] = rng.choice(["bf16", "e4m3", "s16", "s32", "s64"])
    elif op == "copy":
        c["layers"] = _log(rng, 1, 32)
        c["pages"] = _log(rng, 1, 6000 // c["layers"])
        c["pool"] = 2 * c["pages"] + rng.randint(3, 99)
        c["kv"] = rng.choice(["bf16", "e4m3", "s16", "s64"])
    elif op == "fork":
        c["layers"] = _log(rng, 1, 16)
        c["parents"] = _log(rng, 1, 16)
        c["children"] = _log(rng, 1, 64)
        c["context"] = _log(rng, 16, 8192)
        c["pool"] = c["parents"] * (c["context"] // PAGE + 1) + c["children"] + rng.randint(0, 50)
        c["pool"] = max(c["pool"], 8)
        c["kv"] = rng.choice(["bf16", "e4m3", "s32"])
    else:
        c["layers"] = _log(rng, 1, 12)
        c["requests"] = _log(rng, 2, 64)
        c["context"] = _log(rng, 64, max(65, min(4096, 380000 // (c["layers"] * c["requests"]))))
        c["spare"] = rng.randint(0, 60)
        c["kv"] = rng.choice(["bf16", "e4m3", "s32"])
    return c


def _lens(case, n):
    """Context lengths of n requests, fixed by the case."""
    r = np.random.RandomState(case["lengths"])
    top, shape = case["context"], case.get("shape", "uniform")
    if shape == "even":
        lens = np.maximum(1, top - r.randint(0, max(1, top // 16), n))
        lens[0] = top
    elif shape == "uniform":
        lens = r.randint(max(1, top // 4), top + 1, n)
    else:
        lens = np.clip(np.exp(r.normal(math.log(max(2, top // 16)), 1.0, n)), 1, top)
    return lens.astype(np.int64)


def _tree_lens(case):
    """Drafted tokens of each request."""
    n, q_len = case["requests"], case["q_len"]
    if not case["ragged"]:
        return np.full(n, q_len, np.int64)
    r = np.random.RandomState(case["lengths"] + 1)
    got = r.randint((q_len + 1) // 2, q_len + 1, n)
    got[0] = q_len
    return got.astype(np.int64)


def _parents(r, n):
    """A drafted tree: node 0 is its root, most nodes hang from a late one."""
    parent = np.full(n, -1, np.int64)
    for i in range(1, n):
        parent[i] = max(0, i - 1 - min(int(r.exponential(3.0)), i - 1))
    return parent


def _masks(case):
    """Per request and node a word whose bit t says that node t is the node or above it."""
    r = np.random.RandomState(case["lengths"] + 2)
    words = np.zeros((case["requests"], case["q_len"]), np.uint64)
    for b, n in enumerate(_tree_lens(case)):
        parent = _parents(r, int(n))
        for i in range(int(n)):
            above = words[b, parent[i]] if parent[i] >= 0 else np.uint64(0)
            words[b, i] = above | (np.uint64(1) << np.uint64(i))
    return words


def _paths(case):
    """The accepted nodes of each request, ascending, and how many there are."""
    r = np.random.RandomState(case["lengths"] + 3)
    n, q_len = case["requests"], case["q_len"]
    path, count = np.full((n, q_len), -1, np.int64), np.zeros(n, np.int64)
    for b in range(n):
        parent, i, nodes = _parents(r, q_len), int(r.randint(q_len // 2, q_len)), []
        while i >= 0:
            nodes.append(i)
            i = int(parent[i])
        count[b] = len(nodes)
        path[b, :len(nodes)] = nodes[::-1]
    return path, count


def _size(kv):
    return 2 if kv == "bf16" else 1


def _scale_block(kv):
    return int(kv[1:]) if kv.startswith("s") else 0


def _page_bytes(kv):
    sb = _scale_block(kv)
    return PAGE * DQK * _size(kv) + (4 * PAGE // sb if sb else 0)


def work(case):
    op, kv = case["op"], case["kv"]
    row, sb = DQK * _size(kv), _scale_block(kv)
    if op == "tree":
        ctx, nodes, H = _lens(case, case["requests"]), _tree_lens(case), case["heads"]
        seen = sum(bin(int(w)).count("1") for w in _masks(case).reshape(-1))
        pairs = int((ctx * nodes).sum()) + seen
        keys, rows = int((ctx + nodes).sum()), int(nodes.sum()) * H
        every = case["requests"] * case["q_len"]
        return {"bytes": keys * row + (4 * -(-keys // sb) if sb else 0) + rows * row + every * H * (LAT * 2 + 4) +
                8 * every + 4 * -(-keys // PAGE),
                "flops": 2.0 * H * pairs * (DQK + LAT)}
    if op == "accept":
        path, count = _paths(case)
        moved = int(((path != np.arange(path.shape[1])) & (path >= 0)).sum())
        return {"bytes": case["layers"] * moved * row * 2 + 4 * int(count.sum()) + 16 * len(count), "flops": 0}
    if op == "copy":
        return {"bytes": 2.0 * case["pages"] * case["layers"] * _page_bytes(kv), "flops": 0}
    if op == "fork":
        lens = _lens(case, case["parents"])[_fork_from(case)]
        rows = int((lens % PAGE).sum())
        return {"bytes": 2.0 * rows * case["layers"] * row + 24 * int((lens // PAGE + 1).sum()) + 4 * case["pool"],
                "flops": 0}
    pages = -(-_lens(case, case["requests"]) // PAGE)
    moved = min(int(pages[0::2].sum()), int(pages[1::2].sum()))
    total = int(pages.sum())
    return {"bytes": 2.0 * moved * case["layers"] * _page_bytes(kv) + 24 * total, "flops": 0}


# ----------------------------------------------------------------- inputs
def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


def _table(pages, width, r, spare=3):
    """Shuffled pages: (block table [B, width], pages of the pool)."""
    total = int(np.sum(pages)) + spare
    perm = r.permutation(total).astype(np.int32)
    bt = np.full((len(pages), max(1, width)), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = perm[at:at + n]
        at += int(n)
    return bt, total


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, at least MIN_EXP."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _layers(kv, layers, pages, gen):
    """(caches [layers, pages, 64, 576], scales [layers, pages, 64 / sb] or None, k_scale): normal
    rows, under block scales of a size that wanders from block to block."""
    sb = _scale_block(kv)
    if kv == "bf16":
        return torch.randn((layers, pages, PAGE, DQK), generator=gen, device="cuda", dtype=torch.bfloat16), None, 1.0
    caches = torch.empty((layers, pages, PAGE, DQK), device="cuda", dtype=torch.float8_e4m3fn)
    scales = torch.empty((layers, pages, PAGE // sb), device="cuda") if sb else None
    k_scale = 1.0 if sb else 1.0 / 64
    for n in range(layers):
        x = torch.randn((pages, PAGE, DQK), generator=gen, device="cuda")
        if not sb:
            caches[n] = (x / k_scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            continue
        x = x.view(pages, PAGE // sb, sb, DQK)
        x *= torch.exp2(torch.rand((pages, PAGE // sb, 1, 1), generator=gen, device="cuda") * 4.0 - 3.0)
        s = _pow2(_exponent(x.abs().amax(dim=(2, 3))))
        caches[n] = (x / s[..., None, None]).view(pages, PAGE, DQK).to(torch.float8_e4m3fn)
        scales[n] = s
    return caches, scales, k_scale


def _fork_from(case):
    """The parent of each child."""
    return np.random.RandomState(case["lengths"] + 4).randint(0, case["parents"], case["children"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    r = np.random.RandomState((int(seed) * 31 + case["lengths"]) % (1 << 31))
    op, kv = case["op"], case["kv"]
    st = {"case": case, "turn": 0}
    if op == "tree":
        ctx, nodes = _lens(case, case["requests"]), _tree_lens(case)
        lens = ctx + nodes
        pages = -(-lens // PAGE)
        bt, total = _table(pages, int(pages.max()), r)
        caches, scales, st["k_scale"] = _layers(kv, 1, total, gen)
        st["cache"], st["scales"] = caches[0], None if scales is None else scales[0]
        q = torch.randn((case["requests"], case["q_len"], case["heads"], DQK), generator=gen, device="cuda")
        st["q_scale"] = 1.0 if kv == "bf16" else float(q.abs().max()) / E4M3_MAX * 1.001
        st["q"] = q.to(torch.bfloat16) if kv == "bf16" else (q / st["q_scale"]).to(torch.float8_e4m3fn)
        st["mask"] = torch.as_tensor(_masks(case).view(np.int64), device="cuda")
        st["table"], st["lens"] = _i32(bt), _i32(lens)
        st["nodes"] = _i32(nodes) if case["ragged"] else None
        return st
    if op == "copy":
        caches, scales, _ = _layers(kv, case["layers"], case["pool"], gen)
        perm = r.permutation(case["pool"])
        st["src"], st["dst"] = _i32(perm[:case["pages"]]), _i32(perm[case["pages"]:2 * case["pages"]])
    elif op == "accept":
        ctx = _lens(case, case["requests"])
        lens = ctx + case["q_len"]
        pages = -(-lens // PAGE)
        bt, total = _table(pages, int(pages.max()), r)
        caches, scales, _ = _layers(kv, case["layers"], total, gen)
        path, count = _paths(case)
        st["table"], st["lens"] = _i32(bt), _i32(lens)
        st["path"], st["count"] = _i32(path), _i32(count)
        st["new_lens"] = torch.empty_like(st["lens"])
    elif op == "fork":
        lens = np.concatenate([_lens(case, case["parents"]), np.zeros(case["children"], np.int64)])
        pages = -(-lens // PAGE)
        bt, total = _table(pages, int(pages.max()), r, max(0, case["pool"] - int(pages.sum())))
        caches, scales, _ = _layers(kv, case["layers"], total, gen)
        st["table"], st["lens"], st["freed"] = _i32(bt), _i32(lens), _i32(lens)
        st["refs"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        st["refs"][torch.as_tensor(bt[bt >= 0], device="cuda").long()] = 1
        st["from"] = _i32(_fork_from(case))
        st["to"] = _i32(case["parents"] + np.arange(case["children"]))
    else:
        lens = _lens(case, case["requests"])
        pages = -(-lens // PAGE)
        bt, total = _table(pages, int(pages.max()), r, case["spare"])
        caches, scales, _ = _layers(kv, case["layers"], total, gen)
        st["table"], st["lens"], st["full"] = _i32(bt), _i32(lens), _i32(lens)
        st["refs"] = torch.zeros(total, dtype=torch.int32, device="cuda")
        st["refs"][torch.as_tensor(bt[bt >= 0], device="cuda").long()] = 1
        which = np.arange(case["requests"]) % 2
        st["staying"] = [_i32(np.where(which == k, lens, 0)) for k in (0, 1)]   # in turn
    st["caches"], st["scales"] = caches, scales
    # what a program has of each layer
    st["layers"] = list(caches)
    st["layer_scales"] = None if scales is None else list(scales)
    st["pools"] = st["layers"] + (st["layer_scales"] or [])
    return st


# ------------------------------------------------------------ plain forms
def _u8(x):
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x


def _plain_tree(st):
    case = st["case"]
    q, table, lens = st["q"], st["table"].long(), st["lens"].long()
    B, q_len, H, _ = q.shape
    nodes = torch.full_like(lens, q_len) if st["nodes"] is None else st["nodes"].long()
    ctx = lens - nodes
    j = torch.arange(table.shape[1] * PAGE, device="cuda")
    at = j - ctx[:, None]                                                    # [B, n]: node of key j
    bit = torch.bitwise_right_shift(st["mask"][:, :, None], at.clamp(0, 63)[:, None, :]) & 1
    see = (at < 0)[:, None, :] | ((bit != 0) & ((at >= 0) & (at < nodes[:, None]))[:, None, :])
    see = see & (torch.arange(q_len, device="cuda") < nodes[:, None])[..., None]          # [B, q_len, n]
    rows = (table[:, j // PAGE] * PAGE + j % PAGE).clamp(min=0)
    if st["scales"] is not None:
        kv = _values(st["cache"], st["scales"], rows)
    else:
        kv = st["cache"].view(torch.uint8).view(-1, DQK * st["cache"].element_size())[rows]
        kv = kv.view(st["cache"].dtype).float() * st["k_scale"]
    kv = torch.where((j < lens[:, None])[..., None], kv, torch.zeros((), device="cuda"))
    qf = (q.float() * st["q_scale"]).view(B, q_len * H, DQK)
    s = torch.matmul(qf, kv.transpose(1, 2)).view(B, q_len, H, -1) * SM_SCALE
    s = s.masked_fill(~see[:, :, None, :], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - m.clamp(min=-1e30))
    z = e.sum(dim=-1, keepdim=True)
    e = e / torch.where(z > 0, z, torch.ones_like(z))
    out = torch.matmul(e.view(B, q_len * H, -1), kv[..., :LAT]).view(B, q_len, H, LAT)
    return {"out": out.to(torch.bfloat16), "lse": (m + torch.log(z))[..., 0]}


def _values(cache, scales, rows):
    """Values of the flat cache rows `rows` of a block-scaled cache, in 32 bits."""
    x = cache.view(torch.uint8).view(-1, DQK)[rows].view(torch.float8_e4m3fn).float()
    return x * scales.reshape(-1)[rows // (PAGE // scales.shape[-1])][..., None]


def _moves(st):
    """Slots [B, P] that the accepted rows come from and go to, and the place in the path (behind a
    path's end all is said of its first row again, so that equal places are written alike)."""
    table, path = st["table"].long(), st["path"].long()
    base = st["lens"].long() - st["case"]["q_len"]
    i = torch.arange(path.shape[1], device="cuda")
    i = torch.where(i < st["count"][:, None], i, 0)

    def slot(pos):
        return table.gather(1, pos // PAGE) * PAGE + pos % PAGE

    return slot(base[:, None] + path.gather(1, i)), slot(base[:, None] + i), i, base


def _plain_accept(st):
    sb = _scale_block(st["case"]["kv"])
    src, dst, i, base = _moves(st)
    st["new_lens"].copy_(base + st["count"])
    if not sb:
        flat = _u8(st["caches"]).flatten(1, 2)
        flat[:, dst] = flat[:, src]
        return _outputs(st, {"lens": st["new_lens"]})
    # the blocks [B, n] that rows go to, from the first one on (behind the last one the first again)
    which = (base[:, None] + i) // sb - (base // sb)[:, None]
    t = torch.arange((i.shape[1] - 1) // sb + 2, device="cuda")
    t = torch.where(t <= which.amax(dim=1, keepdim=True), t, 0)
    at = ((base // sb)[:, None] + t) * sb
    block = st["table"].long().gather(1, at // PAGE) * (PAGE // sb) + at % PAGE // sb
    fresh = at >= base[:, None]
    every = block[..., None] * sb + torch.arange(sb, device="cuda")
    for cache, scales in zip(st["layers"], st["layer_scales"]):
        codes, flat = cache.view(torch.uint8).view(-1, DQK), scales.view(-1)
        rows = _values(cache, scales, src)                                   # [B, P, 576]
        amax = torch.zeros(t.shape, device="cuda").scatter_reduce(1, which, rows.abs().amax(dim=-1), "amax")
        amax = amax.gather(1, t)
        old = torch.where(fresh, torch.zeros_like(amax), flat[block])
        new = torch.maximum(old, _pow2(_exponent(amax)))
        # the rows that stay follow a scale that grew
        kept = codes[every]
        moved = (kept.view(torch.float8_e4m3fn).float() * (old / new)[..., None, None]).to(torch.float8_e4m3fn)
        grew = (old > 0) & (new > old)
        codes[every] = torch.where(grew[..., None, None], moved.view(torch.uint8), kept)
        flat[block] = new
        codes[dst] = (rows / new.gather(1, which)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return _outputs(st, {"lens": st["new_lens"]})


def _outputs(st, more):
    """The caches (16-bit values as whole numbers: their bits move) and what else there is."""
    if st["scales"] is not None:
        more["scales"] = st["scales"]
    caches = st["caches"]
    return {"caches": caches.view(torch.int16) if caches.dtype == torch.bfloat16 else caches, **more}


def _plain_copy(st):
    src, dst = st["src"].long(), st["dst"].long()
    for pool in st["pools"]:
        pool = _u8(pool)
        pool[dst] = pool[src]
    return _outputs(st, {})


def _plain_resize(refs, table, lens, new):
    """Every sequence to its new length: pages behind it go, then missing ones come, the lowest
    first, to the sequences in their order as long as there are any."""
    col = torch.arange(table.shape[1], device="cuda")
    had, need = (lens + PAGE - 1) // PAGE, (new + PAGE - 1) // PAGE
    drop = (col >= need[:, None]) & (col < had[:, None])
    refs.index_add_(0, torch.where(drop, table, 0).view(-1), -drop.int().view(-1))
    table.masked_fill_(drop, -1)
    more = (need - had).clamp(min=0)
    end, free = torch.cumsum(more, 0), torch.cumsum(refs == 0, 0)
    got = end <= free[-1]
    grow = (col >= had[:, None]) & (col < need[:, None]) & got[:, None]
    page = torch.searchsorted(free, (end - more - had)[:, None] + col + 1).int()
    page = torch.where(grow, page, 0)
    refs.index_add_(0, page.view(-1), grow.int().view(-1))
    table.copy_(torch.where(grow, page, table))
    lens.copy_(torch.where(got | (more == 0), new, lens))


def _plain_fork(st):
    refs, table, lens = st["refs"], st["table"], st["lens"]
    _plain_resize(refs, table, lens, st["freed"])
    p, c = st["from"].long(), st["to"].long()
    n, col = lens[p], torch.arange(table.shape[1], device="cuda")
    full, part = n // PAGE, n % PAGE
    end, free = torch.cumsum(part > 0, 0), torch.cumsum(refs == 0, 0)
    ok = (part == 0) | (end <= free[-1])
    of = table[p]
    share = (col < full[:, None]) & ok[:, None]
    own_page = (col == full[:, None]) & (ok & (part > 0))[:, None]
    page = torch.searchsorted(free, end).int()
    refs.index_add_(0, torch.where(share, of, 0).view(-1), share.int().view(-1))
    got = torch.where(share, of, torch.where(own_page, page[:, None], -1))
    refs.index_add_(0, torch.where(own_page, page[:, None], 0).view(-1), own_page.int().view(-1))
    table[c] = got
    lens[c] = torch.where(ok, n, lens[c])
    # the tokens of the last page, where there is one of its own; elsewhere a page onto itself
    src = of.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].clamp(min=0).long()
    some = ok & (part > 0)
    dst = torch.where(some, page.clamp(max=refs.shape[0] - 1).long(), src)
    rows = (torch.arange(PAGE, device="cuda") < part[:, None])[..., None]
    for pool in st["layers"]:
        pool = _u8(pool)
        pool[dst] = torch.where(rows & some[:, None, None], pool[src], pool[dst])
    for pool in st["layer_scales"] or []:
        pool[dst] = pool[src]
    return _outputs(st, {"refs": refs, "table": table, "lens": lens})


def _plain_compact(st):
    refs, table, lens = st["refs"], st["table"], st["lens"]
    _plain_resize(refs, table, lens, st["staying"][st["turn"]])
    live = refs > 0
    count = live.sum(dtype=torch.int32)
    page = torch.arange(refs.shape[0], device="cuda")
    high, low = live & (page >= count), ~live & (page < count)
    from_, to = torch.cumsum(high, 0), torch.cumsum(low, 0)
    # pairs of pages, behind the last one a page onto itself
    k = torch.arange(1, refs.shape[0] // 2 + 1, device="cuda")
    some, last = k <= from_[-1], refs.shape[0] - 1
    src = torch.where(some, torch.searchsorted(from_, k), last)
    dst = torch.where(some, torch.searchsorted(to, k), last)
    for pool in st["pools"]:
        pool = _u8(pool)
        pool[dst] = pool[src]
    now = torch.where(high, torch.searchsorted(to, from_), page).int()
    table.copy_(torch.where(table >= 0, now[table.clamp(min=0).long()], table))
    moved = torch.searchsorted(from_, to).clamp(max=last)
    refs.copy_(torch.where(low, refs[moved], torch.where(high, 0, refs)))
    _plain_resize(refs, table, lens, st["full"])
    return _outputs(st, {"refs": refs, "table": table, "lens": lens, "live": count.view(1)})


# ---------------------------------------------------------- the library's
def _own_call(st):
    import mla_latent_kv_uk_gb300 as mla

    case = st["case"]
    op = case["op"]
    if op == "tree":
        out, lse = mla.mla_decode_paged_tree(st["q"], st["cache"], st["table"], st["lens"], st["mask"],
                                             sm_scale=SM_SCALE, tree_lens=st["nodes"], kv_scales=st["scales"],
                                             q_scale=st["q_scale"], k_scale=st["k_scale"])
        return {"out": out, "lse": lse}
    if op == "accept":
        mla.mla_cache_accept(st["layers"], st["table"], st["lens"], st["path"], st["count"], case["q_len"],
                             kv_scales=st["layer_scales"], new_lens=st["new_lens"])
        return _outputs(st, {"lens": st["new_lens"]})
    if op == "copy":
        mla.mla_cache_copy(st["pools"], st["src"], st["dst"])
        return _outputs(st, {})
    seqs = st["refs"], st["table"], st["lens"]
    more = {"refs": st["refs"], "table": st["table"], "lens": st["lens"]}
    if op == "fork":
        mla.mla_cache_resize(*seqs, st["freed"])
        mla.mla_cache_fork(st["pools"], *seqs, st["from"], st["to"])
    else:
        mla.mla_cache_resize(*seqs, st["staying"][st["turn"]])
        more["live"] = mla.mla_cache_compact(st["pools"], *seqs)
        mla.mla_cache_resize(*seqs, st["full"])
    return _outputs(st, more)


PLAIN = {"tree": _plain_tree, "accept": _plain_accept, "copy": _plain_copy, "fork": _plain_fork,
         "compact": _plain_compact}


def run(state):
    got = _own_call(state) if own else PLAIN[state["case"]["op"]](state)
    state["turn"] ^= 1
    return got


# -------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    if case["op"] == "accept" and _scale_block(case["kv"]):
        return _exact_accept(prepare(case, seed))
    if case["op"] != "tree":
        return None
    st = prepare(case, seed)
    B, q_len, H = case["requests"], case["q_len"], case["heads"]
    out = torch.zeros((B, q_len, H, LAT), dtype=torch.float64, device="cuda")
    lse = torch.full((B, q_len, H), -math.inf, dtype=torch.float64, device="cuda")
    words, nodes, lens = _masks(case), _tree_lens(case), st["lens"].tolist()
    for b in range(B):
        n, ctx = int(nodes[b]), lens[b] - int(nodes[b])
        pos = torch.arange(lens[b])
        pg, off = st["table"].cpu()[b, pos // PAGE].long().cuda(), (pos % PAGE).cuda()
        raw = st["cache"].view(torch.uint8).view(-1, PAGE, DQK * st["cache"].element_size())[pg, off]
        kv = raw.view(st["cache"].dtype).double() * st["k_scale"]
        if st["scales"] is not None:
            kv *= st["scales"].double()[pg, off // _scale_block(case["kv"])][:, None]
        for i in range(n):
            keys = list(range(ctx)) + [ctx + t for t in range(n) if int(words[b, i]) >> t & 1]
            mine = kv if len(keys) == lens[b] else kv[torch.tensor(keys, device="cuda")]
            s = (st["q"][b, i].double() * st["q_scale"]) @ mine.T * SM_SCALE
            lse[b, i] = torch.logsumexp(s, dim=1)
            out[b, i] = torch.exp(s - lse[b, i][:, None]) @ mine[:, :LAT]
    return {"out": out, "lse": lse}


def _e4m3(x):
    """The nearest e4m3 value (ties to even) of float64 values within +-448."""
    a = np.abs(x)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0) - 3.0)
    return np.sign(x) * np.rint(a / step) * step


def _exact_accept(st):
    case, sb = st["case"], _scale_block(st["case"]["kv"])
    table, lens = st["table"].cpu().numpy(), st["lens"].cpu().numpy()
    path, count = _paths(case)
    caches = st["caches"].double().cpu().numpy().reshape(case["layers"], -1, DQK)
    scales = st["scales"].double().cpu().numpy().reshape(case["layers"], -1)
    for b in range(case["requests"]):
        base = int(lens[b]) - case["q_len"]

        def slot(pos):
            return int(table[b, pos // PAGE]) * PAGE + pos % PAGE

        for n in range(case["layers"]):
            src = [slot(base + int(i)) for i in path[b, :count[b]]]
            rows = {base + i: caches[n, s] * scales[n, s // sb] for i, s in enumerate(src)}
            for first in range(base // sb * sb, base + int(count[b]), sb):
                mine = {p: x for p, x in rows.items() if first <= p < first + sb}
                g = slot(first) // sb
                old = 0.0 if first >= base else scales[n, g]
                amax = max(max(np.abs(x).max() for x in mine.values()), 1e-300)
                e = max(MIN_EXP, math.ceil(math.log2(amax / E4M3_MAX)))
                scales[n, g] = max(old, 2.0 ** e)
                if 0.0 < old < scales[n, g]:
                    caches[n, g * sb:(g + 1) * sb] = _e4m3(caches[n, g * sb:(g + 1) * sb] * (old / scales[n, g]))
                for p, x in mine.items():
                    caches[n, slot(p)] = _e4m3(x / scales[n, g])
    return {"caches": caches.reshape(st["caches"].shape), "scales": scales.reshape(st["scales"].shape), "lens": None}
