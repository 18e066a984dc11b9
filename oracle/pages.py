"""Reference of the cache-page calls, one step after another (test infrastructure
only; see the package docstring).

refs, table and lens are NumPy integer arrays and pools lists of arrays
[num_blocks, ...]; all are changed in place.  Each call returns the set of error
names that it raises: "pages", "range", "len", "block"."""

from __future__ import annotations

import numpy as np

from . import codecs
from .mla import BLOCK
from .window import block_scale


def _pages(n):
    return -(-int(n) // BLOCK)


def copy(pools, src, dst):
    errors = set()
    nb = pools[0].shape[0]
    pairs = []
    for s, d in zip(src, dst):
        if s >= nb or d >= nb:
            errors.add("block")
        pairs.append((int(s), int(d)) if 0 <= s < nb and 0 <= d < nb and s != d else None)
    before = [p.copy() for p in pools]
    sources = {p[0] for p in pairs if p}
    for p in pairs:
        if not p:
            continue
        if p[1] in sources:
            errors.add("pages")
            continue
        for old, new in zip(before, pools):
            new[p[1]] = old[p[0]]
    return errors


def _free(refs):
    return [int(i) for i in np.flatnonzero(refs == 0)]


def resize(refs, table, lens, new_lens):
    errors = set()
    most = table.shape[1] * BLOCK
    ok = [0 <= o <= most and 0 <= n <= most for o, n in zip(lens, new_lens)]
    if not all(ok):
        errors.add("len")
    for b, good in enumerate(ok):
        if not good:
            continue
        for k in range(_pages(new_lens[b]), _pages(lens[b])):
            page, table[b, k] = int(table[b, k]), -1
            if not 0 <= page < len(refs):
                errors.add("block")
            elif refs[page] <= 0:
                errors.add("pages")
            else:
                refs[page] -= 1
    free, wanted = _free(refs), 0
    for b, good in enumerate(ok):
        if not good:
            continue
        had, need = _pages(lens[b]), max(0, _pages(new_lens[b]) - _pages(lens[b]))
        wanted += need
        if need and wanted > len(free):
            errors.add("pages")
            continue
        for k in range(need):
            page = free[wanted - need + k]
            table[b, had + k] = page
            refs[page] = 1
        lens[b] = new_lens[b]
    return errors


def fork(pools, refs, table, lens, parents, children, by_rows=None):
    """by_rows: whether a pool's page is 64 rows (None: all of them are); else the whole page
    is copied."""
    errors = set()
    B, most = table.shape[0], table.shape[1] * BLOCK
    free, wanted, seen = _free(refs), 0, set()
    refs0, table0, lens0 = refs.copy(), table.copy(), lens.copy()

    def held(p, k):
        """The parent's k-th page; -1 where the entry is none, or one that nobody holds."""
        page = int(table0[p, k])
        if not 0 <= page < len(refs0):
            errors.add("block")
        elif refs0[page] <= 0:
            errors.add("pages")
        else:
            return page
        return -1

    for p, c in zip(parents, children):
        p, c = int(p), int(c)
        if not (0 <= p < B and 0 <= c < B):
            errors.add("range")
            if 0 <= c < B:
                seen.add(c)
            continue
        if c in seen or lens0[c] != 0:
            errors.add("pages")
            seen.add(c)
            continue
        seen.add(c)
        n = int(lens0[p])
        if not 0 <= n <= most:
            errors.add("len")
            continue
        part = n % BLOCK
        last = held(p, n // BLOCK) if part else -1
        wanted += last >= 0
        if last >= 0 and wanted > len(free):
            errors.add("pages")
            continue
        for k in range(n // BLOCK):
            page = table[c, k] = held(p, k)
            if page >= 0:
                refs[page] += 1
        if part and last < 0:
            table[c, n // BLOCK] = -1
        elif part:
            dst = table[c, n // BLOCK] = free[wanted - 1]
            refs[dst] = 1
            for k, pool in enumerate(pools):
                rows = by_rows is None or by_rows[k]
                flat = pool.reshape(pool.shape[0], BLOCK if rows else 1, -1)
                flat[dst, :part if rows else 1] = flat[last, :part if rows else 1]
        lens[c] = n
    return errors


def compact(pools, refs, table, lens):
    """Returns (pages in use, errors)."""
    errors = set()
    n = int((refs > 0).sum())
    high = [i for i in range(n, len(refs)) if refs[i] > 0]
    low = [i for i in range(n) if not refs[i] > 0]
    now = dict(zip(high, low))
    for s, d in now.items():
        for pool in pools:
            pool[d] = pool[s]
        refs[d], refs[s] = refs[s], 0
    for b in range(table.shape[0]):
        if not 0 <= lens[b] <= table.shape[1] * BLOCK:
            errors.add("len")
        for k in range(min(max(_pages(lens[b]), 0), table.shape[1])):
            page = int(table[b, k])
            if not 0 <= page < len(refs):
                errors.add("block")
            elif page >= n:
                if page in now:
                    table[b, k] = now[page]
                else:
                    errors.add("pages")
    return n, errors


def accept(caches, scales, table, lens, tree_lens, q_len, path, path_lens):
    """caches: arrays [num_blocks, 64, 576] (bits); scales: None, or arrays [num_blocks, 64/sb] and
    the caches e4m3 codes.  Returns (new_lens, errors)."""
    errors = set()
    new_lens = lens.copy()
    for b in range(len(lens)):
        n = q_len if tree_lens is None else int(tree_lens[b])
        length, k = int(lens[b]), int(path_lens[b])
        if not 0 <= length <= table.shape[1] * BLOCK or not 0 <= n <= q_len:
            errors.add("len")
            continue
        base = length - n
        nodes = [int(x) for x in path[b, :max(k, 0)]]
        if not 0 <= k <= min(n, path.shape[1]) or (k and base < 0) or \
                any(x <= y for x, y in zip(nodes, [-1] + nodes)) or any(x >= n for x in nodes):
            errors.add("range")
            continue
        if base < 0:
            continue

        def slot(pos):
            page = int(table[b, pos // BLOCK])
            if not 0 <= page < caches[0].shape[0]:
                errors.add("block")
                return None
            return page * BLOCK + pos % BLOCK

        src, dst = [slot(base + x) for x in nodes], [slot(base + i) for i in range(k)]
        if None in src or None in dst:
            continue
        new_lens[b] = base + k
        for c, cache in enumerate(caches):
            flat = cache.reshape(-1, cache.shape[-1])
            rows = flat[src].copy()
            if scales is None:
                flat[dst] = rows
                continue
            sb = BLOCK // scales[c].shape[1]
            sc = scales[c].reshape(-1)
            size = np.array([sc[s // sb] for s in src], np.float32)
            size = np.where((size >= 0) & (size <= np.float32(2.0 ** 120)), size, np.float32(np.nan))
            for first in range(base // sb * sb, base + k, sb):
                mine = [i for i in range(k) if first <= base + i < first + sb]
                if not mine:
                    continue
                g = dst[mine[0]] // sb
                x = codecs.e4m3_to_f64(rows[mine]) * size[mine].astype(np.float64)[:, None]
                x = np.abs(x[np.isfinite(x)])
                old = np.float32(sc[g])
                if first >= base or not 0 < old <= np.float32(2.0 ** 120):
                    old = np.float32(0)
                new = max(old, np.float32(block_scale(x.max() if x.size else 0.0)))
                if 0 < old < new:
                    for s in range(g * sb, (g + 1) * sb):
                        if s not in dst:
                            flat[s] = codecs.f32_to_e4m3(codecs.e4m3_to_f64(flat[s]).astype(np.float32) * (old / new))
                for i in mine:
                    v = codecs.e4m3_to_f64(rows[i]).astype(np.float32) * (size[i] / new)
                    flat[dst[i]] = codecs.f32_to_e4m3(v)
                sc[g] = new
    return new_lens, errors
