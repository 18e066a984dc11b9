"""fp64 reference of the decode of a tree of drafted tokens (test infrastructure
only; see the package docstring)."""

from __future__ import annotations

import math

import numpy as np

from .mla import L, attend, page_rows


def visible(length, n, word):
    """Ascending positions that a drafted token with this mask word sees, of a
    sequence of `length` tokens of which the last n are drafted."""
    ctx = length - n
    keys = list(range(max(ctx, 0)))
    return np.array(keys + [ctx + t for t in range(n) if int(word) >> t & 1 and ctx + t >= 0], dtype=np.int64)


def chain(q_len):
    """The words of a chain."""
    return np.array([(2 << i) - 1 for i in range(q_len)], dtype=np.uint64)


def words(parents):
    """The words of a tree: a token sees itself and all above it (parent -1: a root; parents stand
    in front of their children)."""
    w = np.zeros(len(parents), np.uint64)
    for i, p in enumerate(parents):
        w[i] = (w[p] if p >= 0 else np.uint64(0)) | np.uint64(1) << np.uint64(i)
    return w


def tree_decode(q, cache, block_table, seq_lens, masks, tree_lens, sm_scale):
    """q [B,q_len,H,576] over cache [num_blocks,64,576] (both dequantised):
    out [B,q_len,H,512], lse [B,q_len,H]; masks [B,q_len] words."""
    B, q_len, H, _ = q.shape
    out = np.zeros((B, q_len, H, L))
    lse = np.full((B, q_len, H), -math.inf)
    for b in range(B):
        n = q_len if tree_lens is None else int(tree_lens[b])
        for i in range(n):
            keys = visible(int(seq_lens[b]), n, masks[b, i])
            blk, off = page_rows(block_table[b], keys)
            rows = cache[blk, off]
            out[b, i], lse[b, i] = attend(q[b, i], rows, rows[:, :L], sm_scale)
    return out, lse
