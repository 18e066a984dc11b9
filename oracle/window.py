"""fp64 reference of the sliding-window and block-scaled-cache steps (test
infrastructure only; see the package docstring).

A query at position p sees key j iff j <= p and (no window, or j > p - window,
or j < sinks).  A block-scaled cache stands for scale * e4m3(code), one scale
for each `sb` rows of the flattened cache."""

from __future__ import annotations

import math

import numpy as np

from . import codecs
from .mla import BLOCK, L, attend, page_rows

E4M3_MAX = 448.0
MIN_EXP = -100


def visible(p, window, sinks):
    """Ascending positions of the keys that the query at position p sees."""
    return np.array([j for j in range(p + 1)
                     if window == 0 or j > p - window or j < sinks], dtype=np.int64)


def scaled_values(codes, scales):
    """fp64 values [num_blocks, 64, 576] of e4m3 codes (uint8) and their
    scales [num_blocks, 64/sb]."""
    sb = BLOCK // scales.shape[1]
    return codecs.e4m3_to_f64(codes) * np.repeat(scales.astype(np.float64), sb, axis=1)[..., None]


def window_decode(q, cache, block_table, seq_lens, sm_scale, window, sinks):
    """Absorbed decode of q [B,q_len,H,576] over cache [num_blocks,64,576]
    (both dequantised): out [B,q_len,H,512], lse [B,q_len,H]."""
    B, q_len, H, _ = q.shape
    out = np.zeros((B, q_len, H, L))
    lse = np.full((B, q_len, H), -math.inf)
    for b in range(B):
        for i in range(q_len):
            keys = visible(int(seq_lens[b]) - q_len + i, window, sinks)
            blk, off = page_rows(block_table[b], keys)
            rows = cache[blk, off]
            out[b, i], lse[b, i] = attend(q[b, i], rows, rows[:, :L], sm_scale)
    return out, lse


def window_prefill(q, k, v, cu_q, cu_k, sm_scale, window, sinks):
    """Causal prefill attention with a window: q [Tq,H,192], k [Nk,H,192],
    v [Nk,H,128]; query i of nq stands at position i + nk - nq."""
    Tq, H, _ = q.shape
    out = np.zeros((Tq, H, v.shape[2]))
    lse = np.full((Tq, H), -math.inf)
    for b in range(len(cu_q) - 1):
        nq, nk = int(cu_q[b + 1] - cu_q[b]), int(cu_k[b + 1] - cu_k[b])
        for i in range(nq):
            keys = int(cu_k[b]) + visible(i + nk - nq, window, sinks)
            t = int(cu_q[b]) + i
            for h in range(H):
                o, e = attend(q[t, h][None], k[keys, h], v[keys, h], sm_scale)
                out[t, h], lse[t, h] = o[0], e[0]
    return out, lse


def block_scale(amax):
    """2^max(-100, ceil(log2(amax / 448)))."""
    if amax == 0:
        return 2.0 ** MIN_EXP
    return 2.0 ** max(MIN_EXP, math.ceil(math.log2(amax / E4M3_MAX)))


def append(codes, scales, rows, slots):
    """The append of bf16 rows [T,576] (fp64 values) at `slots` to a
    block-scaled cache: (codes [num_blocks,64,576] uint8, scales), new arrays.
    Negative and out-of-range slots store nothing; the last of equal slots
    stays."""
    sb = BLOCK // scales.shape[1]
    flat = codes.reshape(-1, codes.shape[-1]).copy()
    sc = scales.astype(np.float64).reshape(-1).copy()
    last = {}
    for t, s in enumerate(np.asarray(slots).tolist()):
        if 0 <= s < flat.shape[0]:
            last[s] = t
    blocks = sorted({s // sb for s in last})
    for g in blocks:
        mine = {s: t for s, t in last.items() if s // sb == g}
        x = np.stack([rows[t] for t in mine.values()])
        fin = np.abs(x[np.isfinite(x)])
        old = sc[g]
        if g * sb in mine or not (0.0 < old <= 2.0 ** 120):
            old = 0.0
        new = max(old, block_scale(fin.max() if fin.size else 0.0))
        if 0.0 < old < new:
            ratio = np.float32(old) / np.float32(new)
            for s in range(g * sb, (g + 1) * sb):
                if s not in mine:
                    v = codecs.e4m3_to_f64(flat[s]).astype(np.float32) * ratio
                    flat[s] = codecs.f32_to_e4m3(v)
        for s, t in mine.items():
            flat[s] = codecs.f32_to_e4m3(rows[t].astype(np.float32) / np.float32(new))
        sc[g] = new
    return flat.reshape(codes.shape), sc.reshape(scales.shape).astype(np.float32)
