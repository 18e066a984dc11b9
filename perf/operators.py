"""Cases of the window, sink and block-scaled-cache operators, with their plain forms.

Five operators of the latent-attention serving path:

append    rotary embedding of the new tokens' q_pe / k_pe and the append of kv_c | k_pe rows to a
          paged e4m3 cache that has one scale for each block of tokens
gather    dequantising gather of context rows out of that cache
scaled    absorbed decode attention over that cache (optionally windowed)
window    absorbed decode attention with a sliding window and sinks over a bf16 or e4m3 cache
prefill   causal prefill attention of expanded heads with a sliding window and sinks

``own`` selects the library's calls; otherwise ``run`` computes the same with elementary torch
operations.  ``exact`` states each operator again, in 64 bits, request by request.
"""

import math

import numpy as np
import torch

own = False

PAGE, LAT, ROPE, DQK, DV, DQ = 64, 512, 64, 576, 128, 192
SM_SCALE = 1.0 / math.sqrt(192.0)
E4M3_MAX = 448.0
MIN_EXP = -100           # the smallest scale is 2^-100
BASE = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a busy server: one new token for each of 32 requests
        dict(name="append step", op="append", requests=32, new=1, heads=128, history=4096,
             scale_block=64, layout="interleaved", lengths=1),
        # the chunk of a chunked prefill: up to 512 new tokens for each of four requests,
        # starting anywhere in a page
        dict(name="append chunk", op="append", requests=4, new=512, heads=128, history=2000,
             scale_block=32, layout="half", lengths=2),
        # a short context chunk of a few requests, starting inside their sequences
        dict(name="gather ragged", op="gather", requests=5, rows=300, start=77, scale_block=16,
             lengths=3),
        # the context step of a chunked prefill: 4 x 8192 rows
        dict(name="gather context", op="gather", requests=4, rows=8192, start=0, scale_block=64,
             lengths=0),
        # two short chats on one shard of the heads: latency counts
        dict(name="scaled tiny", op="scaled", requests=2, q_len=1, heads=16, shape="even",
             context=130, scale_block=64, window=0, sinks=0, lengths=4),
        # a full batch at mixed lengths, every earlier token visible
        dict(name="scaled batch", op="scaled", requests=64, q_len=1, heads=128, shape="uniform",
             context=16384, scale_block=64, window=0, sinks=0, lengths=5),
        # one long document, finest scales
        dict(name="scaled long", op="scaled", requests=1, q_len=1, heads=128, shape="even",
             context=131072, scale_block=16, window=0, sinks=0, lengths=6),
        # one chat on a small model's heads, a short window
        dict(name="window tiny", op="window", requests=1, q_len=1, heads=16, shape="even",
             context=700, kv="bf16", window=128, sinks=4, lengths=7),
        # the usual decode batch with a window of 1024
        dict(name="window batch", op="window", requests=32, q_len=1, heads=128, shape="even",
             context=4096, kv="bf16", window=1024, sinks=4, lengths=8),
        # speculative decode: two tokens a request, long tail of lengths, a wide window
        dict(name="window speculative", op="window", requests=128, q_len=2, heads=128,
             shape="lognormal", context=32768, kv="bf16", window=4096, sinks=16, lengths=9),
        # a ragged batch of short prompts on one shard of the heads
        dict(name="prefill ragged", op="prefill", requests=3, new=333, context=200, heads=16,
             window=96, sinks=4, lengths=10),
        # 512 new tokens for each of four requests over 8192 tokens of context
        dict(name="prefill chunk", op="prefill", requests=4, new=512, context=8192, heads=128,
             window=1024, sinks=4, lengths=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gather", "scaled", "scaled", "window", "window", "prefill"])
    c = dict(op=op, lengths=rng.randrange(1, 1 << 20))
    if op == "append":
        c["new"] = _log(rng, 1, 512)
        c["requests"] = _log(rng, 1, max(1, min(128, 2048 // c["new"])))
        c["heads"] = rng.choice([8, 16, 33, 64, 128])
        c["history"] = _log(rng, 1, 4096)
        c["scale_block"] = rng.choice([16, 32, 64])
        c["layout"] = rng.choice(["interleaved", "half"])
    elif op == "gather":
        c["rows"] = _log(rng, 1, 8192)
        c["requests"] = _log(rng, 1, max(1, min(64, 32768 // c["rows"])))
        c["start"] = rng.choice([0, 0, 31, 640])
        c["scale_block"] = rng.choice([16, 32, 64])
    elif op == "prefill":
        c["heads"] = rng.choice([1, 5, 16, 40, 128])
        c["new"] = _log(rng, 1, 512)
        c["context"] = rng.choice([0, _log(rng, 1, 8192)])
        c["requests"] = rng.randint(1, 4)
        c["window"] = _log(rng, 16, 2048)
        c["sinks"] = rng.choice([0, 1, 4, 130])
    else:
        c["context"] = _log(rng, 64, 32768)
        c["requests"] = _log(rng, 1, max(1, min(96, 400000 // c["context"])))
        c["q_len"] = rng.choice([1, 1, 1, 2, 4])
        c["heads"] = rng.choice([16, 20, 64, 128])
        c["shape"] = rng.choice(["even", "uniform", "lognormal"])
        c["window"] = rng.choice([0, _log(rng, 32, 8192)])
        c["sinks"] = rng.choice([0, 4, 70]) if c["window"] else 0
        if op == "scaled":
            c["scale_block"] = rng.choice([16, 32, 64])
        else:
            c["kv"] = rng.choice(["bf16", "e4m3"])
    return c


def _context_lens(case):
    """Sequence lengths of a decode case, fixed by the case."""
    r = np.random.RandomState(case["lengths"])
    n, top = case["requests"], case["context"]
    if case["shape"] == "even":
        lens = np.maximum(1, top - r.randint(0, max(1, top // 16), n))
        lens[0] = top
    elif case["shape"] == "uniform":
        lens = r.randint(max(1, top // 16), top + 1, n)
    else:
        lens = np.clip(np.exp(r.normal(math.log(max(2, top // 16)), 1.0, n)), 2, top)
    return np.maximum(lens.astype(np.int64), case["q_len"])


def _ragged(case, key, r):
    """`requests` counts up to case[key], the first of them whole."""
    n = case[key]
    got = np.maximum(1, n - r.randint(0, n // 4 + 1, case["requests"])) if case["lengths"] else \
        np.full(case["requests"], n)
    got[0] = n
    return got.astype(np.int64)


def _append_lens(case):
    r = np.random.RandomState(case["lengths"])
    return r.randint(0, case["history"] + 1, case["requests"]).astype(np.int64), _ragged(case, "new", r)


def _gather_lens(case):
    return _ragged(case, "rows", np.random.RandomState(case["lengths"]))


def _prefill_lens(case):
    r = np.random.RandomState(case["lengths"])
    nq = _ragged(case, "new", r)
    ctx = np.full(case["requests"], case["context"], np.int64)
    if case["lengths"]:
        ctx = r.randint(case["context"] // 2, case["context"] + 1, case["requests"]).astype(np.int64)
    return nq, nq + ctx


def _visible(pos, window, sinks):
    """Number of tokens that the query at position pos sees."""
    n = pos + 1
    if window == 0 or n <= window:
        return n
    return window + min(sinks, n - window)


def _union(first, last, window, sinks):
    """Number of tokens that the queries at positions first .. last see together."""
    n = last + 1
    lo = max(0, first - window + 1) if window else 0
    return (n - lo) + min(sinks, lo)


def work(case):
    op = case["op"]
    if op == "append":
        _, new = _append_lens(case)
        T = int(new.sum())
        row = T * (DQK * 2 + DQK)                       # kv_c | k_pe in, one cache row out
        rot = T * case["heads"] * ROPE * 2 * 2 + T * ROPE * 2 + T * 8
        return {"bytes": row + rot + 8 * -(-T // case["scale_block"]),
                "flops": 6 * (T * case["heads"] * ROPE / 2 + T * ROPE / 2) + 3 * T * DQK}
    if op == "gather":
        n = int(_gather_lens(case).sum())
        return {"bytes": n * (DQK + 2 * DQK) + 4 * -(-n // case["scale_block"]) + 4 * -(-n // PAGE),
                "flops": n * DQK}
    if op == "prefill":
        nq, nk = _prefill_lens(case)
        H, w, s = case["heads"], case["window"], case["sinks"]
        pairs = sum(_visible(p, w, s) for a, b in zip(nq, nk) for p in range(b - a, b))
        keys = sum(_union(b - a, b - 1, w, s) for a, b in zip(nq, nk))
        tq = int(nq.sum())
        return {"bytes": H * (int(keys) * (DQ + DV) * 2 + tq * ((DQ + DV) * 2 + 4)),
                "flops": 2.0 * H * int(pairs) * (DQ + DV)}
    lens, q_len, H = _context_lens(case), case["q_len"], case["heads"]
    w, s = case["window"], case["sinks"]
    size = 1 if op == "scaled" or case["kv"] == "e4m3" else 2
    keys = int(sum(_union(n - q_len, n - 1, w, s) for n in lens))
    pairs = int(sum(_visible(n - q_len + i, w, s) for n in lens for i in range(q_len)))
    rows = case["requests"] * q_len * H
    scales = 4 * -(-keys // case["scale_block"]) if op == "scaled" else 0
    return {"bytes": keys * DQK * size + scales + rows * (DQK * size + LAT * 2 + 4) + 4 * -(-keys // PAGE),
            "flops": 2.0 * H * pairs * (DQK + LAT)}


# ----------------------------------------------------------------- inputs
def _table(lens, seed):
    """Shuffled pages of requests of `lens` tokens: (block table [B, max_blocks], pages)."""
    r = np.random.RandomState(seed % (1 << 31))
    pages = -(-np.asarray(lens) // PAGE)
    total = int(pages.sum()) + 3
    perm = r.permutation(total).astype(np.int32)
    bt = np.full((len(lens), max(1, int(pages.max()))), -1, np.int32)
    at = 0
    for b, n in enumerate(pages):
        bt[b, :n] = perm[at:at + n]
        at += int(n)
    return bt, total


def _owned(bt, lens, total):
    """Rows of the pool that hold a token of a request, as a flat boolean array."""
    m = np.zeros((total, PAGE), bool)
    for b, n in enumerate(lens):
        k = int(n) // PAGE
        m[bt[b, :k]] = True
        if n % PAGE:
            m[bt[b, k], :n % PAGE] = True
    return m.reshape(-1)


def _exponent(amax):
    """Smallest e with amax <= 448 * 2^e, at least MIN_EXP."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)


def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _scaled_cache(total, sb, gen):
    """An e4m3 pool [pages, 64, 576] of normal rows whose size wanders from block to block, and
    its scales [pages, 64 / sb]."""
    x = torch.randn((total * PAGE // sb, sb, DQK), generator=gen, device="cuda")
    x *= torch.exp2(torch.rand((x.shape[0], 1, 1), generator=gen, device="cuda") * 1.5 - 1.0)
    s = _pow2(_exponent(x.abs().amax(dim=(1, 2))))
    codes = (x / s[:, None, None]).to(torch.float8_e4m3fn)
    return codes.view(total, PAGE, DQK), s.view(total, PAGE // sb)


def _i32(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    op = case["op"]
    st = {"case": case}

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)

    if op == "append":
        hist, new = _append_lens(case)
        bt, total = _table(hist + new, seed)
        pos = np.concatenate([h + np.arange(n) for h, n in zip(hist, new)])
        req = np.repeat(np.arange(len(new)), new)
        slots = bt[req, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE
        T = len(pos)
        st["cache"], st["scales"] = _scaled_cache(total, case["scale_block"], gen)
        # kv_c | k_pe as the projection leaves them, in one row; q_pe behind the nope part
        kv = normal(T, DQK, std=1.5)
        st["kv_c"], st["k_pe"] = kv[:, :LAT], kv[:, LAT:]
        st["q_pe"] = normal(T, case["heads"], DQ)[:, :, DV:]
        st["q_out"] = torch.empty((T, case["heads"], ROPE), dtype=torch.bfloat16, device="cuda")
        st["k_out"] = torch.empty((T, ROPE), dtype=torch.bfloat16, device="cuda")
        st["positions"], st["slots"] = _i32(pos), _i32(slots)
    elif op == "gather":
        rows = _gather_lens(case)
        lens = rows + case["start"] + 5
        bt, total = _table(lens, seed)
        st["cache"], st["scales"] = _scaled_cache(total, case["scale_block"], gen)
        st["table"], st["lens"] = _i32(bt), _i32(lens)
        st["starts"] = _i32(np.full(len(rows), case["start"]))
        st["cu"] = _i32(np.concatenate([[0], np.cumsum(rows)]))
        st["rows"] = int(rows.sum())
    elif op == "prefill":
        nq, nk = _prefill_lens(case)
        H = case["heads"]
        st["q"] = normal(int(nq.sum()), H, DQ)
        st["k"] = normal(int(nk.sum()), H, DQ)
        st["v"] = normal(int(nk.sum()), H, DV)
        st["cu_q"] = _i32(np.concatenate([[0], np.cumsum(nq)]))
        st["cu_k"] = _i32(np.concatenate([[0], np.cumsum(nk)]))
        st["max_q"], st["max_k"] = int(nq.max()), int(nk.max())
    else:
        lens = _context_lens(case)
        bt, total = _table(lens, seed)
        stale = torch.as_tensor(~_owned(bt, lens, total), device="cuda")
        q = torch.randn((case["requests"], case["q_len"], case["heads"], DQK), generator=gen, device="cuda")
        st["q_scale"], st["k_scale"] = 1.0, 1.0
        if op == "scaled":
            st["cache"], st["scales"] = _scaled_cache(total, case["scale_block"], gen)
        else:
            st["cache"] = torch.randn((total, PAGE, DQK), generator=gen, device="cuda")
            if case["kv"] == "e4m3":
                st["k_scale"] = float(st["cache"].abs().max()) / E4M3_MAX
                st["cache"] = (st["cache"] / (st["k_scale"] * 1.001)).to(torch.float8_e4m3fn)
                st["k_scale"] *= 1.001
            else:
                st["cache"] = st["cache"].to(torch.bfloat16)
        if st["cache"].dtype == torch.float8_e4m3fn:
            st["q_scale"] = float(q.abs().max()) / E4M3_MAX * 1.001
            q = (q / st["q_scale"]).to(torch.float8_e4m3fn)
            st["cache"].view(torch.uint8).view(-1, DQK)[stale] = 0x7F     # rows that no token owns: NaN
        else:
            q = q.to(torch.bfloat16)
            st["cache"].view(-1, DQK)[stale] = math.nan
        st["q"], st["table"], st["lens"] = q, _i32(bt), _i32(lens)
    return st


# ------------------------------------------------------------ plain forms
def _rotate(x, pos, layout):
    """Rotary embedding of x [T, ..., 64] by positions [T], in 64 bits, rounded to bf16 once."""
    i = torch.arange(ROPE // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None] * torch.exp2(-(2.0 * i / ROPE) * math.log2(BASE))
    ang = ang.view((x.shape[0],) + (1,) * (x.dim() - 2) + (ROPE // 2,))
    c, s = torch.cos(ang), torch.sin(ang)
    x = x.double()
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2).to(torch.bfloat16)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * c - b * s, a * s + b * c], dim=-1).to(torch.bfloat16)


def _plain_append(st):
    case = st["case"]
    sb = case["scale_block"]
    cache, scales = st["cache"], st["scales"]
    st["q_out"].copy_(_rotate(st["q_pe"], st["positions"], case["layout"]))
    st["k_out"].copy_(_rotate(st["k_pe"], st["positions"], case["layout"]))
    rows = torch.cat([st["kv_c"], st["k_out"]], dim=1).float()
    slot = st["slots"].long()
    blocks, which = torch.unique(slot // sb, return_inverse=True)
    n = blocks.shape[0]
    amax = torch.zeros(n, device="cuda").scatter_reduce(0, which, rows.abs().amax(dim=1), "amax")
    # a block whose first row is written begins afresh
    fresh = torch.zeros(n, device="cuda").scatter_reduce(0, which, (slot % sb == 0).float(), "amax") > 0
    flat = scales.view(-1)
    old = torch.where(fresh, torch.zeros_like(amax), flat[blocks])
    new = torch.maximum(old, _pow2(_exponent(amax)))
    # rows that are there already follow a scale that grew
    codes = cache.view(-1, sb, DQK)
    kept = codes.view(torch.uint8)[blocks]
    ratio = (old / new)[:, None, None]
    moved = (kept.view(torch.float8_e4m3fn).float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8)
    grew = (old > 0) & (new > old)
    codes.view(torch.uint8)[blocks] = torch.where(grew[:, None, None], moved, kept)
    flat[blocks] = new
    put = (rows / new[which][:, None]).to(torch.float8_e4m3fn)
    cache.view(torch.uint8).view(-1, DQK)[slot] = put.view(torch.uint8)
    return {"q": st["q_out"], "k": st["k_out"], "cache": cache, "scales": scales}


def _dequantised(cache, scales, rows):
    """Values of the flat cache rows `rows`, in 32 bits."""
    x = cache.view(torch.uint8).view(-1, DQK)[rows].view(torch.float8_e4m3fn).float()
    sb = PAGE // scales.shape[1]
    return x * scales.reshape(-1)[rows // sb][..., None]


def _plain_gather(st):
    cu = st["cu"].long()
    at = torch.arange(st["rows"], device="cuda")
    b = torch.bucketize(at, cu[1:], right=True)
    pos = st["starts"].long()[b] + at - cu[b]
    rows = st["table"].long()[b, pos // PAGE] * PAGE + pos % PAGE
    return _dequantised(st["cache"], st["scales"], rows).to(torch.bfloat16)


def _plain_decode(st):
    case = st["case"]
    q, table, lens = st["q"], st["table"].long(), st["lens"].long()
    B, q_len, H, _ = q.shape
    j = torch.arange(table.shape[1] * PAGE, device="cuda")
    p = lens[:, None] - q_len + torch.arange(q_len, device="cuda")           # [B, q_len]
    see = (j <= p[..., None]) & (j < lens[:, None, None])                    # [B, q_len, n]
    if case["window"]:
        see &= (j > p[..., None] - case["window"]) | (j < case["sinks"])
    some = see.any(dim=1)                                                    # [B, n]
    rows = (table[:, j // PAGE] * PAGE + j % PAGE).clamp(min=0)
    if case["op"] == "scaled":
        kv = _dequantised(st["cache"], st["scales"], rows)
    else:
        kv = st["cache"].view(torch.uint8).view(-1, DQK * st["cache"].element_size())[rows]
        kv = kv.view(st["cache"].dtype).float() * st["k_scale"]
    kv = torch.where(some[..., None], kv, torch.zeros((), device="cuda"))
    qf = (q.float() * st["q_scale"]).view(B, q_len * H, DQK)
    s = torch.matmul(qf, kv.transpose(1, 2)).view(B, q_len, H, -1) * SM_SCALE
    s = s.masked_fill(~see[:, :, None, :], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - m)
    z = e.sum(dim=-1, keepdim=True)
    out = torch.matmul((e / z).view(B, q_len * H, -1), kv[..., :LAT]).view(B, q_len, H, LAT)
    return {"out": out.to(torch.bfloat16), "lse": (m + torch.log(z))[..., 0]}


def _plain_prefill(st):
    case = st["case"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    i = torch.arange(st["max_q"], device="cuda")
    j = torch.arange(st["max_k"], device="cuda")
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    qi = (cu_q[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)               # [B, max_q]
    kj = (cu_k[:-1, None] + j).clamp(max=st["k"].shape[0] - 1)
    p = i + (nk - nq)[:, None]                                               # [B, max_q]
    see = (j <= p[..., None]) & ((j > p[..., None] - case["window"]) | (j < case["sinks"]))
    see &= (j < nk[:, None])[:, None, :]
    q = st["q"][qi].float().transpose(1, 2)                                  # [B, H, max_q, 192]
    k = st["k"][kj].float().permute(0, 2, 3, 1)                              # [B, H, 192, max_k]
    v = st["v"][kj].float().transpose(1, 2)                                  # [B, H, max_k, 128]
    s = (torch.matmul(q, k) * SM_SCALE).masked_fill(~see[:, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - m)
    z = e.sum(dim=-1, keepdim=True)
    out = (torch.matmul(e, v) / z).transpose(1, 2)                           # [B, max_q, H, 128]
    lse = (m + torch.log(z))[..., 0].transpose(1, 2)                         # [B, max_q, H]
    t = torch.arange(st["q"].shape[0], device="cuda")
    b = torch.bucketize(t, cu_q[1:], right=True)
    return {"out": out[b, t - cu_q[b]].to(torch.bfloat16), "lse": lse[b, t - cu_q[b]]}


def _own_call(st):
    import mla_latent_kv_uk_gb300 as mla

    case = st["case"]
    op = case["op"]
    if op == "append":
        mla.mla_rope_cache_append(st["q_pe"], st["k_pe"], st["kv_c"], st["positions"], st["slots"],
                                  st["cache"], st["scales"], rope_base=BASE, layout=case["layout"],
                                  q_out=st["q_out"], k_out=st["k_out"])
        return {"q": st["q_out"], "k": st["k_out"], "cache": st["cache"], "scales": st["scales"]}
    if op == "gather":
        return mla.mla_gather_cache_scaled(st["cache"], st["scales"], st["table"], st["lens"], st["cu"],
                                           st["rows"], seq_starts=st["starts"])
    if op == "scaled":
        out, lse = mla.mla_decode_paged_scaled(st["q"], st["cache"], st["scales"], st["table"], st["lens"],
                                               sm_scale=SM_SCALE, q_scale=st["q_scale"],
                                               window=case["window"], sinks=case["sinks"])
    elif op == "window":
        out, lse = mla.mla_decode_paged_window(st["q"], st["cache"], st["table"], st["lens"],
                                               sm_scale=SM_SCALE, window=case["window"],
                                               sinks=case["sinks"], q_scale=st["q_scale"],
                                               k_scale=st["k_scale"])
    else:
        out, lse = mla.mla_prefill_attn_window(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"],
                                               st["max_q"], window=case["window"],
                                               sinks=case["sinks"], sm_scale=SM_SCALE)
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own_call(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op == "gather":
        return _plain_gather(state)
    if op == "prefill":
        return _plain_prefill(state)
    return _plain_decode(state)


# -------------------------------------------------------- in 64 bits, apart
def _attend64(q, k, v, seen):
    """Rows q [n, d] over the keys of each row's mask [n, m]: outputs and natural-log LSE."""
    s = (q @ k.T) * SM_SCALE
    s[~seen] = -math.inf
    lse = torch.logsumexp(s, dim=1)
    return torch.exp(s - lse[:, None]) @ v, lse


def _seen64(first, n, keys, window, sinks):
    """Mask of queries at positions first .. first + n - 1 over the token positions `keys`."""
    p = first + torch.arange(n, device="cuda")[:, None]
    return (keys <= p) & ((p - keys < (window or 1 << 40)) | (keys < sinks))


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        return _exact_append(st)
    if op == "gather":
        got = []
        cu, table = st["cu"].tolist(), st["table"].cpu()
        sb = case["scale_block"]
        for b in range(len(cu) - 1):
            pos = torch.arange(case["start"], case["start"] + cu[b + 1] - cu[b])
            pg = table[b, pos // PAGE].long().cuda()
            off = (pos % PAGE).cuda()
            codes = st["cache"].view(torch.uint8)[pg, off].view(torch.float8_e4m3fn).double()
            got.append(codes * st["scales"].double()[pg, off // sb][:, None])
        return torch.cat(got)
    if op == "prefill":
        H = case["heads"]
        cu_q, cu_k = st["cu_q"].tolist(), st["cu_k"].tolist()
        out = torch.empty((cu_q[-1], H, DV), dtype=torch.float64, device="cuda")
        lse = torch.empty((cu_q[-1], H), dtype=torch.float64, device="cuda")
        for b in range(len(cu_q) - 1):
            nq, nk = cu_q[b + 1] - cu_q[b], cu_k[b + 1] - cu_k[b]
            # the tokens that any query of the request sees
            lo = max(0, nk - nq - case["window"] + 1)
            keys = torch.cat([torch.arange(min(case["sinks"], lo)), torch.arange(lo, nk)]).cuda()
            seen = _seen64(nk - nq, nq, keys, case["window"], case["sinks"])
            for h in range(H):
                o, e = _attend64(st["q"][cu_q[b]:cu_q[b + 1], h].double(),
                                 st["k"][cu_k[b] + keys, h].double(), st["v"][cu_k[b] + keys, h].double(), seen)
                out[cu_q[b]:cu_q[b + 1], h], lse[cu_q[b]:cu_q[b + 1], h] = o, e
        return {"out": out, "lse": lse}
    B, q_len, H = case["requests"], case["q_len"], case["heads"]
    out = torch.empty((B, q_len, H, LAT), dtype=torch.float64, device="cuda")
    lse = torch.empty((B, q_len, H), dtype=torch.float64, device="cuda")
    w = case["window"]
    for b, n in enumerate(st["lens"].tolist()):
        lo = max(0, n - q_len - w + 1) if w else 0
        keys = torch.cat([torch.arange(min(case["sinks"], lo)), torch.arange(lo, n)]).cuda()
        pg, off = st["table"][b].long()[keys // PAGE], keys % PAGE
        raw = st["cache"].view(torch.uint8).view(-1, PAGE, DQK * st["cache"].element_size())[pg, off]
        kv = raw.view(st["cache"].dtype).double() * st["k_scale"]
        if op == "scaled":
            kv = kv * st["scales"].double()[pg, off // case["scale_block"]][:, None]
        qb = st["q"][b].double() * st["q_scale"]
        seen = _seen64(n - q_len, q_len, keys, w, case["sinks"])
        o, e = _attend64(qb.reshape(q_len * H, DQK), kv, kv[:, :LAT],
                         seen[:, None, :].expand(q_len, H, len(keys)).reshape(q_len * H, -1))
        out[b], lse[b] = o.view(q_len, H, LAT), e.view(q_len, H)
    return {"out": out, "lse": lse}


def _e4m3(x):
    """The nearest e4m3 value (ties to even) of float64 values within +-448."""
    a = np.abs(x)
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -30))), -6.0) - 3.0)
    return np.sign(x) * np.rint(a / step) * step


def _bf16(x):
    """The nearest bf16 value (ties to even) of float64 values."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256.0), e - 8)


def _exact_append(st):
    case = st["case"]
    sb, pos = case["scale_block"], st["positions"].cpu().numpy().astype(np.float64)
    turn = pos[:, None] * BASE ** (-np.arange(ROPE // 2) / (ROPE // 2))

    def rotated(x):
        z = x.reshape(x.shape[0], -1, ROPE // 2, 2) if case["layout"] == "interleaved" else \
            x.reshape(x.shape[0], -1, 2, ROPE // 2).swapaxes(2, 3)
        z = (z[..., 0] + 1j * z[..., 1]) * np.exp(1j * turn)[:, None]
        z = np.stack([z.real, z.imag], axis=-1)
        return (z if case["layout"] == "interleaved" else z.swapaxes(2, 3)).reshape(x.shape)

    q = rotated(st["q_pe"].double().cpu().numpy())
    k = rotated(st["k_pe"].double().cpu().numpy())
    rows = np.concatenate([st["kv_c"].double().cpu().numpy(), _bf16(k)], axis=1)
    cache = st["cache"].double().cpu().numpy().reshape(-1, DQK)
    scales = st["scales"].double().cpu().numpy().reshape(-1)
    slot = st["slots"].cpu().numpy().astype(np.int64)
    for g in np.unique(slot // sb):
        mine = np.flatnonzero(slot // sb == g)
        old = 0.0 if (slot[mine] % sb == 0).any() else scales[g]
        e = max(MIN_EXP, math.ceil(math.log2(max(np.abs(rows[mine]).max(), 1e-300) / E4M3_MAX)))
        scales[g] = max(old, 2.0 ** e)
        if 0.0 < old < scales[g]:
            cache[g * sb:(g + 1) * sb] = _e4m3(cache[g * sb:(g + 1) * sb] * (old / scales[g]))
        cache[slot[mine]] = _e4m3(rows[mine] / scales[g])
    return {"q": q, "k": k, "cache": cache.reshape(-1, PAGE, DQK), "scales": scales.reshape(-1, PAGE // sb)}
