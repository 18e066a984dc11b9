/*
 * mla.h — C ABI of the GB300 (sm_103a) absorbed Multi-head Latent Attention
 * decode library.
 *
 * Sources of the operations (page title, section):
 *   [Q-REP]   prhub digest of vLLM PR 45964, "MLA DCP 中通过 query 复制跳过
 *             all-gather 通信"
 *   [FP8]     prhub digest of vLLM PR 44044, "支持 DCP + FP8 KV Cache 在 MLA
 *             解码中协同"
 *   [BLOG]    "DeepSeek MLA 在 DCP 分布式环境中的 Prefill 阶段解析"
 *
 * Conventions shared by every entry point
 *   - Every tensor pointer is a caller-owned DEVICE pointer (unless the
 *     argument says "host"), contiguous and row-major in the layout given.
 *     The library never allocates or frees device memory: scratch space is a
 *     caller workspace whose size a *_workspace_size query returns.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream) and returns an int status.  Arguments are
 *     validated on the host before any launch and without a device sync;
 *     a bad argument returns MLA_ERR_INVALID_ARG and launches nothing.
 *   - Device-side data the host cannot see (block ids, seq_lens) is checked
 *     inside the kernels: a bad value sets a bit in a device error word and
 *     the offending row is skipped (never read out of bounds).  Read and
 *     clear that word with mla_get_device_error().
 *   - Dtype codes: MLA_BF16 (bf16), MLA_E4M3 (OCP fp8 e4m3, "fn" variant:
 *     no inf, max 448), MLA_F32 (IEEE float32).  Scales are per-tensor fp32.
 *   - Sizes: L = 512 latent rank, R = 64 rope width, 576 = L + R, nope and
 *     value head widths 128, cache page size 64 tokens.
 *   - Kernels run on the current CUDA device of the calling thread; every
 *     pointer must belong to it.
 */
#ifndef MLA_GB300_H_
#define MLA_GB300_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *mla_stream_t; /* identical to cudaStream_t */

enum mla_status {
  MLA_OK = 0,
  MLA_ERR_INVALID_ARG = 1, /* bad pointer / size / dtype combination        */
  MLA_ERR_UNSUPPORTED = 2, /* valid request the library does not implement */
  MLA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than required    */
  MLA_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed          */
};

enum mla_dtype { MLA_BF16 = 0, MLA_E4M3 = 1, MLA_F32 = 2 };

/* Bits of the device error word (mla_get_device_error). */
enum mla_device_error {
  MLA_DEVERR_BLOCK_ID = 1,    /* block-table entry < 0 or >= num_blocks     */
  MLA_DEVERR_SEQ_LEN = 2,     /* seq_len < 0 or > max_blocks * 64           */
  MLA_DEVERR_RANGE = 4,       /* gather range beyond seq_len / workspace    */
  MLA_DEVERR_TIMEOUT = 8,     /* a bounded wait inside a kernel gave up     */
  MLA_DEVERR_PAGES = 16,      /* no free page, or a page operation refused  */
};

/* Self-test of the failure detection every kernel relies on (no
 * counterpart on the pages): one thread waits, through the same bounded
 * mbarrier wait the kernels use, on a barrier that nothing completes; after
 * limit_cycles SM cycles (1 .. 1e9) it gives up and raises
 * MLA_DEVERR_TIMEOUT in the device error word, the way a kernel whose
 * producer or peer stalls reports it.  Faults nothing, and the context stays
 * usable.  MLA_ERR_INVALID_ARG for a limit out of range. */
int mla_selftest_wait_timeout(long long limit_cycles, mla_stream_t stream);

/* Human-readable text of a status code (static storage, never NULL). */
const char *mla_status_string(int status);

/* Library ABI version, currently 1. */
int mla_version(void);

/* Synchronises `stream`, stores the device error word (bitwise OR of
 * mla_device_error values raised since the last call) into *code (host
 * pointer) and clears it.  Returns MLA_ERR_CUDA if the sync fails. */
int mla_get_device_error(int *code, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * A1/A2  Query absorption and concat(-quant)
 * [Q-REP] §实现拆解 5 (decode BMM of the query against W_UK_T);
 * [BLOG] §MLA Prefill vs Decode (Q absorbed into the latent space by an
 * einsum, one latent head of width L+R); [FP8] §关键源码片段
 * mla_attention.py (nope ‖ pe -> (B, N, L+P); _decode_concat_quant_fp8_op).
 *
 *   ql[t,h,l] = sum_p q_nope[t,h,p] * w_uk_t[h,p,l]       (fp32 accumulate)
 *   q_out[t,h,0:512]   = cast(ql[t,h,:]),  q_out[t,h,512:576] = cast(q_pe)
 *
 * q_nope [T,H,128] bf16, q_pe [T,H,64] bf16, w_uk_t [H,128,512] bf16.
 * out_dtype MLA_BF16: round-to-nearest-even of the fp32 value;
 *           MLA_E4M3: e4m3 code of (fp32 value) / q_scale (IEEE fp32
 *                     division, round to nearest even, saturate to +-448);
 *           MLA_F32 : the fp32 value itself.
 * q_out [T,H,576] of out_dtype.  T == 0 is a no-op.  1 <= H <= 4096.
 * q_scale must be finite and > 0 for MLA_E4M3 (ignored otherwise). */
int mla_absorb_q(const void *q_nope, const void *q_pe, const void *w_uk_t,
                 int T, int H, int out_dtype, float q_scale, void *q_out,
                 mla_stream_t stream);

/* ---------------------------------------------------------------------
 * A3/A4/A5  Paged latent decode (forward_mqa) with split-KV and merge
 * [FP8] §关键源码片段 mla_attention.py (forward_mqa(mqa_q, kv_cache, ...)
 * returns attn_out and lse) and §关键源码片段 flashmla.py (split scheduler
 * metadata from seq_lens and the true query-head count); [BLOG] §MLA
 * Prefill vs Decode.
 *
 * For request b, query token i < q_len, head h < H:
 *   range: lo = kv_starts ? max(0, kv_starts[b]) : 0
 *          hi = min(seq_lens[b], causal ? seq_lens[b] - q_len + i + 1 : inf,
 *                   kv_ends ? kv_ends[b] : inf)
 *   s_j  = sm_scale * q_deq[b,i,h,:] . K_j        (j in [lo, hi))
 *   K_j  = kv_deq[slot(b,j), 0:576],  V_j = kv_deq[slot(b,j), 0:512]
 *   slot(b,j) = block_table[b, j/64] * 64 + j%64
 *   lse[b,i,h] = ln sum_j exp(s_j)   (natural log; -inf for an empty range)
 *   out[b,i,h,:] = sum_j exp(s_j - lse) V_j           (0 for an empty range)
 * q_deq = q (bf16) or q_scale * e4m3(q); kv_deq = kv (bf16) or
 * k_scale * e4m3(kv).  q_dtype must equal kv_dtype.
 *
 * q [B,q_len,H,576]; kv_cache [num_blocks,64,576]; block_table
 * [B,max_blocks] int32 (entries past the used pages are ignored);
 * seq_lens [B] int32; kv_starts / kv_ends [B] int32 or NULL (an explicit
 * key shard, e.g. one DCP rank's slice); out [B,q_len,H,512] of out_dtype
 * (MLA_BF16 or MLA_F32); lse [B,q_len,H] fp32.
 *
 * The split of the key ranges over CTAs is planned on the device
 * (mla_decode_plan) and partial results are merged on the device; no host
 * synchronisation.  split_tiles = 0 lets the planner choose; > 0 forces
 * spans of that many 64-token key tiles (testing / tuning).  workspace must
 * hold mla_decode_workspace_size(B, q_len, H, max_blocks*64, split_tiles)
 * bytes (16-byte aligned).
 * Limits: 1 <= B, 1 <= q_len <= 64, 1 <= H <= 4096, 1 <= max_blocks,
 * 1 <= num_blocks < 2^25. */
int mla_decode_workspace_size(int B, int q_len, int H, int max_seq_len,
                              int split_tiles, size_t *bytes);

int mla_decode_paged(const void *q, int q_dtype, float q_scale,
                     const void *kv_cache, int kv_dtype, float k_scale,
                     const int32_t *block_table, const int32_t *seq_lens,
                     const int32_t *kv_starts, const int32_t *kv_ends, int B,
                     int q_len, int H, int max_blocks, int num_blocks,
                     float sm_scale, int causal, int split_tiles, void *out,
                     int out_dtype, float *lse, void *workspace,
                     size_t ws_bytes, mla_stream_t stream);

/* mla_decode_paged without a caller workspace, for callers that cannot
 * allocate device memory at call time: serving runtimes whose device
 * memory is carved up once before traffic starts, plug-in hosts that forbid
 * allocation on the call path, and C callers with no allocator of their
 * own.  No counterpart on the source pages: it is a packaging
 * variant of A3/A4/A5.
 *
 * The plan and the split partials live in one static device array of
 * MLA_NOALLOC_SCRATCH_BYTES (64 MiB) inside the library.  Every GPU on
 * which the library's decode module is loaded holds it until the process
 * exits; with CUDA's default lazy module loading the 64 MiB is committed
 * the first time the decode code is used on a device (the first decode
 * call of any kind), so make that first call before device memory is
 * carved up, and before any stream capture (it also looks the array's
 * device address up once, with cudaGetSymbolAddress, and caches it per
 * device index).  cudaDeviceReset is not supported once the library has
 * been used: the cached address would belong to the old context.
 *
 * Size limit, in caller terms: the workspace is the plan plus one slot of
 * 256.5 KB (a 128 x 512 fp32 partial and its 128 LSEs) for each of
 * J + G partials, J = B * q_len * ceil(H / 128) jobs and G = the number of
 * CTA pairs (76 on a 152-SM GB300) with the automatic split, or
 * ceil(J * (max_blocks + 4) / split_tiles) with a forced
 * split.  About 255 slots fit, so with the automatic split on a GB300 up
 * to about 179 jobs run: the DeepSeek-V3 decode shape (B = 32, q_len 1,
 * H = 128, J = 32) and B = 64 fp8 decode (J = 64) fit; B = 128 with
 * q_len = 2 (J = 256) is rejected.  Larger requests return
 * MLA_ERR_WORKSPACE, after every argument check of mla_decode_paged (a
 * bad argument still returns MLA_ERR_INVALID_ARG).
 * The library never allocates here: no cudaMalloc, cudaFree or allocating
 * library routine.  Every call shares the one array, so calls that overlap
 * on the GPU (different streams, or devices sharing a context) race and
 * must be serialised by the caller.  Nothing in the array needs to start at
 * zero: the plan is rewritten and every partial is written before it is
 * read on each call.  Arguments and results are those of mla_decode_paged. */
#define MLA_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)

int mla_decode_paged_noalloc(const void *q, int q_dtype, float q_scale,
                             const void *kv_cache, int kv_dtype, float k_scale,
                             const int32_t *block_table,
                             const int32_t *seq_lens, const int32_t *kv_starts,
                             const int32_t *kv_ends, int B, int q_len, int H,
                             int max_blocks, int num_blocks, float sm_scale,
                             int causal, int split_tiles, void *out,
                             int out_dtype, float *lse, mla_stream_t stream);

/* A3 on its own: writes the split plan that mla_decode_paged computes.
 * Jobs are (i, b, head group of 128) in that nesting order (query token
 * outermost: with an even number of CTA pairs, the pairs working on the
 * query tokens of a request then read the same key tiles at about the same
 * time, so the later read finds them in L2); with the tile
 * size tk = 64 tokens (both kv dtypes; kv_dtype is kept so the tile may
 * differ by format), job j covers key tiles [lo/tk, ceil(hi/tk)); the jobs
 * are concatenated into one flat space where a non-empty job takes 4 units
 * (the cost of switching a CTA pair to it, in tile-equivalents, no keys)
 * followed by its tiles, `total` units in all, and CTA group p owns units
 * [p*C, (p+1)*C) with C = split_tiles if > 0, else
 * max(4, ceil(total / n_groups)), i.e. the tiles of every job it meets.
 * plan [4 + 4*(J+1)] int32 receives: [0] total, [1] C, [2] J, [3] number
 * of spans, then unit_prefix[J+1] (units per job, prefix-summed),
 * seg_prefix[J+1] (partial results per job, prefix-summed), job_lo[J+1],
 * job_hi[J+1] (last entries 0).
 * n_groups = 0 uses half the device's SM count. */
int mla_decode_plan(const int32_t *seq_lens, const int32_t *kv_starts,
                    const int32_t *kv_ends, int B, int q_len, int H,
                    int max_blocks, int causal, int kv_dtype, int split_tiles,
                    int n_groups, int32_t *plan, size_t plan_bytes,
                    mla_stream_t stream);

/* ---------------------------------------------------------------------
 * Before the path: rotary position embedding and the cache write
 * [Q-REP] §关键源码片段 mla.py (rotary_emb(positions, q[..., qk_nope_head_dim:],
 * k_pe) runs before mla_attn); [BLOG] §Chunked Prefill 与 LSE Merge (the
 * new tokens' KV is already in the cache when attention runs).  The pages
 * name the rotation but not its variant: this is RoFormer's rotary
 * embedding (Su et al. 2021), pair i of a 64-wide vector turned by
 *   theta = positions[t] * rope_base^(-2i/64):
 *   (a, b) -> (a cos theta - b sin theta, a sin theta + b cos theta),
 * pairs (2i, 2i+1) for MLA_ROPE_INTERLEAVED, (i, i+32) for MLA_ROPE_HALF.
 * Angles and their sine / cosine are computed in fp64, the rotation in
 * fp32, rounded to bf16 once.
 * For each new token t < T:
 *   q_pe [T,H,64] bf16 (NULL: no query) is rotated in place;
 *   k_pe [T,64] bf16 is rotated in place;
 *   row slot_mapping[t] (= block * 64 + offset) of kv_cache
 *   [num_blocks,64,576] receives kv_c[t] [512] bf16 ‖ the rotated k_pe[t]:
 *   the bits for kv_dtype MLA_BF16, e4m3(fp32(x) / k_scale) (RNE,
 *   saturating) for MLA_E4M3.
 * A negative slot is padding and writes nothing; a slot >= num_blocks*64
 * sets MLA_DEVERR_BLOCK_ID and writes nothing.  positions, slot_mapping
 * [T] int32.  1 < rope_base < inf.  T == 0 is a no-op. */
enum mla_rope_layout { MLA_ROPE_INTERLEAVED = 0, MLA_ROPE_HALF = 1 };

int mla_rope_cache_write(void *q_pe, void *k_pe, const void *kv_c,
                         const int32_t *positions, const int32_t *slot_mapping,
                         int T, int H, float rope_base, int rope_layout,
                         void *kv_cache, int kv_dtype, float k_scale,
                         int num_blocks, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * A5/A10  LSE-rescaling merge of partial attention states
 * [BLOG] §Chunked Prefill 与 LSE Merge (merge_attn_states: elementwise
 * O(B*N*V) rescaling) and §DCP 在 Prefill 与 Decode 中的不同角色 (decode
 * combines per-rank partial outputs by LSE weighting).
 *
 * Per row (t,h): m = max_s lse_s; w_s = exp(lse_s - m) (0 if lse_s = -inf)
 *   out = sum_s w_s * part_s / sum_s w_s;  out_lse = m + ln sum_s w_s.
 * All parts -inf: out = 0, out_lse = -inf.  S = 2 is the pages'
 * prefix/suffix form.
 * parts_out [S,T,H,D] (MLA_BF16 or MLA_F32); parts_lse [S,T,H] fp32;
 * out [T,H,D] (MLA_BF16 or MLA_F32); out_lse [T,H] fp32 or NULL.
 * 1 <= S <= 256, D % 8 == 0, D <= 1024. */
int mla_merge_states(const void *parts_out, int parts_dtype,
                     const float *parts_lse, int S, int T, int H, int D,
                     void *out, int out_dtype, float *out_lse,
                     mla_stream_t stream);

/* ---------------------------------------------------------------------
 * A6  Value up-projection
 * [BLOG] §MLA Prefill vs Decode (W_UV expands the latent output back to
 * per-head values); [Q-REP] §关键源码片段 mla.py (output viewed as
 * (tokens, num_heads * v_head_dim)).
 *   out[t,h,v] = sum_l o_lat[t,h,l] * w_uv[h,v,l]   (fp32 accumulate, RNE)
 * o_lat [T,H,512] bf16, w_uv [H,128,512] bf16, out [T,H,128] bf16.
 * T == 0 is a no-op.  1 <= H <= 4096. */
int mla_v_up(const void *o_lat, const void *w_uv, int T, int H, void *out,
             mla_stream_t stream);

/* ---------------------------------------------------------------------
 * A7  Paged gather (cp_gather_cache / gather_and_maybe_dequant_cache)
 * [BLOG] §与非 DCP 的流程对比 and §关于 cp_gather_cache 的命名澄清 (a gather
 * with no dequantisation); [FP8] §实现拆解 3-4 (dequantising gather,
 * seq_starts).
 *   out[cu_out[b] + j] = cast(kv_cache[slot(b, s_b + j)])
 *   for j < cu_out[b+1] - cu_out[b], s_b = seq_starts ? seq_starts[b] : 0.
 * out_dtype == kv_dtype: exact bit copy (bf16 or e4m3 rows).
 * kv_dtype MLA_E4M3, out_dtype MLA_BF16: bf16(RNE)(fp32(e4m3) * k_scale).
 * cu_out [B+1] int32 device; total_rows (host) >= cu_out[B] sizes out
 * [total_rows, 576] and the launch; rows past cu_out[B] are not written.
 * A row with s_b + j >= seq_lens[b] sets MLA_DEVERR_RANGE and is zeroed. */
int mla_gather_cache(const void *kv_cache, int kv_dtype, float k_scale,
                     const int32_t *block_table, const int32_t *seq_lens,
                     const int32_t *seq_starts, const int32_t *cu_out, int B,
                     int max_blocks, int num_blocks, int total_rows,
                     int out_dtype, void *out, mla_stream_t stream);

/* A7  Gather from W interleaved DCP shards and restore sequence order
 * (local cp_gather_cache on every rank + all_gather(dim=0) + reorg_kvcache,
 * fused; the shards live on this one GPU).
 * [BLOG] §与非 DCP 的流程对比 steps 1-4 (rank-major all-gathered buffer,
 * reorg by padded local lengths and every rank's local context lengths).
 * Placement: token t of request r lives on shard k = (t / I) % W at local
 * index j = (t / (I*W)) * I + t % I, in that shard's paged cache.
 *   out[cu_out[r] + t] = cast(shard_cache[k][slot_k(r, j)]),  t < ctx_r
 * with ctx_r = cu_out[r+1] - cu_out[r].
 * shard_caches / shard_block_tables / shard_num_blocks are HOST arrays of
 * W entries (device pointers / host ints); each table is [B, shard_max_blocks].
 * If rank_major_out != NULL it also receives the all-gathered rank-major
 * buffer: row k*sum_p + padded_cu[r] + j holds shard k's local row j of
 * request r, rows j in [n_{r,k}, p_r) are zero, p_r = max_k n_{r,k} =
 * (ctx_r / (I*W)) * I + min(ctx_r % (I*W), I), padded_cu [B+1] int32 device
 * is the prefix sum of p_r and rank_major_rows (host) = W * sum_p.
 * 1 <= W <= 16, 1 <= I. */
int mla_gather_cache_reorg(int W, int interleave,
                           const void *const *shard_caches,
                           const int32_t *const *shard_block_tables,
                           const int *shard_num_blocks, int shard_max_blocks,
                           int kv_dtype, float k_scale, const int32_t *cu_out,
                           int B, int total_rows, int out_dtype, void *out,
                           void *rank_major_out, const int32_t *padded_cu,
                           int rank_major_rows, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * A8  kv_b_proj expansion of latent rows into per-head K and V
 * [BLOG] §MLA Prefill vs Decode (kv_c decompressed through W_UK/W_UV into
 * N heads, K head dim 128+64, V head dim 128) and §与非 DCP 的流程对比 step 5.
 *   K[n,h,0:128]   = sum_l kv[n,l] * w_kvb[h*256 + c, l]         (c < 128)
 *   V[n,h,0:128]   = sum_l kv[n,l] * w_kvb[h*256 + 128 + c, l]
 *   K[n,h,128:192] = kv[n,512:576]                            (k_pe, copied)
 * kv_rows [N,576] bf16 (e.g. mla_gather_cache output), w_kvb [H*256,512]
 * bf16 (nn.Linear layout), k_out [N,H,192] bf16, v_out [N,H,128] bf16.
 * N == 0 is a no-op.  1 <= H <= 1024. */
int mla_expand_kv(const void *kv_rows, const void *w_kvb, int N, int H,
                  void *k_out, void *v_out, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * A9  Prefill multi-head attention with LSE (run_prefill_new_tokens /
 * run_prefill_context_chunk)
 * [BLOG] §Chunked Prefill 与 LSE Merge (new tokens: causal, returns the
 * softmax LSE; context chunks: non-causal).
 * Request b owns query rows [cu_q[b], cu_q[b+1]) and key rows
 * [cu_k[b], cu_k[b+1]); with nq, nk those counts, query i sees keys
 *   j < nk                       (causal = 0)
 *   j <= i + nk - nq             (causal = 1, bottom-right aligned)
 *   s_j = sm_scale * q.k_j;  lse = ln sum exp(s_j);  out = softmax . V
 * q [Tq,H,192], k [Nk,H,192], v [Nk,H,128] bf16; out [Tq,H,128] bf16;
 * lse [Tq,H] fp32.  cu_q / cu_k [B+1] int32 device; max_q_len (host) bounds
 * every nq and sizes the launch.  A query that sees no key gets out = 0,
 * lse = -inf. */
int mla_prefill_attn(const void *q, const void *k, const void *v,
                     const int32_t *cu_q, const int32_t *cu_k, int B, int Tq,
                     int Nk, int H, int max_q_len, int causal, float sm_scale,
                     void *out, float *lse, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * Block-scaled 8-bit cache
 * An e4m3 cache [num_blocks,64,576] with one fp32 scale for each block of
 * scale_block tokens (16, 32 or 64) of its one latent head: kv_scales
 * [num_blocks, 64/scale_block], element (s, c) of the cache standing for
 *   kv_scales[s/64, (s%64)/scale_block] * e4m3(kv_cache[s, c])
 * (s = block*64 + offset).  No calibration is needed: mla_rope_cache_append
 * finds the scales, mla_decode_paged_scaled and mla_gather_cache_scaled
 * read them.  Scales are >= 0 and at most 2^120; 0 stands for rows of zeros
 * (the decode takes 2^-100 for anything below it).  Any other value is no
 * scale: the elements of its block are NaN.
 *
 * Append: mla_rope_cache_write for this cache.  For each new token t < T
 *   q_out[t,h,:] = R(positions[t]) q_pe[t,h,:]      (h < H)
 *   k_out[t,:]   = R(positions[t]) k_pe[t,:]
 * with the rotation R of mla_rope_cache_write, and row slot_mapping[t] of
 * the cache receives kv_c[t] || k_out[t].  For every block that the call
 * writes to, with A the largest finite |element| of its new rows and s the
 * block's scale (0 if the call writes the block's first row: it begins
 * afresh; likewise if s is no scale),
 *   s' = max(s, 2^max(-100, ceil(log2(A / 448))))
 * becomes its scale, the new rows are stored as e4m3(x / s'), and if
 * 0 < s < s' the block's other rows are stored again as e4m3(code * (s/s'))
 * (a power of two where the append found s: only values that fall below the
 * e4m3 normal range are rounded).  Rounding is to nearest even, infinities
 * saturate, NaN stays NaN.  Rows of blocks that the call does not write to
 * keep their bits.  Tokens of a block may stand anywhere in the call; where
 * a slot comes up twice the later token's row stays.  Calls that write to the
 * same block follow one another on a stream.  A negative slot is
 * padding: its q and k are rotated and nothing is stored; a slot >=
 * num_blocks*64 does the same and sets MLA_DEVERR_BLOCK_ID.
 *
 * q_pe [T,H,64] bf16 with strides q_stride_t, q_stride_h (elements), NULL:
 * no query; k_pe [T,64] with row stride k_stride; kv_c [T,512] with row
 * stride c_stride (all rows start on 16 bytes: the strides are multiples of
 * 8, so slices of one projection's output are read in place).  q_out
 * [T,H,64], k_out [T,64] contiguous, or NULL: rotated in place.  positions,
 * slot_mapping [T] int32.  1 < rope_base < inf, 1 <= H <= 4096 with a
 * query, num_blocks < 2^25; T * ceil(H / 128) < 2^31 - 256.  T == 0 is a
 * no-op. */
int mla_rope_cache_append(void *q_pe, int64_t q_stride_t, int64_t q_stride_h,
                          void *k_pe, int64_t k_stride, const void *kv_c,
                          int64_t c_stride, const int32_t *positions,
                          const int32_t *slot_mapping, int T, int H,
                          float rope_base, int rope_layout, void *q_out,
                          void *k_out, void *kv_cache, float *kv_scales,
                          int scale_block, int num_blocks,
                          mla_stream_t stream);

/* Gather: mla_gather_cache out of a block-scaled cache,
 *   out[cu_out[b] + j] = bf16(RNE)(scale * fp32(e4m3))
 * rows, ranges and errors as there. */
int mla_gather_cache_scaled(const void *kv_cache, const float *kv_scales,
                            int scale_block, const int32_t *block_table,
                            const int32_t *seq_lens,
                            const int32_t *seq_starts, const int32_t *cu_out,
                            int B, int max_blocks, int num_blocks,
                            int total_rows, void *out, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * Decode with a sliding window and sinks, and over a block-scaled cache
 * For request b, query token i < q_len at position p = seq_lens[b] - q_len
 * + i (the new tokens are in the cache), head h:
 *   visible: j <= p and (window == 0 or j > p - window or j < sinks)
 *   s_j  = sm_scale * q_deq[b,i,h,:] . K_j
 *   lse[b,i,h] = ln sum_j exp(s_j),  out[b,i,h,:] = sum_j exp(s_j - lse) V_j
 * over the visible j; no visible key (p < 0): out = 0, lse = -inf.  K_j, V_j,
 * q_deq, slots and layouts as in mla_decode_paged; in the scaled form kv_deq
 * takes the block's scale in place of k_scale and q is e4m3.
 * Over an e4m3 cache a weight is held to 2^-8 of itself.  One that (times its
 * key's scale) is less than the largest of its tile of 128 keys may be off by
 * 2^-8 of that one, at most by 2^-3 of itself, and counts as 0 below 2^-11 of
 * it (in tiles whose largest is 2^-27 of the row's or less, below 2^-38 of the
 * row's); lse has all of them.  Scores are fp32: sm_scale * |q_deq . K| < 2^127.
 * Cache rows that no query token of a request sees (past seq_lens, behind
 * the window) are never used, whatever they hold, and block-table entries
 * of pages without a visible key are not read.
 * window >= 0 (0: every earlier token), sinks >= 0 (of no effect without a
 * window).  workspace: mla_decode_window_workspace_size(B, q_len, H,
 * max_blocks*64, window, sinks, split_tiles) bytes, 16-byte aligned, written
 * before it is read (calls on different streams need workspaces of their
 * own); 0 bytes, and workspace may be NULL, where no request can have more
 * than a few tiles.  split_tiles as in mla_decode_paged, in tiles of 128
 * (e4m3) or 64 (bf16) tokens.  Limits as there; k_scale of an e4m3 cache from
 * 2^-100 to 2^120; B * ceil(q_len * H / 128) * (pages + 6) < 2^31, with pages
 * the most that a request can have (max_blocks, or window + sinks in pages). */
int mla_decode_window_workspace_size(int B, int q_len, int H, int max_seq_len,
                                     int window, int sinks, int split_tiles,
                                     size_t *bytes);

int mla_decode_paged_window(const void *q, int q_dtype, float q_scale,
                            const void *kv_cache, int kv_dtype, float k_scale,
                            const int32_t *block_table,
                            const int32_t *seq_lens, int B, int q_len, int H,
                            int max_blocks, int num_blocks, float sm_scale,
                            int window, int sinks, int split_tiles, void *out,
                            int out_dtype, float *lse, void *workspace,
                            size_t ws_bytes, mla_stream_t stream);

int mla_decode_paged_scaled(const void *q, float q_scale, const void *kv_cache,
                            const float *kv_scales, int scale_block,
                            const int32_t *block_table,
                            const int32_t *seq_lens, int B, int q_len, int H,
                            int max_blocks, int num_blocks, float sm_scale,
                            int window, int sinks, int split_tiles, void *out,
                            int out_dtype, float *lse, void *workspace,
                            size_t ws_bytes, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * Decode of a tree of drafted tokens
 * Speculative decode where a request's new tokens are not a chain: their rows
 * are the last n = tree_lens[b] of its seq_lens[b] (n = q_len where tree_lens
 * is NULL), behind a context of c = seq_lens[b] - n tokens, in any order.
 * For query token i < n, head h:
 *   visible: j < c, or j = c + t with t < n and bit t of the word
 *            tree_mask[b * mask_stride + i] set
 *   s_j, lse, out as in mla_decode_paged_window
 * Nothing is implied by the order: a token that sees itself has its own bit
 * set, a tree has those of the token and of all above it, a chain has (2 << i)
 * - 1; any other mask will do.  Keys at a negative position (n > seq_lens[b])
 * are not there.  A row that sees no key, and rows i >= n (whose words and
 * queries may hold anything): out = 0, lse = -inf.
 * mask_stride: q_len or more, or 0: one tree for all requests (tree_lens
 * then cuts it).  tree_lens[b] outside [0, q_len] sets MLA_DEVERR_SEQ_LEN and
 * counts as 0.  kv_scales [num_blocks, 64/scale_block]: a block-scaled e4m3
 * cache (k_scale is not used), else NULL.  Precision, limits, split_tiles, the
 * workspace's use and what is not read as in mla_decode_paged_window; it has
 * mla_decode_tree_workspace_size(B, q_len, H, max_blocks*64, split_tiles) bytes.
 * How a call is cut goes by max_blocks: a table far wider than its sequences
 * costs short calls up to 3 us. */
int mla_decode_tree_workspace_size(int B, int q_len, int H, int max_seq_len,
                                   int split_tiles, size_t *bytes);

int mla_decode_paged_tree(const void *q, int q_dtype, float q_scale,
                          const void *kv_cache, int kv_dtype, float k_scale,
                          const float *kv_scales, int scale_block,
                          const int32_t *block_table, const int32_t *seq_lens,
                          const int32_t *tree_lens, const uint64_t *tree_mask,
                          int64_t mask_stride, int B, int q_len, int H,
                          int max_blocks, int num_blocks, float sm_scale,
                          int split_tiles, void *out, int out_dtype, float *lse,
                          void *workspace, size_t ws_bytes,
                          mla_stream_t stream);

/* ---------------------------------------------------------------------
 * Pages of the cache: who has them, and their copies
 * A cache's pages belong to sequences, rows of block_table [B,max_blocks] of
 * which the first ceil(seq_lens[b] / 64) entries are pages; refs [num_blocks]
 * int32 (16-byte aligned) says how many entries hold each page, 0: it is free.
 * The calls below keep the three in step, on the device and in a stream's
 * order; calls on the same state follow one another on a stream.  Free pages
 * are taken lowest first, so the result depends on the state alone.
 *
 * A page that several entries hold is not to be written: a sequence that was
 * shortened to end inside one is continued by a fork of it, which has a last page
 * of its own.
 *
 * Pools are what a page has in memory: for every layer its cache [num_blocks,
 * 64,576], its block scales, or anything else of num_blocks rows, each given
 * once (no two share memory).  pools and page_bytes are HOST arrays of n_pools
 * (0 to 200) device pointers and of a page's bytes in each: multiples of 4;
 * pools whose page is a multiple of 16 and 1024 or more start on 16 bytes, the
 * others on 4.  num_blocks < 2^25.
 * 1 <= B <= 8192, 1 <= max_blocks <= 2^24, B * max_blocks < 2^31
 * (mla_cache_accept: any B >= 1).
 *
 * Copy: page dst[k] of every pool becomes page src[k], k < n (int32 [n]).
 * A negative id is padding, and so is a page onto itself; an id >= num_blocks
 * sets MLA_DEVERR_BLOCK_ID, and the pair is left out.  Of equal destinations
 * the last one's pair counts.  A destination that is another pair's source is
 * not written and sets MLA_DEVERR_PAGES.  refs and tables are the caller's
 * business here.  0 <= n <= 65536.  Every pair looks at all others, which takes 24 us of 4096
 * pairs, 250 of 16384 and 3.7 ms of 65536: long lists are better cut. */
int mla_cache_copy(void *const *pools, const int64_t *page_bytes, int n_pools,
                   int num_blocks, const int32_t *src, const int32_t *dst,
                   int n, mla_stream_t stream);

/* Resize: sequence b gets the length new_lens[b] [B].  Entries behind it are
 * released (refs - 1, the entry -1: a page that nobody else holds is free);
 * then entries that it lacks get the lowest free pages, sequences in their
 * order, those released by this call among them.  So a new sequence grows from
 * 0, a finished one goes to 0, and a length inside the last page only changes.
 * A sequence whose pages, counted with those for the ones in front of it, are
 * more than are free keeps its length and pages and sets MLA_DEVERR_PAGES;
 * a length < 0 or > max_blocks * 64, old or new: unchanged, MLA_DEVERR_SEQ_LEN.
 * An entry that is no page sets MLA_DEVERR_BLOCK_ID, one that was free already
 * MLA_DEVERR_PAGES.  Pages' contents stay as they are. */
int mla_cache_resize(int32_t *refs, int num_blocks, int32_t *block_table,
                     int32_t *seq_lens, const int32_t *new_lens, int B,
                     int max_blocks, mla_stream_t stream);

/* Fork: for i < n (at most 8192) sequence children[i], of length 0, becomes the
 * tokens of parents[i]: full pages are shared (refs + 1), of a last page that
 * is not full the tokens are copied, in every pool, into a free page: of the
 * first n_by_rows pools, whose pages are 64 rows of equal size (of 4-byte words),
 * their rows; of the others (scales) the page.
 * Parents are as they were before the call.  Left out, with MLA_DEVERR_PAGES:
 * a child that has tokens or came up before, and from where free pages run
 * out on every fork that needs one; a row outside [0, B): MLA_DEVERR_RANGE; a
 * parent's length out of range: MLA_DEVERR_SEQ_LEN.  Where a parent's entry is
 * no page (MLA_DEVERR_BLOCK_ID), or a free one (MLA_DEVERR_PAGES), the child's
 * is -1: nothing is shared, copied or taken for it.
 * workspace: mla_cache_fork_workspace_size(n) bytes, 4-byte aligned. */
int mla_cache_fork_workspace_size(int n, size_t *bytes);

int mla_cache_fork(void *const *pools, const int64_t *page_bytes, int n_pools,
                   int n_by_rows, int32_t *refs, int num_blocks,
                   int32_t *block_table, int32_t *seq_lens, int B, int max_blocks,
                   const int32_t *parents, const int32_t *children, int n,
                   void *workspace, size_t ws_bytes, mla_stream_t stream);

/* Compact: with N pages in use, those from page N on move, in their order, to
 * the free pages below N, in theirs: copied in every pool, their refs and all
 * entries of the B sequences with them.  *n_live (device) becomes N: pages
 * from N on are free.  What they held stays.  Every page in use is held by
 * these sequences, or by entries that the caller has elsewhere and updates
 * himself.  An entry that is no page sets MLA_DEVERR_BLOCK_ID, one that is
 * free and not below N MLA_DEVERR_PAGES; both stay.  A length out of range sets
 * MLA_DEVERR_SEQ_LEN and counts as the nearest in it.
 * workspace: mla_cache_compact_workspace_size(num_blocks) bytes, 8-byte
 * aligned. */
int mla_cache_compact_workspace_size(int num_blocks, size_t *bytes);

int mla_cache_compact(void *const *pools, const int64_t *page_bytes,
                      int n_pools, int32_t *refs, int num_blocks,
                      int32_t *block_table, const int32_t *seq_lens, int B,
                      int max_blocks, int32_t *n_live, void *workspace,
                      size_t ws_bytes, mla_stream_t stream);

/* Accept: of the n = tree_lens[b] (NULL: q_len) drafted tokens that end
 * sequence b (mla_decode_paged_tree) keeps those of its path, k =
 * path_lens[b] of them: row c + path[b * path_width + i] of every layer's cache
 * becomes row c + i, i < k, c = seq_lens[b] - n.  A path ascends.  new_lens[b]
 * [B] = c + k (mla_cache_resize then takes the length and the pages behind).
 * Rows behind c + k, and seq_lens, stay as they are.  The rows' pages are the
 * sequence's own.
 * kv_scales (a HOST array of n_pools device pointers, each [num_blocks,
 * 64/scale_block], or NULL): block-scaled e4m3 caches.  The rows are then
 * appended to their new blocks by the rule of mla_rope_cache_append, from what
 * they stand for: with A the largest finite of a block's new rows and s its
 * scale (0 if its first row is among them, or s is no scale), s' = max(s,
 * 2^max(-100, ceil(log2(A / 448)))); a row of scale r is stored as e4m3(code *
 * (r / s')), the block's other rows, where s grew, as e4m3(code * (s / s')).
 * A path that is no such list, k > n or path_width, or c < 0 with k > 0:
 * MLA_DEVERR_RANGE; lengths out of range: MLA_DEVERR_SEQ_LEN; an entry that is
 * no page: MLA_DEVERR_BLOCK_ID: the sequence stays as it is, new_lens[b] =
 * seq_lens[b] (as where c < 0 and k = 0).  pools [num_blocks,64,576] of kv_dtype, 16-byte
 * aligned.  1 <= q_len, path_width <= 64.  new_lens shares no memory with the
 * arrays that are read. */
int mla_cache_accept(void *const *pools, int kv_dtype, float *const *kv_scales,
                     int scale_block, int n_pools, int num_blocks,
                     const int32_t *block_table, const int32_t *seq_lens,
                     const int32_t *tree_lens, int q_len, const int32_t *path,
                     int path_width, const int32_t *path_lens, int B,
                     int max_blocks, int32_t *new_lens, mla_stream_t stream);

/* ---------------------------------------------------------------------
 * Prefill attention with a sliding window and sinks
 * mla_prefill_attn, causal, where query i of a request with nq queries and
 * nk keys stands at p = i + nk - nq and sees the keys
 *   j <= p and (j > p - window or j < sinks),     window >= 1, sinks >= 0.
 * The window is the same whether the keys before the queries are new tokens
 * or gathered context, so one call attends to both.  What a query does not
 * see does not reach its row, NaN and infinities included, in rows behind
 * cu_k[B] too (a NaN or infinite value that some queries of its key tile do
 * not see makes the call take about twice as long).  A request whose rows are not
 * all in [0, Tq) and [0, Nk) sets MLA_DEVERR_RANGE and is left out.
 * B * H * ceil(max_q_len / 256) < 2^31 - 1024. */
int mla_prefill_attn_window(const void *q, const void *k, const void *v,
                            const int32_t *cu_q, const int32_t *cu_k, int B,
                            int Tq, int Nk, int H, int max_q_len, int window,
                            int sinks, float sm_scale, void *out, float *lse,
                            mla_stream_t stream);

/* ---------------------------------------------------------------------
 * Host staging of a step's inputs and results
 * [BLOG] §MLA Prefill vs Decode (each decode step takes the new tokens'
 * queries in and hands the attention output on).  No page defines the
 * transfer itself.
 * Copies `bytes` from src to dst, where exactly one of the two is
 * page-locked, device-mapped HOST memory (cudaHostAlloc / cudaHostRegister,
 * e.g. a pinned torch tensor) and the other is memory of the current
 * device; the SMs load and store over the host link (no copy engine), so
 * the call is a kernel launch like every other entry point (asynchronous on
 * `stream`, capturable in a CUDA graph; it waits for the previous kernel in
 * the stream before reading src).  Both pointers 16-byte aligned, bytes a
 * multiple of 16.  bytes == 0 is a no-op.
 * Pageable host memory, host-to-host, device-to-device or another device's
 * memory: MLA_ERR_INVALID_ARG, nothing launched. */
int mla_stage_copy(void *dst, const void *src, size_t bytes, mla_stream_t stream);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* MLA_GB300_H_ */
