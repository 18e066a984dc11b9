// Paged latent decode with a sliding window and sinks, over a bf16, an e4m3
// or a block-scaled e4m3 cache (mla_decode_paged_window, _scaled).
//
// Rows and keys.  The q_len * H query rows of a request (query token outer,
// head inner) all attend to the same latent rows, so they are taken in groups
// of 128: per tile of T keys (e4m3: 128, bf16: 64) S = Q K^T is a dense
// [128 x T x 576] product and O += P V a [128 x 512 x T] one.  A request's keys
// are a list of 64-token pages, the sinks' pages and then those from the
// window's first key to the last query; only the list's pages are loaded.  Each
// row masks the keys that it does not see.
//
// CTA pairs.  The fp32 output of 128 rows x 512 columns would fill one SM's
// tensor memory, so two CTAs of a cluster run each product as one
// tcgen05 MMA of cta_group::2 with M = 128: CTA c holds rows [64c, 64c + 64)
// of Q, S, P and O (S and O in the layout of that shape: lanes 0..63 the
// first half of the columns, lanes 64..127 the second), for Q K^T half c of
// the tile's keys, and for P V the value columns [256c, 256c + 256) of all
// of them.  Scores and probabilities never cross
// the pair; each key row is fetched twice, once as a key by its page's CTA
// and once, by then from L2, as a value by halves.  Measured on the GB300: a
// 32-byte K step costs 32 cycles at N = 128 (Q K^T: 18 or 36 per tile) and 66
// at N = 256 (P V: 16 per tile in either format).
//
// e4m3 probabilities.  P as one e4m3 value would be off by up to 2^-4 and the
// output with it; P is held as the sum of two values, hi = e4m3(p) and lo =
// e5m2(p - hi), at twice the P V steps: off by at most 2^-8 p where p is 2^-6 or
// more, by 2^-14 (and 2^-3 p) below, and by all of it below 2^-17.  So that
// thousands of small p do not lose a part of their weight together behind a row's
// few large ones (a sink 10 nats above 16384 keys of one score: 34 % of their
// weight with lo = e4m3), a row's reference also follows its tiles down: where a
// tile's largest p falls below 2^-6, to 1, with O (fp32) scaled up; at most 2^16
// below the highest, so 2^-21 of the row's largest p and more are held like that.
// A weight is then off by 2^-8 of itself; where it (times its key's scale) is less
// than the largest of its 128 keys, by up to 2^-8 of that one or 2^-3 of itself,
// whichever is less; and lost below 2^-11 of that one.  None of it grows with the
// number of keys.
// (e4m3 for both: half the error on rows whose scores are alike, 7e-4 instead of
// 1.3e-3 of an output's rms where its own rounding is 1.7e-3.  e5m2 for both
// has the range without the steps down, at 2.3e-3.)
//
// Block scales.  With sigma the scale of a key's block and c = sm_scale *
// log2(e) * q_scale, the scores in the log2 domain are sigma * c * raw, and
// P' = sigma * 2^(s - m) = 2^(raw * (sigma c) + log2 sigma - m) goes against
// the raw codes of V: one FMA and one exponential per score whatever the
// scales.  m follows the largest s + log2 sigma.  The normaliser has a unit of
// its own, n = the largest s of the thread's keys so far: sum 2^(s - n) is the
// sum over the blocks of 2^(m - log2 sigma - n) sum P'.  Where the keys with
// the weight have a scale 2^100 below those that m follows, P' would vanish in
// fp32 and their scores are taken again from tensor memory.
//
// Warps: 0 walks the split plan, publishes the segments and loads Q and K,
// 1 issues the MMAs (leader CTA), 2 loads V, 4..11 turn scores into
// probabilities (two groups taking the tiles in turn, one row and half of the
// tile's keys per thread) and write the results.  Lazy rescaling: O is rescaled
// when a row's reference would be exceeded by more than 2^kLazy (e4m3: or a tile's
// largest p is below 2^kLow).
//
// Split: every row group of a request is a job of its list's tiles plus
// kJobCost units for the switch; jobs lie end to end and pair p takes units
// [pC, (p+1)C).  Each CTA works the plan out for itself from the lengths
// (no plan kernel).  A job that is cut leaves partials in the workspace,
// which a merge kernel combines: at most two per span, whatever the number
// of jobs.  Partials for a bf16 output are fp16 with a unit for every row and
// 128 columns: off by 2^-11 of themselves, or 2^-39 of the largest of these,
// which adds nothing to the output's own rounding (bf16 partials took a batch's
// error from 2.3e-3 to 2.7e-3 of its rms; fp32 ones are twice the bytes, 2 to 5
// us of a merge).
//
// What bounds it now (each key row takes 128 x 1088 x 2 operations a row group;
// times of graph replays, in brackets of calls on changing inputs): 64 e4m3
// requests of up to 16384 tokens 94 us (100), at 1.6 of the 1.9 PFLOP/s that a
// bf16 product reaches, near the 1632 cycles of a tile's MMAs; 128 bf16 requests
// of two tokens and a window of 4096 147 us (155), 1.14 PFLOP/s, where Q K^T of 64
// keys takes as long as one of 128; one e4m3 request of 131072 tokens 35.6 us (35.0),
// the smallest calls 8.4: 3 us until the first keys are there, 4 from the last
// scores to the results, and 3 for the merge where there is one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <climits>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "merge_row.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;              // warps 4..11
constexpr int kMinPages = 6;               // smallest automatic span, in pages (4 and 8 measure the same)
// What switching to a job costs, in pages: with 4 / 6 / 8 of them the mixed
// e4m3 batch (64 requests) takes 93.6 / 91.2 / 90.5 us, the speculative bf16
// batch (128 requests, two row groups each) 145.8 / 146.2 / 148.4.
constexpr int kJobPages = 6;
// Jobs that cannot have more pages than this are not cut: each is one pair's
// from end to end, written directly, and no merge kernel follows.  Two e4m3
// requests of 130 tokens: 8.0 us, cut 10.3; a window of 128: 8.8, cut 11.5; but
// 32 requests of 18 pages: 24.8, cut 22.4.
constexpr int kSoloPages = 6;
constexpr int kSegSlots = 4;
constexpr uint32_t kColO = 0, kColS = 256;   // O [0,256), then the S tiles
constexpr int kSBufs = 4;                    // Q K^T runs two tiles ahead of P V

// What differs between the formats.  K and V come through rings of slots.
// The bf16 tile is one page: its query takes 72 KB, and the other 152 KB then
// hold two tiles of keys and values, so that a tile's values are on their way
// while the last one's are read.  (A two-page tile runs Q K^T at twice the
// rate, but there is room for one only, in slots that wait 2500 cycles for
// their next load: the speculative batch took 140 us instead of 146, a window
// of 128 10.3 instead of 8.8, the batch of 32 the same.)
template <bool FP8>
struct Fmt {
  static constexpr int kEsz = FP8 ? 1 : 2;
  static constexpr int kPages = FP8 ? 2 : 1;               // pages of a tile
  static constexpr int kTile = kPages * kPage;             // its keys: 128 / 64
  static constexpr int kMine = kTile / 2;                  // keys of one softmax thread
  static constexpr int kMinUnits = (kMinPages + kPages - 1) / kPages;
  static constexpr int kJobCost = kJobPages / kPages;      // in tiles, as all units
  static constexpr int kCols = 128 / kEsz;                 // columns of a 128-byte box row
  static constexpr int kQBytes = 64 * kDqk * kEsz;         // 64 query rows: 36 / 72 KB
  static constexpr int kKRows = kTile / 2;                 // key rows of one CTA
  static constexpr int kKBox = kKRows * 128;
  static constexpr int kBoxes = FP8 ? 4 : 9;               // whole box columns of a cache row
  // A slot is one load: what a loading warp does for one (wait, expect, issue)
  // takes about 500 cycles, so three loads a tile set the pace themselves.
  static constexpr int kKSlotBytes = kKRows * kDqk * kEsz; // 36 KB
  static constexpr int kKSlots = 2;
  static constexpr int kVTok = kPage;                      // keys of a V slot
  static constexpr int kVBoxes = 256 / kCols;              // 2 / 4
  static constexpr int kVBox = kVTok * 128;                // 8 KB
  static constexpr int kVSlotBytes = kVBoxes * kVBox;      // 16 / 32 KB
  static constexpr int kVPer = kPages;                     // slots of a tile
  static constexpr int kVSteps = kVTok * kEsz / 32;        // K steps of a slot: 2 / 4
  static constexpr int kVSlots = FP8 ? 5 : 2;
  static constexpr int kPBytes = 64 * 128 * (FP8 ? 2 : 1); // hi and lo, or bf16: 128 bytes a row
  static constexpr int kPBufs = 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kOffQ + kQBytes;
  static constexpr int kOffV = kOffK + kKSlots * kKSlotBytes;
  static constexpr int kOffP = kOffV + kVSlots * kVSlotBytes;
  // [2][128] maxima, [2][64] references, [256] sums, e4m3: [256] units of the sums
  static constexpr int kOffX = kOffP + kPBufs * kPBytes;
  static constexpr int kOffSeg = kOffX + (256 + 128 + 256 + (FP8 ? 256 : 0)) * 4;
  static constexpr int kOffBars = kOffSeg + kSegSlots * 32;
  static constexpr int kBarBytes = 384;
  static constexpr int kSmem = kOffBars + kBarBytes;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
  static_assert(kKSlotBytes % 1024 == 0 && kQBytes % 1024 == 0 && kKBox % 1024 == 0, "swizzled tiles");
  // p' of a row's largest key after the reference moved, as a power of two
  static constexpr float kTop = FP8 ? 5.f : 0.f;
  // p' is at most 2^kLazy before it moves again: e4m3 holds 448 > 2^8.75
  static constexpr float kLazy = FP8 ? 8.75f : 16.f;
  // e4m3: p' of a tile's largest key at which the reference follows it down, at
  // most kDepth below the highest one (-3 in place of -6: on 16384 keys of a
  // deviation of 3 nats 57 passes over O in 128 tiles and not 21, and no less error;
  // 64 requests of 8192 tokens at a deviation of 1.5 / 3 / 5 nats and more: 85.7 /
  // 97.2 / 109 us, 85.0 / 94.0 / 98.5 without going down)
  static constexpr float kLow = -6.f, kDepth = 16.f;
};

struct WindowArgs {
  const float *scales;          // nullptr: k_scale
  int sb_shift;                 // log2(tokens per scale)
  float k_scale;                // cache value of code 1 (bf16: 1)
  float scale_log2, scale_pre;  // sm_scale * log2(e) * q_scale as a product, so that it is in range
  const int32_t *block_table, *seq_lens;
  int B, q_len, H, max_blocks, num_blocks, window, sinks;
  int RG, forced, solo;
  int groups, group_jobs;       // row groups planned apart (RG or 1), jobs of each
  int spans_at_once;            // pairs of a group
  int group_spans;              // most spans of a group
  void *out;
  int out_f32;
  float *lse;
  int *ws_head;                 // C of each group; then per job {first unit, end unit}
  void *ws_o;                   // [slots, 128, 512] fp32, or fp16 for a bf16 output
  float *ws_lse;                // [slots, 128]
  float *ws_unit;               // [slots, 128, 2, 2]: what 1 of the fp16 stands for, by 128 columns (1, 3; 2, 4)
  int *err;
};

// One job: 128 rows of a request over its list of pages.
struct Job {
  int p0, p1;                   // positions of its first and last query
  int lo_page, sink_pages, pages;
  __device__ __forceinline__ int tiles(int per) const { return (pages + per - 1) / per; }
  // page of the list's entry i
  __device__ __forceinline__ int page(int i) const {
    return i < sink_pages ? i : i - sink_pages + lo_page;
  }
};

__device__ __forceinline__ Job job_of(int rg, int len, const WindowArgs &a) {
  Job j;
  int i0 = 0, i1 = a.q_len - 1;               // (one group: no divisions)
  if (a.RG > 1) {
    i0 = rg * 128 / a.H;
    i1 = min(i1, (rg * 128 + 127) / a.H);
  }
  j.p0 = len - a.q_len + i0;
  j.p1 = len - a.q_len + i1;
  const int lo = a.window ? max(0, j.p0 - a.window + 1) : 0;
  j.lo_page = lo / kPage;
  j.sink_pages = min((min(a.sinks, lo) + kPage - 1) / kPage, j.lo_page);
  j.pages = j.p1 < 0 ? 0 : j.sink_pages + j.p1 / kPage + 1 - j.lo_page;
  return j;
}

__device__ __forceinline__ int length_of(int b, const WindowArgs &a, bool tell) {
  const int len = __ldg(a.seq_lens + b), most = a.max_blocks * kPage;
  if (tell && (len < 0 || len > most)) raise_error(a.err, MLA_DEVERR_SEQ_LEN);
  return min(max(len, 0), most);
}

template <bool FP8>
__device__ __forceinline__ int tiles_of(int j, const WindowArgs &a, int &len) {
  const int rg = a.RG > 1 ? j / a.B : 0;
  len = length_of(j - rg * a.B, a, blockIdx.x == 0 && rg == 0);
  return job_of(rg, len, a).tiles(Fmt<FP8>::kPages);
}

struct Seg {
  int b, rg, len;
  int tile0, ntiles;            // ntiles 0: a job without a key (uncut jobs only); < 0: the end
  int whole, slot;
};

__device__ __forceinline__ int warp_incl_scan(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The segments of one CTA pair, found by a whole warp.  Lane k holds the
// jobs [k*per, (k+1)*per) in sum for the search of a span's first job, and
// job base + k of the 32 that are being walked.
//
// even: where every job can be cut into parts of at most C tiles with no more
// parts than pairs, each pair has one part of one job instead of C units of
// what lies end to end: nobody then switches jobs (a second segment ends
// about 4 us after a first one of the same tiles).  A part is the unit, C = 1.
template <bool FP8>
struct Walk {
  static constexpr int kHeld = 3;   // jobs of a lane that fit (the pairs are fewer than 96)
  int J, job0, per, lane_excl, total, C, span, span_lo, span_hi;
  int base, k, len, units, excl;
  int even;                         // C of the test, or 0
  int slot0;
  bool open;

  __device__ int units_of(int tiles) const {
    if (even) return (tiles + even - 1) / even;
    return tiles > 0 ? tiles + Fmt<FP8>::kJobCost : 0;
  }
  __device__ void init(const WindowArgs &a, int lane) {
    const int pair = blockIdx.x >> 1, group = pair / a.spans_at_once;
    J = group < a.groups ? a.group_jobs : 0;
    job0 = group * J;
    slot0 = group * a.group_spans;
    span = pair - group * a.spans_at_once;
    per = (J + 31) / 32;
    even = 0;
    int sum = 0, held[kHeld];
    len = 0;
    if (per <= kHeld) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        held[i] = i < per && lane * per + i < J ? tiles_of<FP8>(job0 + lane * per + i, a, len) : 0;
        sum += units_of(held[i]);
      }
    } else {
      for (int j = lane * per; j < min(J, (lane + 1) * per); ++j)
        sum += units_of(tiles_of<FP8>(job0 + j, a, len));
    }
    total = __reduce_add_sync(0xffffffffu, sum);
    C = a.forced > 0 ? a.forced : max(Fmt<FP8>::kMinUnits, (total - 1) / a.spans_at_once + 1);
    if (a.forced == 0 && J <= a.spans_at_once && per <= kHeld) {
      even = C;
      int parts = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) parts += units_of(held[i]);
      const int all = __reduce_add_sync(0xffffffffu, parts);
      if (all <= a.spans_at_once) {
        sum = parts;
        total = all;
        C = 1;
      } else {
        even = 0;
      }
    }
    lane_excl = warp_incl_scan(sum, lane) - sum;
    units = sum;                // (one job a lane: the walk's window is there already)
    excl = lane_excl;
    base = 0;
    open = false;
    if (span == 0 && J > 0 && (blockIdx.x & 1) == 0 && lane == 0) a.ws_head[group] = C;
  }
  __device__ void init_solo(const WindowArgs &a) {
    J = a.B * a.RG;
    span = blockIdx.x >> 1;
  }
  // Uncut: jobs span, span + pairs, ...
  __device__ bool next_solo(const WindowArgs &a, Seg &s) {
    if (span >= J) return false;
    s.rg = a.RG > 1 ? span / a.B : 0;
    s.b = span - s.rg * a.B;
    s.len = length_of(s.b, a, s.rg == 0);
    s.tile0 = 0;
    s.ntiles = job_of(s.rg, s.len, a).tiles(Fmt<FP8>::kPages);
    s.whole = 1;
    s.slot = 0;
    span += a.spans_at_once;
    return true;
  }
  __device__ void load(const WindowArgs &a, int at, int before, int lane) {
    base = at;
    k = 0;
    units = 0;
    len = 0;
    if (base + lane < J) units = units_of(tiles_of<FP8>(job0 + base + lane, a, len));
    const int incl = warp_incl_scan(units, lane);
    excl = before + incl - units;
  }
  __device__ bool next(const WindowArgs &a, Seg &s, int lane) {
    while (true) {
      if (!open) {
        if (static_cast<int64_t>(span) * C >= total) return false;
        span_lo = span * C;
        span_hi = min(total, span_lo + C);
        // the last lane whose jobs begin at or before the span
        const uint32_t le = __ballot_sync(0xffffffffu, lane_excl <= span_lo);
        const int own = 31 - __clz(le);
        if (per == 1) k = own;
        else load(a, own * per, __shfl_sync(0xffffffffu, lane_excl, own), lane);
        open = true;
      }
      if (k == 32) load(a, base + 32, __shfl_sync(0xffffffffu, excl + units, 31), lane);
      const int j = job0 + base + k;
      const int t0 = __shfl_sync(0xffffffffu, excl, k & 31);
      const int n = __shfl_sync(0xffffffffu, units, k & 31);
      const int l = __shfl_sync(0xffffffffu, len, k & 31);
      if (base + k >= J || t0 >= span_hi) {
        span += a.spans_at_once;
        open = false;
        continue;
      }
      ++k;
      const int first = t0 + (even ? 0 : Fmt<FP8>::kJobCost), end = t0 + n;
      const int u0 = max(span_lo, first), u1 = min(span_hi, end);
      if (n == 0 || u1 <= u0) continue;
      s.rg = a.RG > 1 ? j / a.B : 0;
      s.b = j - s.rg * a.B;
      s.len = l;
      s.tile0 = u0 - first;
      s.ntiles = u1 - u0;
      if (even) {               // part tile0 of n, of sizes that differ by one at most
        const int tiles = job_of(s.rg, l, a).tiles(Fmt<FP8>::kPages), small = tiles / n,
                  more = tiles - small * n, i = s.tile0;
        s.tile0 = i * small + min(i, more);
        s.ntiles = small + (i < more ? 1 : 0);
      }
      s.whole = first >= span_lo && end <= span_hi;
      // two partials a span at most: one of a job that began before it, one
      // of a job that goes on behind it
      s.slot = 2 * (slot0 + span) + (first >= span_lo ? 1 : 0);
      if (first >= span_lo && (blockIdx.x & 1) == 0 && lane == 0) {
        a.ws_head[a.groups + 2 * j] = first;
        a.ws_head[a.groups + 2 * j + 1] = end;
      }
      return true;
    }
  }
};

// ------------------------------------------------- pair forms of the PTX
__device__ __forceinline__ void pair_alloc(uint32_t *dst) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)), "r"(512) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(512)
               : "memory");
}
// Cluster barrier without release: nothing that one CTA wrote is read by the
// other's threads, and the barriers' initialisation has a fence of its own.
// (With release the last one waits for the results' stores to arrive.)
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// One lane of a converged warp, chosen the same way every time.  The MMA
// warp runs its loops as a whole with this lane's instructions predicated on:
// addresses and descriptors then stay in uniform registers, and the 18 MMAs
// of a tile's Q K^T issue in 574 cycles (32 each, their full rate), against
// 1070 when one lane runs a branch of its own.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(e));
  return e;
}
template <bool FP8>
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t acc, uint32_t me) {
  if constexpr (FP8)
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(me) : "memory");
  else
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(me) : "memory");
}
// Arrives once on the barrier at this offset in both CTAs when every MMA so
// far of this thread has completed.
__device__ __forceinline__ void pair_commit(uint64_t *bar, uint32_t me) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
               "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
               ".multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
               "h"(static_cast<uint16_t>(3)), "r"(me) : "memory");
}
// A load into this CTA whose bytes count on a barrier of either CTA.
// (Maps: columns of a 128-byte box row, rows, box columns of the cache row; a
// slot of several boxes is one load.)
__device__ __forceinline__ void pair_load(void *dst, const CUtensorMap *map, uint32_t bar_cluster,
                                          int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
               ".cta_group::2 [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void load_3d_hint(void *dst, const CUtensorMap *map, uint64_t *bar, int x,
                                             int y, int z, uint64_t policy) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
               ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z),
               "l"(policy) : "memory");
}
// Bounded wait that first tests the phase: most waits here find it complete,
// and a test costs about 70 cycles where try_wait costs about 190.  What the
// barriers order across the pair is read by the tensor cores and the TMA
// only, so no wait needs cluster-scope acquire (one took about 200 cycles
// more, and a cluster-scope release of the probabilities 1600 a tile): either
// SM's tensor core reads its rows of P in its own CTA's shared memory, where the
// CTA-scope release in front of the remote arrival has put them.  That this is
// enough for a CTA of the pair to say so to the other is how the hardware
// behaves; the PTX memory model does not promise it without cluster scope.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  return mbar_test(bar, parity) || mbar_wait(bar, parity, abort_flag);
}

// Shared-memory descriptors as a constant high word and an address word, to
// which a step adds its offset in 16-byte units.
template <uint32_t SBO, uint32_t SWIZZLE>
__device__ __forceinline__ uint64_t desc_at(uint32_t lo) {
  constexpr uint32_t hi = (SBO >> 4) | (1u << 14) | (SWIZZLE << 29);
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ uint32_t desc_lo(const void *p, uint32_t lbo) {
  return ((smem_u32(p) & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}

// Named barrier of `count` threads that tells each whether `v` held for all.
__device__ __forceinline__ bool named_and(uint32_t id, uint32_t count, bool v) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %3, 0;\n\t"
               "barrier.cta.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r) : "r"(id), "r"(count), "r"(static_cast<uint32_t>(v)) : "memory");
  return r != 0;
}

// Probabilities (a, b) as pairs of e4m3 codes, hi, and of e5m2 codes, lo.
__device__ __forceinline__ void split_fp8(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 p = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(p, __NV_SATFINITE, __NV_E4M3);
  const __half2_raw back = __nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3);
  // exact: both are multiples of p's last place (or of 2^-24)
  const __half2 rest = __hsub2(p, *reinterpret_cast<const __half2 *>(&back));
  hi = h;
  lo = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E5M2);
}

// sum 2^(s - n) over the seen keys of the blocks whose P' is 2^-95 of that or less
// (of the others none of 2^-31 of the sum vanishes), by a whole warp; apart, as the
// kernel is 2 % slower with it in its loop.
__device__ __noinline__ float far_sum(uint32_t scores, uint64_t seen, float4 c, float4 lg, float base, float n) {
  float sum = 0.f;
#pragma unroll 1
  for (int g = 0; g < 4; ++g, seen >>= 16) {
    const uint32_t take = base - lg.x - n > 95.f ? static_cast<uint32_t>(seen) : 0;
    float x[16];
    tmem_ld_x16(scores + 16 * g, reinterpret_cast<uint32_t *>(x));
#pragma unroll
    for (int k = 0; k < 16; ++k) sum += take & (1u << k) ? ex2(fmaf(x[k], c.x, -n)) : 0.f;
    c = make_float4(c.y, c.z, c.w, c.x);
    lg = make_float4(lg.y, lg.z, lg.w, lg.x);
  }
  return sum;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads, 1)
window_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_kr,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_q,
              const __grid_constant__ CUtensorMap tm_qr, const __grid_constant__ WindowArgs args) {
  using F = Fmt<FP8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw;   // (no static shared memory: starts on 1024 bytes)
  uint8_t *sm_q = smem + F::kOffQ, *sm_k = smem + F::kOffK, *sm_v = smem + F::kOffV;
  uint8_t *sm_p = smem + F::kOffP;
  float *xchg = reinterpret_cast<float *>(smem + F::kOffX);
  Seg *segq = reinterpret_cast<Seg *>(smem + F::kOffSeg);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + F::kOffBars);
  // leader: written by both CTAs' loads or warps; the others exist in both
  uint64_t *k_full = bars;                    // [kKSlots] leader
  uint64_t *k_empty = k_full + F::kKSlots;    // [kKSlots]
  uint64_t *v_full = k_empty + F::kKSlots;    // [kVSlots]
  uint64_t *v_empty = v_full + F::kVSlots;    // [kVSlots]
  uint64_t *s_full = v_empty + F::kVSlots;    // [kSBufs]
  uint64_t *p_full = s_full + kSBufs;         // [2] leader
  uint64_t *pv_done = p_full + 2;             // [2]
  uint64_t *q_full = pv_done + 2;             // leader
  uint64_t *q_empty = q_full + 1;
  uint64_t *seg_full = q_empty + 1;           // [kSegSlots]
  uint64_t *seg_empty = seg_full + kSegSlots; // [kSegSlots]
  uint64_t *ref_there = seg_empty + kSegSlots;   // [2 groups][2 row blocks]
  uint64_t *sum_there = ref_there + 4;        // [2 row blocks]
  uint64_t *l_read = sum_there + 2;           // [2 row blocks] bf16: the sums in x_max have been read
  uint64_t *o_free = l_read + 2;           // leader: the last segment's O has been read
  uint64_t *drain = o_free + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert((2 * (F::kKSlots + F::kVSlots) + kSBufs + 4 + 2 + 2 * kSegSlots + 10) * 8 + 8 <= F::kBarBytes,
                "barriers");
  static_assert(sizeof(Seg) <= 32, "segment slot");

  if (smem_u32(smem) & 1023u) {   // (never seen: the swizzled tiles need it)
    if (threadIdx.x == 0) raise_error(args.err, MLA_DEVERR_TIMEOUT);
    return;
  }
  // (a shuffle: the same for the warp, as far as the compiler can tell)
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(warp_id()), 0), lane = lane_id();
  const int rank = static_cast<int>(cluster_rank());
  if (threadIdx.x == 0) {
    for (int s = 0; s < F::kKSlots; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < F::kVSlots; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < kSBufs; ++s) mbar_init(&s_full[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&p_full[s], kSoftWarps);      // a softmax group of either CTA
      mbar_init(&pv_done[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < kSegSlots; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], kSoftWarps + (rank == 0 ? 2 : 1));   // V, softmax, the leader's MMAs
    }
    for (int s = 0; s < 4; ++s) mbar_init(&ref_there[s], 2);   // the two warps of a row block
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sum_there[s], 4);            // its four, of both groups
      mbar_init(&l_read[s], 1);
    }
    mbar_init(o_free, 2 * kSoftWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) pair_alloc(tmem_slot);
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    if (FP8) {
      prefetch_tmap(&tm_qr);
      prefetch_tmap(&tm_kr);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pair_sync();                                // both CTAs' barriers and memory are there
  grid_dep_wait();
  grid_dep_launch();

  // Every consuming warp takes the segments in order.
  auto take_seg = [&](int ns, Seg &s) -> bool {
    const int slot = ns % kSegSlots;
    if (!__all_sync(0xffffffffu, wait_for(&seg_full[slot], (ns / kSegSlots) & 1, abort_flag)))
      return false;
    s = segq[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_empty[slot]);
    return s.ntiles >= 0;
  };
  // Block ids of a segment's pages: lane k holds those of list entry
  // base + k, as loaded; entries behind the list and bad ids give -1.
  struct Pages {
    int base, blk;
  };
  auto fetch_blocks = [&](Pages &pg, const Job &job, int b, int entry) {
    pg.base = entry;
    const int e = entry + lane;
    pg.blk = e < job.pages
                 ? __ldg(args.block_table + static_cast<int64_t>(b) * args.max_blocks + job.page(e))
                 : -1;
  };
  auto block_at = [&](Pages &pg, const Job &job, int b, int entry) -> int {   // whole warp
    if (entry >= pg.base + 32) fetch_blocks(pg, job, b, entry);
    const int v = __shfl_sync(0xffffffffu, pg.blk, entry - pg.base);
    if (v >= 0 && v < args.num_blocks) return v;
    if (entry < job.pages && lane == 0) raise_error(args.err, MLA_DEVERR_BLOCK_ID);
    return -1;
  };
  // rows out of the cache: TMA fills in zeros
  const int no_row = args.num_blocks * kPage;

  if (warp == 0) {
    // ------------------------------------------------- plan, Q and K
    Walk<FP8> walk;
    if (args.solo) {
      walk.init_solo(args);
    } else {
      walk.init(args, lane);
    }
    Seg sg;
    int ns = 0, nq = 0, kc = 0;             // segments, queries, K slots so far
    bool ok = true;
    auto publish = [&](const Seg &s) -> bool {
      const int slot = ns % kSegSlots;
      if (ns >= kSegSlots && !wait_for(&seg_empty[slot], ((ns / kSegSlots) - 1) & 1, abort_flag))
        return false;
      if (lane == 0) {
        segq[slot] = s;
        mbar_arrive(&seg_full[slot]);
      }
      __syncwarp();
      return true;
    };
    const uint32_t q_bar = peer_smem(q_full, 0);
    while (ok && (args.solo ? walk.next_solo(args, sg) : walk.next(args, sg, lane))) {
      const Job job = job_of(sg.rg, sg.len, args);
      Pages pg;
      fetch_blocks(pg, job, sg.b, F::kPages * sg.tile0);
      if (!(ok = publish(sg))) break;
      ++ns;
      if (sg.ntiles == 0) continue;
      // Q, once the last segment's last Q K^T has read it
      if (nq > 0 && !(ok = wait_for(q_empty, (nq - 1) & 1, abort_flag))) break;
      ++nq;
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * F::kQBytes);
        const int row = sg.b * args.q_len * args.H + sg.rg * 128 + 64 * rank;
        pair_load(sm_q, &tm_q, q_bar, 0, row, 0);
        if (FP8) pair_load(sm_q + 4 * 8192, &tm_qr, q_bar, kLatent, row, 0);
      }
      for (int t = 0; ok && t < sg.ntiles; ++t) {
        // this CTA's key rows: a page of the two, or half of the one
        const int blk = block_at(pg, job, sg.b, F::kPages * (sg.tile0 + t) + (F::kPages - 1) * rank);
        const int row = blk < 0 ? no_row : blk * kPage + (2 - F::kPages) * F::kKRows * rank;
        const int s = kc % F::kKSlots;
        if (kc >= F::kKSlots &&
            !(ok = wait_for(&k_empty[s], ((kc / F::kKSlots) - 1) & 1, abort_flag)))
          break;
        ++kc;
        if (lane == 0) {
          if (rank == 0) mbar_arrive_expect_tx(&k_full[s], 2 * F::kKSlotBytes);
          const uint32_t bar = peer_smem(&k_full[s], 0);
          pair_load(sm_k + s * F::kKSlotBytes, &tm_k, bar, 0, row, 0);
          if (FP8) pair_load(sm_k + s * F::kKSlotBytes + 4 * F::kKBox, &tm_kr, bar, kLatent, row, 0);
        }
      }
    }
    if (ok) {
      sg.ntiles = -1;
      publish(sg);
    }
    // neither CTA leaves before the last signals to it have arrived
    if (ok) {
      for (int u = max(0, kc - F::kKSlots); ok && u < kc; ++u)
        ok = wait_for(&k_empty[u % F::kKSlots], (u / F::kKSlots) & 1, abort_flag);
      if (ok && nq > 0) wait_for(q_empty, (nq - 1) & 1, abort_flag);
    }
    if (*abort_flag && rank == 0 && lane == 0) {   // what is on its way lands first
      volatile int no_abort = 0;
      for (int u = max(0, kc - F::kKSlots); u < kc; ++u)
        wait_for(&k_full[u % F::kKSlots], (u / F::kKSlots) & 1, &no_abort);
      if (nq > 0) wait_for(q_full, (nq - 1) & 1, &no_abort);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------- V
    const uint64_t policy = l2_evict_first_policy();   // the rows' second and last read
    Seg sg;
    int vc = 0;
    bool ok = true;
    for (int ns = 0; ok && take_seg(ns, sg); ++ns) {
      const Job job = job_of(sg.rg, sg.len, args);
      Pages pg;
      fetch_blocks(pg, job, sg.b, F::kPages * sg.tile0);
      for (int t = 0; ok && t < sg.ntiles; ++t) {
        for (int v = 0; v < F::kVPer; ++v, ++vc) {
          const int blk = block_at(pg, job, sg.b, F::kPages * (sg.tile0 + t) + v);
          const int s = vc % F::kVSlots;
          if (vc >= F::kVSlots &&
              !(ok = wait_for(&v_empty[s], ((vc / F::kVSlots) - 1) & 1, abort_flag)))
            break;
          const int row = blk < 0 ? no_row : blk * kPage;
          if (lane == 0) {
            mbar_arrive_expect_tx(&v_full[s], F::kVSlotBytes);
            load_3d_hint(sm_v + s * F::kVSlotBytes, &tm_v, &v_full[s], 0, row, F::kVBoxes * rank, policy);
          }
        }
      }
    }
    for (int u = max(0, vc - F::kVSlots); ok && u < vc; ++u)
      ok = wait_for(&v_empty[u % F::kVSlots], (u / F::kVSlots) & 1, abort_flag);
    if (*abort_flag && lane == 0) {
      volatile int no_abort = 0;
      for (int u = max(0, vc - F::kVSlots); u < vc; ++u)
        wait_for(&v_full[u % F::kVSlots], (u / F::kVSlots) & 1, &no_abort);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------------------------------------------------- MMAs
      const uint32_t idesc_qk = FP8 ? idesc_e4m3(128, F::kTile, false, false)
                                    : idesc_bf16(128, F::kTile, false, false);
      const uint32_t idesc_pv = FP8 ? idesc_e4m3(128, 256, false, true)
                                    : idesc_bf16(128, 256, false, true);
      const uint32_t idesc_lo = idesc_pv | kIdescA_e5m2;
      const uint32_t me = elect_one();
      const uint32_t qd = desc_lo(sm_q, 16);
      auto wait = [&](uint64_t *bar, int phase) -> bool {
        return __all_sync(0xffffffffu, wait_for(bar, phase & 1, abort_flag));
      };
      int kc = 0, vc = 0, uc = 0;             // K slots, V slots, tiles so far
      bool ok = true;
      auto issue_qk = [&](int u) -> bool {
        const uint32_t d = tmem + kColS + F::kTile / 2 * (u % kSBufs);
        const int s = kc % F::kKSlots;
        if (!wait(&k_full[s], kc / F::kKSlots)) return false;
        ++kc;
        tc_fence_after();
        // one descriptor a slot; steps add to its address field (16-byte units)
        const uint32_t kd = desc_lo(sm_k + s * F::kKSlotBytes, 16);
#pragma unroll
        for (int k = 0; k < 4 * F::kBoxes; ++k)
          pair_mma<FP8>(d, desc_at<1024, kSwizzle128B>(qd + (k >> 2) * 512 + (k & 3) * 2),
                        desc_at<1024, kSwizzle128B>(kd + (k >> 2) * (F::kKBox / 16) + (k & 3) * 2),
                        idesc_qk, k > 0, me);
        if constexpr (FP8) {
#pragma unroll
          for (int k = 0; k < 2; ++k)         // the rope columns: rows of 64 bytes
            pair_mma<FP8>(d, desc_at<512, kSwizzle64B>(qd + 4 * 512 + 2 * k),
                          desc_at<512, kSwizzle64B>(kd + 4 * (F::kKBox / 16) + 2 * k), idesc_qk, 1, me);
        }
        pair_commit(&k_empty[s], me);
        pair_commit(&s_full[u % kSBufs], me);
        return true;
      };
      // All steps of one accumulator, then of the other: an MMA that adds to
      // what the last but one wrote waits for it (232 cycles a change).
      auto issue_pv = [&](int u, bool first) {
        const uint32_t pd = desc_lo(sm_p + (u % F::kPBufs) * F::kPBytes, 16);
#pragma unroll
        for (int j = 0; j < 2; ++j) {         // value columns 128j .. 128j + 127 of either CTA
#pragma unroll
          for (int v = 0; v < F::kVPer; ++v) {
            const int s = (vc + v) % F::kVSlots;
            const uint32_t vd = desc_lo(sm_v + s * F::kVSlotBytes, F::kVBox);
#pragma unroll
            for (int kk = 0; kk < F::kVSteps; ++kk) {   // 32 bytes of P: 32 e4m3 or 16 bf16 keys
              const int step = F::kVSteps * v + kk;
              const uint32_t pa = pd + step * 2;
              const uint64_t bd = desc_at<1024, kSwizzle128B>(
                  vd + (FP8 ? j * F::kVBox + kk * 4096 : 2 * j * F::kVBox + kk * 2048) / 16);
              pair_mma<FP8>(tmem + kColO + 128 * j, desc_at<1024, kSwizzle128B>(pa), bd, idesc_pv,
                            first && step == 0 ? 0u : 1u, me);
              if constexpr (FP8)
                pair_mma<FP8>(tmem + kColO + 128 * j, desc_at<1024, kSwizzle128B>(pa + 512), bd,
                              idesc_lo, 1, me);
            }
            if (j == 1) pair_commit(&v_empty[s], me);
          }
        }
        vc += F::kVPer;
        pair_commit(&pv_done[u & 1], me);
      };
      Seg sg;
      int nq = 0;
      for (int ns = 0; ok && take_seg(ns, sg); ++ns) {
        const int n = __shfl_sync(0xffffffffu, sg.ntiles, 0);
        if (n == 0) continue;
        if (!(ok = wait(q_full, nq++))) break;
        if (!(ok = issue_qk(uc))) break;
        if (n > 1 && !(ok = issue_qk(uc + 1))) break;
        if (n <= 2) pair_commit(q_empty, me);
        for (int t = 0; t < n; ++t, ++uc) {
          // the scores of tile t + 2 go where tile t - 2's were: read before
          // its probabilities were handed over
          if (t + 2 < n) {
            if (!(ok = issue_qk(uc + 2))) break;
            if (t + 3 == n) pair_commit(q_empty, me);
          }
          if (t == 0 && nq > 1 && !(ok = wait(o_free, nq - 2))) break;
          if (!(ok = wait(&p_full[uc & 1], uc >> 1))) break;
          tc_fence_after();
          issue_pv(uc, t == 0);
        }
      }
      if (ok && nq > 0) wait(o_free, nq - 1);   // (the other CTA's last signals are in)
      if (*abort_flag) {
        pair_commit(drain, me);
        volatile int no_abort = 0;
        wait_for(drain, 0, &no_abort);
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------ softmax and results
    // Two groups of four warps take the tiles in turn (group 0 the even ones,
    // over all segments), so that one tile's exponentials overlap the next
    // one's scores.  In a group two threads share a row, each with kMine of
    // the tile's keys (`half`: the TMEM lanes, which CTA's key rows).  What
    // tile t + 1 needs of tile t is the row's reference; it is handed on
    // through shared memory as soon as the row's maximum is known.
    const int quarter = warp & 3, half = quarter >> 1, group = (warp - 4) >> 2;
    const int block = quarter & 1;                      // row block: rows 32 block ..
    const int r = block * 32 + lane;                    // row of this CTA
    const uint32_t lane_base = tmem + ((quarter * 32u) << 16);
    const uint32_t p_bar[2] = {peer_smem(&p_full[0], 0), peer_smem(&p_full[1], 0)};
    const uint32_t o_bar = peer_smem(o_free, 0);
    float *x_max = xchg + 128 * group, *x_ref = xchg + 256, *x_sum = xchg + 384, *x_unit = xchg + 640;
    // The hardware barrier of the two warps has no limit, so neither may leave
    // the other in it: it takes along whether all is well, a warp whose wait
    // ran out goes through it once more before it leaves, and the other leaves
    // behind it.
    bool told = false;
    auto pair_max = [&](float &v) -> bool {             // over the row's two threads
      x_max[64 * half + r] = v;
      told = !named_and(1 + 2 * group + block, 64, true);
      v = fmaxf(v, x_max[64 * (half ^ 1) + r]);
      return !told;
    };
    auto all_ok = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    Seg sg;
    int uc = 0, segs = 0;                               // tiles and segments (with tiles) so far
    bool ok = true;
    for (int ns = 0; ok && take_seg(ns, sg); ++ns) {
      const int R = args.q_len * args.H;
      if (sg.ntiles == 0) {
        const int row0 = sg.rg * 128 + 64 * rank, n = min(64, R - row0);
        const int64_t at = static_cast<int64_t>(sg.b) * R + row0;
        const int chunks = kLatent * (args.out_f32 ? 4 : 2) / 16;
        uint4 *o = static_cast<uint4 *>(args.out) + at * chunks;
        const int tid = threadIdx.x - 128;
        for (int k = tid; k < n * chunks; k += 32 * kSoftWarps) o[k] = make_uint4(0, 0, 0, 0);
        if (tid < n) args.lse[at + tid] = -INFINITY;
        continue;
      }
      const Job job = job_of(sg.rg, sg.len, args);
      const int grow = sg.rg * 128 + 64 * rank + r;     // row of the request
      // (rows behind the request's last are computed and dropped)
      const int p = grow < R ? sg.len - args.q_len + grow / args.H : job.p1;
      const int wlo = args.window ? p - args.window + 1 : 0;
      // every query row of the job sees keys [clean_lo, job.p0] and the sinks
      const int clean_lo = args.window ? job.p1 - args.window + 1 : 0;
      // scales of this thread's keys, a tile of its group ahead
      const int32_t *bt = args.block_table + static_cast<int64_t>(sg.b) * args.max_blocks;
      auto load_blk = [&](int t) -> int {
        const int e = F::kPages * (sg.tile0 + t) + half;
        if (!FP8 || !args.scales || t >= sg.ntiles || e >= job.pages) return -1;
        return __ldg(bt + job.page(e));   // (looked at a tile later: nothing waits for it here)
      };
      constexpr int kBlocks = FP8 ? 4 : 1;   // scales of 64 keys
      auto load_scales = [&](int blk, float *sc) {
#pragma unroll
        for (int g = 0; g < kBlocks; ++g)
          sc[g] = blk < 0 || blk >= args.num_blocks
                      ? args.k_scale
                      : __ldg(args.scales + ((static_cast<int64_t>(blk) * kPage + 16 * g) >> args.sb_shift));
      };
      const int t_first = (uc ^ group) & 1;             // this group's first tile
      float sc[kBlocks], sc_next[kBlocks];
      int blk_next = load_blk(t_first + 2);
      load_scales(load_blk(t_first), sc);
      const int uc0 = uc;
      uc += sg.ntiles;
      // e4m3: the sum in units of 2^ln.  bf16: sums in units of 2^ref, of the
      // probabilities for the logarithm and of their rounded values for the
      // results, where a large one's rounding then is in the numerator and the
      // denominator (16 rows of 132 keys: 2.1e-3 of the output's rms against 64
      // bits, 1.7e-3 of it the output's own rounding; divided by the unrounded sum
      // 2.3e-3, of one set in seven more than 2.5e-3)
      float ref = -INFINITY, l = 0.f, lr = 0.f, ln = -INFINITY;
      float highest = -INFINITY;                        // reference so far
      for (int t = t_first; t < sg.ntiles; t += 2) {
        const int u = uc0 + t, half_u = u >> 1;         // (group u & 1)
        load_scales(blk_next, sc_next);
        blk_next = load_blk(t + 4);
        const int e0 = F::kPages * (sg.tile0 + t);
        const int page0 = job.page(e0) * kPage;
        const int page1 = F::kPages == 2 && e0 + 1 < job.pages ? job.page(e0 + 1) * kPage : 1 << 30;
        const int key0 = (F::kPages == 2 ? (half ? page1 : page0) : page0 + F::kKRows * half);
        const bool masked = key0 + F::kMine - 1 > p || (key0 < wlo && key0 + F::kMine > args.sinks);
        auto clean = [&](int k0) {
          return k0 == 1 << 30 ||
                 (k0 + kPage - 1 <= job.p0 && (k0 >= clean_lo || k0 + kPage <= args.sinks));
        };
        const bool all_clean = clean(page0) && clean(page1);
        auto seen_keys = [&] {
          return low_bits(p - key0 + 1) & (~low_bits(wlo - key0) | low_bits(args.sinks - key0));
        };
        constexpr int kRun = F::kMine / kBlocks;        // keys of one scale: 16 / 32
        float c[kBlocks], lg[kBlocks];
#pragma unroll
        for (int g = 0; g < kBlocks; ++g) {
          // (a scale of 0 stands for zeros: so does the smallest one; what is no scale is NaN)
          const bool is_scale = !FP8 || (sc[g] >= 0.f && sc[g] <= 0x1p120f);
          const float sigma = is_scale ? fmaxf(sc[g], 0x1p-100f) : __uint_as_float(0x7FC00000u);
          // (at least 2^-126, which makes any score 0 as well as less does: masked
          // scores of -inf times 0 would be NaN)
          c[g] = fminf(fmaxf(sigma * args.scale_pre * args.scale_log2, 0x1p-126f), 0x1.fffffep127f);
          lg[g] = FP8 ? log2f(sigma) : 0.f;
        }
        float lg_min = lg[0], lg_max = lg[0];
#pragma unroll
        for (int g = 1; g < kBlocks; ++g) {
          lg_min = fminf(lg_min, lg[g]);
          lg_max = fmaxf(lg_max, lg[g]);
        }
        if (!(ok = all_ok(wait_for(&s_full[u % kSBufs], (u / kSBufs) & 1, abort_flag)))) break;
        tc_fence_after();
        float x[F::kMine];
        const uint32_t s_at = lane_base + kColS + F::kTile / 2 * (u % kSBufs);
        if constexpr (FP8) tmem_ld_x64(s_at, reinterpret_cast<uint32_t *>(x));
        else tmem_ld_x32(s_at, reinterpret_cast<uint32_t *>(x));
        if (masked) {
          const uint64_t seen = seen_keys();
#pragma unroll
          for (int k = 0; k < F::kMine; ++k) x[k] = seen & (uint64_t(1) << k) ? x[k] : -INFINITY;
          if constexpr (FP8) {                          // (NaN is for rows that see a key of the block)
#pragma unroll
            for (int g = 0; g < kBlocks; ++g)
              if (!(seen >> (kRun * g) & 0xFFFFu)) lg[g] = 0.f;
          }
        }
        float top = -INFINITY, raw[kBlocks];            // largest s + log2 sigma; of a block's scores
#pragma unroll
        for (int g = 0; g < kBlocks; ++g) {
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < kRun; k += 4) {
            m0 = fmax3(m0, x[kRun * g + k], x[kRun * g + k + 1]);
            m1 = fmax3(m1, x[kRun * g + k + 2], x[kRun * g + k + 3]);
          }
          raw[g] = fmaxf(m0, m1);
          top = fmaxf(top, fmaf(raw[g], c[g], lg[g]));
        }
        const float high_low = fmaxf(ln, top - lg_max);   // the largest s is no less
        if (!FP8 && t <= 1 && segs > 0 &&
            !(ok = all_ok(wait_for(&l_read[block], (segs - 1) & 1, abort_flag))))
          break;
        if (!(ok = pair_max(top))) break;
        // a reference above this goes down (none, where the row sees no key of the tile)
        const float above = top > -INFINITY ? fmaxf(top - F::kLow, highest - F::kDepth) : INFINITY;
        // the reference that the tile before left, and what this one makes of it
        float old = -INFINITY;
        if (t > 0) {
          if (!(ok = all_ok(wait_for(&ref_there[2 * (group ^ 1) + block], ((u - 1) >> 1) & 1, abort_flag))))
            break;
          old = x_ref[64 * (group ^ 1) + r];
        }
        // Where one of the warp's rows has to move, all that can go up do so: the
        // pass over O is paid for, and the next one is further off.  (The row's
        // other thread, in a warp of the same rows, decides alike.)
        const bool down = FP8 && old > above;
        const bool moves = __any_sync(0xffffffffu, top - F::kLazy > old || down);
        const bool up = moves && top - F::kTop > old, move = up || down;
        float now = up ? top - F::kTop : old;
        if (down) now = fmaxf(top, fmaxf(highest, old) - F::kDepth);
        if (half == 0) x_ref[64 * group + r] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ref_there[2 * group + block]);
        const bool rescale = t > 0 && moves;
        const float f = move ? (old == -INFINITY ? 0.f : ex2(old - now)) : 1.f;
        if (!FP8 && ref != now && l != 0.f) {
          const float by = ex2(ref - now);
          l *= by;
          lr *= by;
        }
        ref = now;
        if constexpr (FP8) highest = fmaxf(highest, fmaxf(old, now));
        float part[kBlocks], rest = 0.f;                // (the sum waits until the probabilities are handed over)
        const float base = ref == -INFINITY ? 0.f : ref;
        // a P' that is 2^-95 of its 2^(s - n) or less, below
        const bool again = FP8 && __any_sync(0xffffffffu, high_low > -INFINITY && base - lg_min - high_low > 95.f);
#pragma unroll
        for (int g = 0; g < kBlocks; ++g) {
          const float d = lg[g] - base;
          float s0 = 0.f, s1 = 0.f, r0 = 0.f, r1 = 0.f;
#pragma unroll
          for (int k = kRun * g; k < kRun * g + kRun; k += 2) {
            fma_f32x2(x[k], x[k + 1], x[k], x[k + 1], c[g], c[g], d, d);
            x[k] = ex2(x[k]);
            x[k + 1] = ex2(x[k + 1]);
            add_f32x2(s0, s1, s0, s1, x[k], x[k + 1]);
            if constexpr (!FP8) {
              const uint32_t pk = bf16x2_rn(x[k], x[k + 1]);
              x[k] = __uint_as_float(pk);               // (both: stored as they are)
              add_f32x2(r0, r1, r0, r1, __uint_as_float(pk << 16), __uint_as_float(pk & 0xFFFF0000u));
            }
          }
          if constexpr (FP8) {
            part[g] = s0 + s1;
          } else {
            l += s0 + s1;
            lr += r0 + r1;
          }
        }
        // P goes where the P V of this group's last tile read
        if (u >= 2 && !(ok = all_ok(wait_for(&pv_done[group], (half_u - 1) & 1, abort_flag)))) break;
        uint8_t *pbuf = sm_p + group * F::kPBytes;
        if constexpr (FP8) {
          uint4 *hi = reinterpret_cast<uint4 *>(pbuf + r * 128);
          uint4 *lo = reinterpret_cast<uint4 *>(pbuf + 8192 + r * 128);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t h[4], w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h0, h1, l0, l1;
              split_fp8(x[16 * q + 4 * k], x[16 * q + 4 * k + 1], h0, l0);
              split_fp8(x[16 * q + 4 * k + 2], x[16 * q + 4 * k + 3], h1, l1);
              h[k] = h0 | (h1 << 16);
              w[k] = l0 | (l1 << 16);
            }
            const int ch = (4 * half + q) ^ (r & 7);
            hi[ch] = make_uint4(h[0], h[1], h[2], h[3]);
            lo[ch] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          uint4 *row = reinterpret_cast<uint4 *>(pbuf + r * 128);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            row[(4 * half + q) ^ (r & 7)] =
                make_uint4(__float_as_uint(x[8 * q]), __float_as_uint(x[8 * q + 2]),
                           __float_as_uint(x[8 * q + 4]), __float_as_uint(x[8 * q + 6]));
        }
        auto next_unit = [&] {
          float n = ln;
#pragma unroll
          for (int g = 0; g < kBlocks; ++g) n = fmaxf(n, raw[g] * c[g]);
          return n;
        };
        if constexpr (FP8) {
          if (again)
            rest = far_sum(s_at, masked ? seen_keys() : ~uint64_t(0), make_float4(c[0], c[1], c[2], c[3]),
                           make_float4(lg[0], lg[1], lg[2], lg[3]), base, next_unit());
        }
        if (rescale) {
          // O follows the reference, now that the last P V is done
          if (!(ok = all_ok(wait_for(&pv_done[group ^ 1], ((u - 1) >> 1) & 1, abort_flag)))) break;
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < 256; q += 64) {
            uint32_t o[64];
            tmem_ld_x64(lane_base + kColO + q, o);
#pragma unroll
            for (int k = 0; k < 64; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st_x32(lane_base + kColO + q, o);
            tmem_st_x32(lane_base + kColO + q + 32, o + 32);
          }
        }
        // the values are here (the MMA thread goes by this CTA's word)
#pragma unroll
        for (int v = 0; v < F::kVPer; ++v) {
          const int w = F::kVPer * u + v;
          ok = ok && wait_for(&v_full[w % F::kVSlots], (w / F::kVSlots) & 1, abort_flag);
        }
        if (ok && !all_clean) {
          // rows that not every query row sees: 0 where none does, and where
          // some do, 0 in place of what is not finite (0 times it in the
          // others).  A row of this CTA's columns is one (bf16) or half a
          // (e4m3) warp's 16-byte chunks.
          constexpr int kChunks = F::kVBoxes * 8, kRowsAtOnce = 32 / kChunks;
          const int lr = lane / kChunks, at = ((lane % kChunks) >> 3) * F::kVBox + (lane & 7) * 16;
#pragma unroll 1
          for (int h = 0; h < F::kPages; ++h) {
            const int page = h ? page1 : page0;
            if (clean(page)) continue;
            // all rows see [0, a) (sinks) and [b, c) of the page's 64
            const int c = min(max(job.p0 + 1 - page, 0), kPage);
            const int b = min(max(clean_lo - page, 0), c), a = min(max(args.sinks - page, 0), b);
            const int n = b - a + kPage - c;
#pragma unroll 1
            for (int i = quarter * kRowsAtOnce + lr; i < n; i += 4 * kRowsAtOnce) {
              const int tok = i < b - a ? a + i : c + i - (b - a);
              const int slot = (F::kVPer * u + (h * kPage + tok) / F::kVTok) % F::kVSlots;
              uint4 *w = reinterpret_cast<uint4 *>(sm_v + slot * F::kVSlotBytes + at +
                                                   (tok % F::kVTok) * 128);
              uint4 val = make_uint4(0, 0, 0, 0);
              const int key = page + tok;
              if (job.p0 != job.p1 && key <= job.p1 &&
                  (!args.window || key < args.sinks || key > job.p0 - args.window)) {
                val = *w;
                uint32_t *e4 = reinterpret_cast<uint32_t *>(&val);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if constexpr (FP8) {
                    const uint32_t nan = (((e4[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
                    e4[k] &= ~(nan * 0xFFu);
                  } else {
                    if ((e4[k] & 0x7F80u) == 0x7F80u) e4[k] &= 0xFFFF0000u;
                    if ((e4[k] & 0x7F800000u) == 0x7F800000u) e4[k] &= 0xFFFFu;
                  }
                }
              }
              *w = val;
            }
          }
        }
        if (!(ok = all_ok(ok))) break;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(p_bar[group]);
        if constexpr (FP8) {
          const float n = next_unit();
          l = fmaf(l, ln == n ? 1.f : ex2(ln - n), rest);
          ln = n;
#pragma unroll
          for (int g = 0; g < kBlocks; ++g) {
            const float e = base - lg[g] - (n == -INFINITY ? 0.f : n);
            l = fmaf(part[g], e > 95.f ? 0.f : ex2(e), l);
          }
        }
#pragma unroll
        for (int g = 0; g < kBlocks; ++g) sc[g] = sc_next[g];
      }
      if (!ok) break;
      // ---- results: O / l of this row, value columns [256 half + 128 group, +128)
      const int last = uc - 1, lg_last = last & 1;
      if (!(ok = all_ok(wait_for(&ref_there[2 * lg_last + block], (last >> 1) & 1, abort_flag) &&
                        wait_for(&pv_done[lg_last], (last >> 1) & 1, abort_flag))))
        break;
      tc_fence_after();
      const float end_ref = x_ref[64 * lg_last + r];
      if (!FP8 && l != 0.f) {
        const float by = ex2(ref - end_ref);
        l *= by;
        lr *= by;
      }
      ref = end_ref;
      if constexpr (FP8) x_unit[128 * group + 64 * half + r] = ln;
      // (of x_max the row's four have taken the last maximum)
      x_sum[128 * group + 64 * half + r] = FP8 ? l : lr;
      if (!FP8) x_max[64 * half + r] = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sum_there[block]);
      if (!(ok = all_ok(wait_for(&sum_there[block], segs & 1, abort_flag)))) break;
      ++segs;
      auto total = [&](const float *x) { return (x[r] + x[64 + r]) + (x[128 + r] + x[192 + r]); };
      float sum, unit = ref;                            // (the logarithm's, too)
      if constexpr (FP8) {
        unit = fmaxf(fmaxf(x_unit[r], x_unit[64 + r]), fmaxf(x_unit[128 + r], x_unit[192 + r]));
        if (unit == -INFINITY) unit = 0.f;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < 256; k += 64) sum = fmaf(x_sum[k + r], ex2(x_unit[k + r] - unit), sum);
      } else {
        sum = total(x_sum);
      }
      const bool empty = sum == 0.f;
      const float inv = empty ? 0.f : FP8 ? ex2(ref - unit) / sum : 1.f / sum;
      if (half + group == 0) {
        l = FP8 ? sum : total(xchg);
        __syncwarp();
        if (!FP8 && lane == 0) mbar_arrive(&l_read[block]);
      }
      const int64_t row0 = static_cast<int64_t>(sg.b) * R + sg.rg * 128 + 64 * rank;
      const int64_t at = sg.whole ? row0 : static_cast<int64_t>(sg.slot) * 128 + 64 * rank;
      const int nrows = min(64, R - sg.rg * 128 - 64 * rank);
      const int esz = args.out_f32 ? 4 : 2;
      uint8_t *dst0 = static_cast<uint8_t *>(sg.whole ? args.out : args.ws_o) +
                      (at * kLatent + 256 * half + 128 * group) * esz;
      const int64_t rstride = static_cast<int64_t>(kLatent) * esz;
      if (half + group == 0 && r < nrows) {
        const float v = empty ? -INFINITY : (unit + log2f(l)) * 0.69314718055994531f;
        (sg.whole ? args.lse : args.ws_lse)[at + r] = v;
      }
      uint32_t all[128];
      tmem_ld_x64(lane_base + kColO + 128 * group, all);
      tmem_ld_x64(lane_base + kColO + 128 * group + 64, all + 64);
      tc_fence_before();   // (O has been read: the next segment's P V may begin)
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(o_bar);
      const bool fp16 = !sg.whole && !args.out_f32;
      float factor = inv;
      if (fp16) {
        // the largest finite |O| to [2^14, 2^15)
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 128; k += 2)
          top = fmax3(top, fabsf(__uint_as_float(all[k])), fabsf(__uint_as_float(all[k + 1])));
        if (top == INFINITY) {
          top = 0.f;
#pragma unroll
          for (int k = 0; k < 128; ++k) {
            const float a = fabsf(__uint_as_float(all[k]));
            if (a < INFINITY) top = fmaxf(top, a);
          }
        }
        const uint32_t exp = max(__float_as_uint(top) >> 23, 15u);
        factor = __uint_as_float((268u - exp) << 23);
        if (r < nrows)
          args.ws_unit[4 * (at + r) + 2 * group + half] = __uint_as_float((exp - 14u) << 23) * inv;
      }
      // pieces of 64 bytes a row, staged through 2 KB of this warp's own in its
      // group's P tile (in its row block, which the pair writes again behind
      // its next barrier), so that stores cover whole sectors
      uint4 *buf = reinterpret_cast<uint4 *>(sm_p + group * F::kPBytes + block * 4096 + half * 2048);
      static_assert(F::kPBytes >= 4 * 2048, "staging");
      // (a body for each type of element: 0 bf16, 1 fp16, 2 fp32)
      auto write = [&](auto type) {
        constexpr int kType = decltype(type)::value, kPer = kType == 2 ? 16 : 32;   // values of a piece
        auto pack = [&](int k) -> uint32_t {
          const float x = __uint_as_float(all[k]) * factor;
          if constexpr (kType == 2) return __float_as_uint(x);
          const float y = __uint_as_float(all[k + 1]) * factor;
          if constexpr (kType == 0) return bf16x2_rn(x, y);
          const __half2 h = __floats2half2_rn(x, y);
          return *reinterpret_cast<const uint32_t *>(&h);
        };
#pragma unroll
        for (int q = 0; q < 128; q += kPer) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            constexpr int kStep = kPer / 16;
            const int e = q + 4 * kStep * k;
            buf[lane * 4 + (k ^ ((lane >> 1) & 3))] =
                make_uint4(pack(e), pack(e + kStep), pack(e + 2 * kStep), pack(e + 3 * kStep));
          }
          __syncwarp();
          uint8_t *dst = dst0 + static_cast<int64_t>(q) * (64 / kPer);
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int row = it * 8 + (lane >> 2), ch = lane & 3;
            const int rr = block * 32 + row;
            if (rr < nrows)
              reinterpret_cast<uint4 *>(dst + rr * rstride)[ch] = buf[row * 4 + (ch ^ ((row >> 1) & 3))];
          }
        }
      };
      if (args.out_f32) write(std::integral_constant<int, 2>{});
      else if (fp16) write(std::integral_constant<int, 1>{});
      else write(std::integral_constant<int, 0>{});
    }
    if (!told) named_and(1 + 2 * group + block, 64, ok && !*abort_flag);
  }
  __syncthreads();
  pair_sync();                                // neither CTA's MMAs or signals need the other any more
  if (threadIdx.x == 0 && *abort_flag) raise_error(args.err, MLA_DEVERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    pair_dealloc(tmem);
  }
}

// Combines the partials of the jobs that were cut, and writes the rows of
// jobs without a key.  Part k of a job whose first span is s0 lies in slot
// 2 s0 + 1 (k = 0) or 2 (s0 + k).  What it costs is latency, so a round's logs
// and rows are asked for together, the maximum runs along, and the CTAs are all
// resident at once (64 registers where there are most of them).  SPLIT warps
// share a row and take every SPLIT-th part, joined through shared memory.
// Decode and merge over 65536 tokens (e4m3, 128 heads), 1 / 4 / 8 warps a row:
// 1 request (76 parts a row) 49.4 / 23.5 / 20.2 us, 4 requests (19 parts)
// 26.6 / 19.8 / 26.5, 8 requests (9) 22.5 / 22.8 / 34.1.
constexpr int kMergeWarps = 8;

template <typename T, int SPLIT>
__global__ void __launch_bounds__(kMergeWarps * 32, SPLIT == 8 ? 1 : SPLIT == 4 ? 2 : 4)
window_merge_kernel(const __grid_constant__ WindowArgs a) {
  constexpr int kRows = kMergeWarps / SPLIT;    // rows of this CTA
  constexpr int kQuads = sizeof(T);             // 16-byte words of a lane's 16 values
  // parts on their way: of fp16 10 / 6 / 2 (one warp a row: 4 of them, in spilled
  // registers, took 1 us more)
  constexpr int kRound = (SPLIT == 8 ? 20 : SPLIT == 4 ? 12 : 4) / kQuads;
  __shared__ float part_o[SPLIT > 1 ? kMergeWarps : 1][kLatent];
  __shared__ float part_z[kMergeWarps], part_m[kMergeWarps];
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % SPLIT;
  const int j = blockIdx.x, rg = a.RG > 1 ? j / a.B : 0, b = j - rg * a.B;
  const int rr = blockIdx.y * kRows + warp / SPLIT;
  const int R = a.q_len * a.H;
  const bool row_ok = rg * 128 + rr < R;
  if (SPLIT == 1 && !row_ok) return;
  const int64_t row = static_cast<int64_t>(b) * R + rg * 128 + rr;
  T *out = static_cast<T *>(a.out) + row * kLatent;
  const int group = j / a.group_jobs;
  const int C = a.ws_head[group], first = a.ws_head[a.groups + 2 * j], end = a.ws_head[a.groups + 2 * j + 1];
  if (job_of(rg, length_of(b, a, false), a).pages == 0) {   // (the words above hold nothing)
    if (mine == 0 && row_ok) {
      const float zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (int k = 0; k < 2; ++k) store8(out + 8 * (lane + 32 * k), zero);
      if (lane == 0) a.lse[row] = -INFINITY;
    }
    return;
  }
  const int s0 = first / C + group * a.group_spans, n = (end - 1) / C - first / C + 1;
  if (n == 1) return;   // written by its pair
  // lane's values: columns 8 lane .. and 256 + 8 lane ..
  float acc[16], z = 0.f, m = -INFINITY;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int k0 = mine; k0 < n; k0 += kRound * SPLIT) {
    uint4 raw[kRound][kQuads];
    float w[kRound], top = m;
    float2 unit[kRound];                        // (of fp16) by the lane's two runs of columns
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      const int k = k0 + u * SPLIT;
      w[u] = -INFINITY;
      if (k >= n) continue;
      const int64_t at = static_cast<int64_t>(k == 0 ? 2 * s0 + 1 : 2 * (s0 + k)) * 128 + rr;
      const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.ws_o) + at * kLatent);
      w[u] = __ldg(a.ws_lse + at);
      if constexpr (kQuads == 2) unit[u] = __ldg(reinterpret_cast<const float2 *>(a.ws_unit) + 2 * at + (lane >> 4));
#pragma unroll
      for (int i = 0; i < kQuads; ++i)
        raw[u][i] = __ldg(src + i / (kQuads / 2) * 16 * kQuads + lane * (kQuads / 2) + i % (kQuads / 2));
    }
#pragma unroll
    for (int u = 0; u < kRound; ++u) top = fmaxf(top, w[u]);
    const float safe = top == -INFINITY ? 0.f : top, f = expf(m - safe);
    m = top;
    z *= f;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] *= f;
#pragma unroll
    for (int u = 0; u < kRound; ++u) {
      if (k0 + u * SPLIT >= n) continue;
      const float wu = expf(w[u] - safe);
      z += wu;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const uint32_t v[4] = {raw[u][i].x, raw[u][i].y, raw[u][i].z, raw[u][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kQuads == 4) {
            acc[4 * i + e] = fmaf(wu, __uint_as_float(v[e]), acc[4 * i + e]);
          } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[e]));
            const float wf = wu * (i ? unit[u].y : unit[u].x);
            acc[8 * i + 2 * e] = fmaf(wf, f.x, acc[8 * i + 2 * e]);
            acc[8 * i + 2 * e + 1] = fmaf(wf, f.y, acc[8 * i + 2 * e + 1]);
          }
        }
      }
    }
  }
  if constexpr (SPLIT > 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      part_o[warp][8 * lane + e] = acc[e];
      part_o[warp][8 * (lane + 32) + e] = acc[8 + e];
    }
    if (lane == 0) {
      part_z[warp] = z;
      part_m[warp] = m;
    }
    __syncthreads();
    if (!row_ok) return;
    // 512 / SPLIT columns a warp, in the warps' order
    constexpr int kCols = kLatent / SPLIT;
    float f[SPLIT];
#pragma unroll
    for (int w = 0; w < SPLIT; ++w) m = fmaxf(m, part_m[warp - mine + w]);
    const float safe = m == -INFINITY ? 0.f : m;
    z = 0.f;
#pragma unroll
    for (int w = 0; w < SPLIT; ++w) {
      f[w] = expf(part_m[warp - mine + w] - safe);
      z = fmaf(part_z[warp - mine + w], f[w], z);
    }
    const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
    for (int c = lane; c < kCols; c += 32) {
      float x = 0.f;
#pragma unroll
      for (int w = 0; w < SPLIT; ++w) x = fmaf(part_o[warp - mine + w][mine * kCols + c], f[w], x);
      if constexpr (sizeof(T) == 4) out[mine * kCols + c] = x * inv;
      else out[mine * kCols + c] = __float2bfloat16_rn(x * inv);
    }
  } else {
    const float inv = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] *= inv;
    store8(out + 8 * lane, acc);
    store8(out + 8 * (lane + 32), acc + 8);
  }
  // (z NaN where a part's logarithm is, which no maximum shows)
  if (mine == 0 && lane == 0) a.lse[row] = z == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + logf(z);
}

template <typename T, int SPLIT>
cudaError_t launch_merge(const WindowArgs &a, mla_stream_t stream) {
  constexpr int kRows = kMergeWarps / SPLIT;
  const int rows = std::min(128, a.q_len * a.H);
  return launch_pdl(window_merge_kernel<T, SPLIT>, dim3(a.B * a.RG, (rows + kRows - 1) / kRows),
                    dim3(kMergeWarps * 32), 0, stream, a);
}

template <typename T>
cudaError_t merge(int64_t parts, const WindowArgs &a, mla_stream_t stream) {
  return parts > 40   ? launch_merge<T, 8>(a, stream)
         : parts > 10 ? launch_merge<T, 4>(a, stream)
                      : launch_merge<T, 1>(a, stream);
}

// ------------------------------------------------------------------- host
template <bool FP8>
struct PairLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  PairLaunch(int pairs, cudaStream_t stream) {
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Fmt<FP8>::kSmem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

// CTA pairs that are resident at once (a pair needs both SMs in one GPC), at
// most one per two SMs; cached per device, with the kernels' shared memory
// allowance, which is set on the way.
int pairs_for_device() {
  constexpr int kMaxDevices = 64;
  static int cache[kMaxDevices] = {};
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (cache[dev] > 0) return cache[dev];
  const int sms = device_sm_count();
  int g = sms >= 2 ? sms / 2 : 1, n = 0;
  PairLaunch<false> pl(g, nullptr);   // (the larger of the two formats' shared memory)
  if (cudaFuncSetAttribute(window_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Fmt<false>::kSmem) != cudaSuccess ||
      cudaFuncSetAttribute(window_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Fmt<true>::kSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, window_kernel<false>, &pl.cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (n > 0) g = std::min(g, n);
  cache[dev] = g;
  return g;
}

bool shape_ok(int B, int q_len, int H) {
  if (B < 1 || q_len < 1 || q_len > 64 || H < 1 || H > 4096) return false;
  return static_cast<int64_t>(B) * q_len * ((H + 127) / 128) <= (1 << 22);
}

struct WsLayout {
  size_t o_off, lse_off, unit_off, total;
  int groups;
  int64_t group_spans;
  bool solo, fits;              // fits: the units of all jobs count in 32 bits
};

WsLayout ws_layout(int B, int q_len, int H, int max_seq_len, int window, int sinks,
                   int split_tiles, int pairs) {
  const int64_t RG = (static_cast<int64_t>(q_len) * H + 127) / 128, J = B * RG;
  // most pages of a job: the sinks' and the window's, which may begin inside
  // a page and is q_len - 1 tokens longer for the job's queries together
  int64_t pages = (static_cast<int64_t>(max_seq_len) + kPage - 1) / kPage;
  if (window > 0)
    pages = std::min(pages, (static_cast<int64_t>(window) + q_len) / kPage + 2 +
                                (static_cast<int64_t>(sinks) + kPage - 1) / kPage);
  WsLayout w{};
  w.solo = split_tiles == 0 && pages <= kSoloPages;
  w.fits = J * (pages + kJobPages) <= INT_MAX;
  w.groups = 1;
  if (w.solo) return w;   // nothing to keep
  // Row groups of a request read the same pages.  Planned apart, each over its
  // share of the pairs, they do so at the same time, and all but one read from
  // L2 - unless that leaves more than a sixteenth of the pairs idle.
  if (RG <= pairs && pairs / RG * RG * 16 >= static_cast<int64_t>(pairs) * 15) w.groups = static_cast<int>(RG);
  // (a forced split counts tiles: the smaller ones, of one page, make more)
  w.group_spans = split_tiles > 0 ? (J / w.groups * (pages + kJobPages) + split_tiles - 1) / split_tiles
                                  : pairs / w.groups;
  const size_t slots = static_cast<size_t>(2 * w.groups) * w.group_spans;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  w.o_off = up((w.groups + 2 * static_cast<size_t>(J)) * sizeof(int));
  w.lse_off = w.o_off + slots * 128 * kLatent * sizeof(float);
  w.unit_off = w.lse_off + slots * 128 * sizeof(float);
  w.total = w.unit_off + slots * 128 * 4 * sizeof(float);
  return w;
}

int check_window(const void *q, int q_dtype, float q_scale, const void *kv_cache, int kv_dtype,
                 float k_scale, const int32_t *block_table, const int32_t *seq_lens, int B,
                 int q_len, int H, int max_blocks, int num_blocks, float sm_scale, int window,
                 int sinks, int split_tiles, const void *out, int out_dtype, const float *lse) {
  if (!shape_ok(B, q_len, H) || max_blocks < 1 || num_blocks < 1 || num_blocks >= (1 << 25) ||
      window < 0 || sinks < 0 || split_tiles < 0)
    return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_blocks) * kPage > (1ll << 30)) return MLA_ERR_INVALID_ARG;
  if (!q || !kv_cache || !block_table || !seq_lens || !out || !lse) return MLA_ERR_INVALID_ARG;
  if ((q_dtype != MLA_BF16 && q_dtype != MLA_E4M3) || q_dtype != kv_dtype)
    return MLA_ERR_INVALID_ARG;
  if (out_dtype != MLA_BF16 && out_dtype != MLA_F32) return MLA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !(sm_scale < INFINITY)) return MLA_ERR_INVALID_ARG;
  if (kv_dtype == MLA_E4M3 && (!(q_scale > 0.f) || !(q_scale < INFINITY) || !(k_scale > 0.f) ||
                               !(k_scale < INFINITY)))
    return MLA_ERR_INVALID_ARG;
  // (the kernel takes scales from 2^-100 to 2^120)
  if (kv_dtype == MLA_E4M3 && (k_scale < 0x1p-100f || k_scale > 0x1p120f)) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

template <bool FP8>
int launch_pairs(const void *q, const void *kv_cache, int pairs, const WindowArgs &a,
                 mla_stream_t stream) {
  using F = Fmt<FP8>;
  const CUtensorMapDataType dt =
      FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  // {columns of a 128-byte box row, rows, box columns}; the e4m3 rope columns
  // are half a box row and have maps of their own
  const uint64_t row_bytes = static_cast<uint64_t>(kDqk) * F::kEsz;
  const uint64_t strides[2] = {row_bytes, 128};
  const uint64_t kv_rows = static_cast<uint64_t>(a.num_blocks) * kPage;
  const uint64_t q_rows = static_cast<uint64_t>(a.B) * a.q_len * a.H;
  const uint64_t kv_dims[3] = {F::kCols, kv_rows, F::kBoxes}, q_dims[3] = {F::kCols, q_rows, F::kBoxes};
  const uint64_t kvr_dims[3] = {kDqk, kv_rows, 1}, qr_dims[3] = {kDqk, q_rows, 1};
  const uint32_t box_k[3] = {F::kCols, F::kKRows, F::kBoxes}, box_q[3] = {F::kCols, 64, F::kBoxes};
  const uint32_t box_v[3] = {F::kCols, F::kVTok, F::kVBoxes}, box_r[3] = {64, 64, 1};
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B, sw_r = CU_TENSOR_MAP_SWIZZLE_64B;
  CUtensorMap tk, tkr, tv, tq, tqr;
  bool ok = make_tmap(&tk, dt, 3, kv_cache, kv_dims, strides, box_k, sw) &&
            make_tmap(&tv, dt, 3, kv_cache, kv_dims, strides, box_v, sw) &&
            make_tmap(&tq, dt, 3, q, q_dims, strides, box_q, sw);
  if constexpr (FP8) {
    ok = ok && make_tmap(&tkr, dt, 3, kv_cache, kvr_dims, strides, box_r, sw_r) &&
         make_tmap(&tqr, dt, 3, q, qr_dims, strides, box_r, sw_r);
  } else {
    tkr = tk;   // (not used)
    tqr = tq;
  }
  if (!ok) return MLA_ERR_CUDA;
  PairLaunch<FP8> pl(pairs, stream);
  return cudaLaunchKernelEx(&pl.cfg, window_kernel<FP8>, tk, tkr, tv, tq, tqr, a) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

int launch_window(const void *q, bool fp8, float q_scale, const void *kv_cache, float k_scale,
                  const float *scales, int sb_shift, const int32_t *block_table,
                  const int32_t *seq_lens, int B, int q_len, int H, int max_blocks, int num_blocks,
                  float sm_scale, int window, int sinks, int split_tiles, void *out, int out_dtype,
                  float *lse, void *workspace, size_t ws_bytes, mla_stream_t stream) {
  if (!aligned16(workspace)) return MLA_ERR_INVALID_ARG;
  const int pairs = pairs_for_device();
  if (pairs == 0) return MLA_ERR_CUDA;
  const WsLayout w = ws_layout(B, q_len, H, max_blocks * kPage, window, sinks, split_tiles, pairs);
  if (!w.fits) return MLA_ERR_INVALID_ARG;
  if (!w.solo && (!workspace || ws_bytes < w.total)) return MLA_ERR_WORKSPACE;
  WindowArgs a{};
  a.err = device_error_word();
  if (!a.err) return MLA_ERR_CUDA;
  a.scales = scales;
  a.sb_shift = sb_shift;
  a.k_scale = fp8 ? k_scale : 1.f;
  // times a scale of 2^-100 to 2^120 the factor may be in range where it is not by itself
  const double scale = static_cast<double>(sm_scale) * 1.4426950408889634 * (fp8 ? q_scale : 1.f);
  a.scale_pre = scale < 0x1p-60 ? 0x1p-100f : scale > 0x1p100 ? 0x1p100f : 1.f;
  a.scale_log2 = static_cast<float>(scale / a.scale_pre);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.B = B;
  a.q_len = q_len;
  a.H = H;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  // (a table holds at most 2^30 tokens: sums with these stay within 32 bits)
  a.window = std::min(window, 1 << 30);
  a.sinks = std::min(sinks, 1 << 30);
  a.RG = static_cast<int>((static_cast<int64_t>(q_len) * H + 127) / 128);
  a.forced = split_tiles;
  a.solo = w.solo;
  const int64_t jobs = static_cast<int64_t>(B) * a.RG;
  a.groups = w.groups;
  a.group_jobs = static_cast<int>(jobs / w.groups);
  a.group_spans = static_cast<int>(w.group_spans);
  a.spans_at_once = w.solo ? static_cast<int>(std::min<int64_t>(pairs, jobs)) : pairs / w.groups;
  a.out = out;
  a.out_f32 = out_dtype == MLA_F32;
  a.lse = lse;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.ws_head = reinterpret_cast<int *>(ws);
  a.ws_o = ws + w.o_off;
  a.ws_lse = reinterpret_cast<float *>(ws + w.lse_off);
  a.ws_unit = reinterpret_cast<float *>(ws + w.unit_off);
  const int st = fp8 ? launch_pairs<true>(q, kv_cache, a.spans_at_once * w.groups, a, stream)
                     : launch_pairs<false>(q, kv_cache, a.spans_at_once * w.groups, a, stream);
  if (st != MLA_OK || w.solo) return st;
  const int64_t parts = pairs / jobs;   // of a job, about
  const cudaError_t e = a.out_f32 ? merge<float>(parts, a, stream) : merge<__nv_bfloat16>(parts, a, stream);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_decode_window_workspace_size(int B, int q_len, int H, int max_seq_len,
                                                int window, int sinks, int split_tiles,
                                                size_t *bytes) {
  if (!bytes || !shape_ok(B, q_len, H) || max_seq_len < 0 || window < 0 || sinks < 0 ||
      split_tiles < 0)
    return MLA_ERR_INVALID_ARG;
  // (without a device: what an upper bound of pairs needs)
  const int pairs = pairs_for_device();
  const WsLayout w = ws_layout(B, q_len, H, max_seq_len, window, sinks, split_tiles, pairs ? pairs : 128);
  if (!w.fits) return MLA_ERR_INVALID_ARG;
  *bytes = w.total;
  return MLA_OK;
}

extern "C" int mla_decode_paged_window(const void *q, int q_dtype, float q_scale,
                                       const void *kv_cache, int kv_dtype, float k_scale,
                                       const int32_t *block_table, const int32_t *seq_lens, int B,
                                       int q_len, int H, int max_blocks, int num_blocks,
                                       float sm_scale, int window, int sinks, int split_tiles,
                                       void *out, int out_dtype, float *lse, void *workspace,
                                       size_t ws_bytes, mla_stream_t stream) {
  const int st = check_window(q, q_dtype, q_scale, kv_cache, kv_dtype, k_scale, block_table,
                              seq_lens, B, q_len, H, max_blocks, num_blocks, sm_scale, window,
                              sinks, split_tiles, out, out_dtype, lse);
  if (st != MLA_OK) return st;
  return launch_window(q, kv_dtype == MLA_E4M3, q_scale, kv_cache, k_scale, nullptr, 0,
                       block_table, seq_lens, B, q_len, H, max_blocks, num_blocks, sm_scale,
                       window, sinks, split_tiles, out, out_dtype, lse, workspace, ws_bytes,
                       stream);
}

extern "C" int mla_decode_paged_scaled(const void *q, float q_scale, const void *kv_cache,
                                       const float *kv_scales, int scale_block,
                                       const int32_t *block_table, const int32_t *seq_lens, int B,
                                       int q_len, int H, int max_blocks, int num_blocks,
                                       float sm_scale, int window, int sinks, int split_tiles,
                                       void *out, int out_dtype, float *lse, void *workspace,
                                       size_t ws_bytes, mla_stream_t stream) {
  if (scale_block != 16 && scale_block != 32 && scale_block != 64) return MLA_ERR_INVALID_ARG;
  const int st = check_window(q, MLA_E4M3, q_scale, kv_cache, MLA_E4M3, 1.f, block_table, seq_lens,
                              B, q_len, H, max_blocks, num_blocks, sm_scale, window, sinks,
                              split_tiles, out, out_dtype, lse);
  if (st != MLA_OK) return st;
  if (!kv_scales) return MLA_ERR_INVALID_ARG;
  return launch_window(q, true, q_scale, kv_cache, 1.f, kv_scales,
                       scale_block == 64 ? 6 : scale_block == 32 ? 5 : 4, block_table, seq_lens, B,
                       q_len, H, max_blocks, num_blocks, sm_scale, window, sinks, split_tiles, out,
                       out_dtype, lse, workspace, ws_bytes, stream);
}
