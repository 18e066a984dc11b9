// Causal prefill attention with a sliding window and sinks
// (mla_prefill_attn_window).
//
// One work item is (256 queries, head, request): two tiles A and B of 128
// queries that share every K / V tile of 128 keys.  Per key tile and query
// tile g
//   S_g = Q_g K^T   tcgen05 M = 128, N = 128, K = 192 into TMEM,
//   P_g = 2^(S_g c - m) as bf16 over S_g's columns, O_g += P_g V (P from TMEM),
// and the two query tiles alternate on the tensor core.  Only the key tiles
// that hold a sink or a key of the window are loaded, so an item has few of
// them (a window of 1024: eleven) and what comes before its first product and
// after its last one counts as much as the products.  Hence
//   * the CTAs are persistent, one per SM: the barriers, tensor memory and
//     descriptors are there already, and the next item's query and keys load
//     while the last results are written;
//   * two threads share a query row (64 keys each): S_g(t + 1) follows
//     P_g(t) V in the same columns, so a softmax's latency is on the path
//     twice a tile;
//   * query tile B leaves out the key tile that only A's window still holds;
//   * results leave 64 bytes of a row at a time.
// The MMA warp runs converged with one elected lane (descriptors stay in
// uniform registers).
//
// What bounds it: 4 x 512 queries over 8192 keys, 128 heads, a window of 1024
// take 186 us in graph replays (194 in calls on changing inputs), 0.93 PFLOP/s of
// visible pairs (1.14 of the tiles, which are partly masked) of the 1.9 that a
// product reaches.  A key tile of both query
// tiles takes 3650 cycles where its MMAs take 2560: S, softmax, P and O follow
// one another, and tensor memory is full, so no S runs ahead.  About 10000 of an
// item's 50000 cycles pass between its last product and the next item's second
// tile: the results, the query's load, and a first tile without anything beside
// it.  Tried: results by warps of their own (80 registers for the softmax: 232
// us), fewer MMA steps for the sinks' tile (196), the next item's query or keys
// fetched into L2 ahead (196, 188), a barrier for either query tile (188).
//
// Masked keys and values that are not finite: a product over a tile multiplies
// every value row, also by 0, so a NaN that a query does not see would reach
// its row.  Values behind the request's last key (padding, which may hold
// anything) are cleared in shared memory.  Where a row comes out not finite
// although its scores are, the CTA goes through its items a second time: in the
// tiles that some of an item's queries do not see as a whole (seven at most: the
// diagonal, the window's edge, the sinks' end) values that are not finite are
// then cleared as well, and put back into the rows that do see them.  That takes
// 1.9 to 2.6 times as long as without such values, however long the window (256
// queries of 160 heads over 30000 keys: 2.46 ms instead of 1.08; every value NaN:
// 4.0); calls without them pay one test a row.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kBM = 128, kBN = 128;              // query rows per tile, keys per tile
constexpr int kQT = 2;                           // query tiles per item
constexpr int kDq = 192, kDv = 128;
constexpr int kBox = 128 * 128;                  // 128 rows x 64 bf16
constexpr int kQBytes = 3 * kBox, kKBytes = 3 * kBox, kVBytes = 2 * kBox;
constexpr int kKStages = 2;
constexpr int kOffK = kQT * kQBytes;
constexpr int kOffV = kOffK + kKStages * kKBytes;
constexpr int kOffX = kOffV + kVBytes;           // [2][256] row maxima, then sums
constexpr int kOffBars = kOffX + 2 * 256 * 4;
constexpr int kSmemBytes = kOffBars + 256;
constexpr int kSoftWarps = 16;
constexpr int kThreads = (4 + kSoftWarps) * 32;
constexpr float kLazy = 16.f;                    // O follows a maximum that grew by more than 2^16
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

struct Args {
  const int32_t *cu_q, *cu_k;
  int B, H, Tq, Nk, nqp, window, sinks;          // nqp: items per (head, request)
  int items;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
  const __nv_bfloat16 *v;
  int *err;
};

// Work item and the key tiles it takes: the sinks' (list entries
// [0, sink_tiles)), then those from lo_tile on.
struct Item {
  int h, q0, nq, k0, nk, row0;                   // row0: its first query of the request
  int sink_tiles, lo_tile, ntiles;
  bool outside;                                  // the request is not within the tensors: no items
  int rows[kQT], nt[kQT], skip[kQT];             // query tile g takes entries t < nt[g], t != skip[g]

  __device__ __forceinline__ bool load(const Args &a, int i) {
    const int hb = i / a.nqp, qp = i - hb * a.nqp;
    const int b = hb / a.H;
    h = hb - b * a.H;
    q0 = __ldg(a.cu_q + b);
    nq = __ldg(a.cu_q + b + 1) - q0;
    k0 = __ldg(a.cu_k + b);
    nk = __ldg(a.cu_k + b + 1) - k0;
    row0 = qp * kQT * kBM;
    outside = (q0 | nq | k0 | nk) < 0 || nq > a.Tq - q0 || nk > a.Nk - k0;
    if (outside || row0 >= nq) return false;
    const int first = row0 + nk - nq;            // the first query's position
    const int lo = max(0, first - a.window + 1);
    lo_tile = lo / kBN;
    sink_tiles = min((min(a.sinks, lo) + kBN - 1) / kBN, lo_tile);
    ntiles = 0;
#pragma unroll
    for (int g = 0; g < kQT; ++g) {
      rows[g] = max(0, min(kBM, nq - row0 - g * kBM));
      const int end = rows[g] ? max(0, first + g * kBM + rows[g]) : 0;   // behind its last key
      nt[g] = end ? (end + kBN - 1) / kBN - lo_tile + sink_tiles : 0;
      skip[g] = -1;
      ntiles = max(ntiles, nt[g]);
    }
    // the first tile of A's window, where B's begins behind it
    if (nt[1] > 0 && max(0, first + kBM - a.window + 1) / kBN > lo_tile && lo_tile * kBN >= a.sinks)
      skip[1] = sink_tiles;
    return true;
  }
  __device__ __forceinline__ int tile(int t) const {
    return t < sink_tiles ? t : t - sink_tiles + lo_tile;
  }
  __device__ __forceinline__ bool takes(int g, int t) const { return t < nt[g] && t != skip[g]; }
  // every query that takes entry t sees all of its keys
  __device__ __forceinline__ bool whole(const Args &a, int t) const {
    const int key0 = tile(t) * kBN, first = row0 + nk - nq;
    bool all = true;
#pragma unroll
    for (int g = 0; g < kQT; ++g) {
      const int p0 = first + g * kBM, p1 = p0 + rows[g] - 1;
      if (takes(g, t) && (key0 + kBN - 1 > p0 || (key0 <= p1 - a.window && key0 + kBN > a.sinks))) all = false;
    }
    return all;
  }
};

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(e));
  return e;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t me) {
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
               "l"(b), "r"(idesc), "r"(acc), "r"(me) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t me) {
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
               "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc), "r"(me) : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar, uint32_t me) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
               "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
               ::"r"(smem_u32(bar)), "r"(me) : "memory");
}
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
  return mbar_test(bar, parity) || mbar_wait(bar, parity, abort_flag);
}
// Named barrier of 64 threads that tells each whether `v` held for all.
__device__ __forceinline__ bool named_and(uint32_t id, bool v) {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
               "barrier.cta.red.and.pred p, %1, 64, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r) : "r"(id), "r"(static_cast<uint32_t>(v)) : "memory");
  return r != 0;
}

__device__ __forceinline__ bool not_finite(uint32_t bf16_bits) { return (bf16_bits & 0x7F80u) == 0x7F80u; }

// The values of a tile in shared memory, 0 in place of what is not finite, by the
// 256 threads of a query tile.
__device__ __forceinline__ void clear_values(uint8_t *sm_v, int thread) {
  for (int u = thread; u < kVBytes / 16; u += 256) {
    uint4 *at = reinterpret_cast<uint4 *>(sm_v) + u;
    const uint4 v = *at;
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (not_finite(w[e])) any = 1, w[e] &= 0xFFFF0000u;
      if (not_finite(w[e] >> 16)) any = 1, w[e] &= 0xFFFFu;
    }
    if (any) *at = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// What the cleared values of a tile's 128 keys from key0 on leave in 64 columns of
// this thread's row, which sees the keys [0, sinks) and [wlo, lim): a bit for each
// column in marks[0..1] for infinity, [2..3] for -infinity, [4..5] for NaN.  By a
// whole warp; v: column 0 of the 64 in the request's first value row.
__device__ __forceinline__ void mark_values(const __nv_bfloat16 *v, int64_t stride, int key0, int keys, int lim,
                                            int wlo, int sinks, uint32_t *marks) {
  const int lane = lane_id();
  for (int j0 = key0; j0 < min(key0 + kBN, keys); j0 += 32) {
    bool bad = false;
    if (j0 + lane < keys) {
      const uint4 *row = reinterpret_cast<const uint4 *>(v + (j0 + lane) * stride);
      for (int e = 0; e < 8; ++e) {
        const uint4 u = __ldg(row + e);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) bad = bad || not_finite(w[k]) || not_finite(w[k] >> 16);
      }
    }
    for (uint32_t rest = __ballot_sync(0xffffffffu, bad); rest; rest &= rest - 1) {
      const int j = j0 + __ffs(rest) - 1;
      if (j >= lim || (j < wlo && j >= sinks)) continue;
      const uint16_t *row = reinterpret_cast<const uint16_t *>(v + j * stride);
      for (int c = 0; c < 64; ++c) {
        const uint32_t x = __ldg(row + c);
        if (not_finite(x)) marks[(x & 0x7Fu ? 4 : x >> 15 ? 2 : 0) + c / 32] |= 1u << (c % 32);
      }
    }
    __syncwarp();
  }
}

// Entry t of item i, the second time, by a warp of query tile g (rows' first and
// last keys wlo, lim - 1; columns 64 sub ..).  False if a wait ran out.
__device__ __noinline__ bool look_again(Args args, int i, int t, int g, int sub, int lim, int wlo,
                                        uint32_t *marks, uint8_t *sm_v, uint64_t *v_full, uint32_t phase,
                                        volatile int *abort_flag) {
  Item it;
  it.load(args, i);
  if (it.whole(args, t)) return true;
  const int64_t stride = static_cast<int64_t>(args.H) * kDv;
  mark_values(args.v + it.k0 * stride + it.h * kDv + 64 * sub, stride, it.tile(t) * kBN, it.nk, lim, wlo, args.sinks,
              marks);
  if (g != 0 && it.takes(0, t)) return true;     // (the first of the two to use it clears it)
  if (!__all_sync(0xffffffffu, wait_for(v_full, phase, abort_flag))) return false;
  clear_values(sm_v, static_cast<int>(threadIdx.x) & 255);
  fence_proxy_async_smem();
  return true;
}

// Puts what was cleared back into 64 columns of a row.
__device__ __noinline__ void put_back(__nv_bfloat16 *row, const uint32_t *marks) {
  for (int c = 0; c < 64; ++c) {
    const uint32_t bit = 1u << (c % 32);
    if (!((marks[c / 32] | marks[2 + c / 32] | marks[4 + c / 32]) & bit)) continue;
    float x = __bfloat162float(row[c]);
    if (marks[c / 32] & bit) x += INFINITY;
    if (marks[2 + c / 32] & bit) x -= INFINITY;
    if (marks[4 + c / 32] & bit) x = __uint_as_float(0x7FC00000u);
    row[c] = __float2bfloat16_rn(x);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
prefill_window_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args args) {
  extern __shared__ __align__(1024) uint8_t smem[];   // (no static shared memory: starts on 1024 bytes)
  if (smem_u32(smem) & 1023u) {                       // (never seen: the swizzled tiles need it)
    if (threadIdx.x == 0) raise_error(args.err, MLA_DEVERR_TIMEOUT);
    return;
  }
  uint8_t *sm_q = smem, *sm_k = smem + kOffK, *sm_v = smem + kOffV;
  float *xchg = reinterpret_cast<float *>(smem + kOffX);
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + kOffBars);
  uint64_t *k_empty = k_full + kKStages;
  uint64_t *v_full = k_empty + kKStages, *v_empty = v_full + 1;
  uint64_t *s_full = v_empty + 1;              // [kQT]
  uint64_t *p_full = s_full + kQT;             // [kQT]
  uint64_t *pv_done = p_full + kQT;            // [kQT]
  uint64_t *q_full = pv_done + kQT, *q_empty = q_full + 1, *drain = q_empty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  volatile int *unclean = abort_flag + 1;      // a row came out not finite
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(warp_id()), 0), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    mbar_init(v_full, 1);
    mbar_init(v_empty, 1);
    for (int g = 0; g < kQT; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&p_full[g], kSoftWarps / kQT);
      mbar_init(&pv_done[g], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *unclean = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == 2 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();
  grid_dep_launch();
  // Every warp goes through the items once, and together a second time if this says so.
  auto once_more = [&](bool second) -> bool {
    __syncthreads();
    const bool again = !second && *unclean && !*abort_flag;
    if (again) __syncthreads();                // (all read the same before one goes on)
    return again;
  };
  bool second = false;

  if (warp == 0) {
    // ------------------------------------------------------ Q and K
    int kc = 0, n = 0;                         // K tiles, items with tiles so far
    do if (lane == 0) {
      bool ok = true;
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        Item it;
        const bool item = it.load(args, i);
        if (it.outside) raise_error(args.err, MLA_DEVERR_RANGE);
        if (!item || it.ntiles == 0) continue;
        if (n > 0 && !(ok = wait_for(q_empty, (n - 1) & 1, abort_flag))) break;
        ++n;
        mbar_arrive_expect_tx(q_full, (it.rows[1] > 0 ? 2 : 1) * kQBytes);
        for (int g = 0; g < kQT; ++g)
          if (it.rows[g] > 0)
            for (int d = 0; d < 3; ++d)
              tma_load_3d(sm_q + g * kQBytes + d * kBox, &tm_q, q_full, 64 * d, it.h,
                          it.q0 + it.row0 + g * kBM);
        for (int t = 0; t < it.ntiles; ++t, ++kc) {
          const int s = kc % kKStages;
          if (kc >= kKStages && !(ok = wait_for(&k_empty[s], ((kc / kKStages) - 1) & 1, abort_flag)))
            break;
          mbar_arrive_expect_tx(&k_full[s], kKBytes);
          for (int d = 0; d < 3; ++d)
            tma_load_3d(sm_k + s * kKBytes + d * kBox, &tm_k, &k_full[s], 64 * d, it.h,
                        it.k0 + it.tile(t) * kBN);
        }
      }
      if (*abort_flag) {
        volatile int no_abort = 0;
        for (int u = max(0, kc - kKStages); u < kc; ++u)
          mbar_wait(&k_full[u % kKStages], (u / kKStages) & 1, &no_abort);
        if (n > 0) mbar_wait(q_full, (n - 1) & 1, &no_abort);
      }
    } while (once_more(second) && (second = true));
  } else if (warp == 2) {
    // ------------------------------------------------------------ V
    int vc = 0;
    do if (lane == 0) {
      bool ok = true;
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        Item it;
        if (!it.load(args, i)) continue;
        for (int t = 0; t < it.ntiles; ++t, ++vc) {
          if (vc > 0 && !(ok = wait_for(v_empty, (vc - 1) & 1, abort_flag))) break;
          mbar_arrive_expect_tx(v_full, kVBytes);
          for (int d = 0; d < 2; ++d)
            tma_load_3d(sm_v + d * kBox, &tm_v, v_full, 64 * d, it.h, it.k0 + it.tile(t) * kBN);
        }
      }
      if (*abort_flag && vc > 0) {
        volatile int no_abort = 0;
        mbar_wait(v_full, (vc - 1) & 1, &no_abort);
      }
    } while (once_more(second) && (second = true));
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMAs
    const uint32_t me = elect_one();
    const uint32_t idesc_qk = idesc_bf16(128, kBN, false, false);
    const uint32_t idesc_pv = idesc_bf16(128, kDv, false, true);
    auto wait = [&](uint64_t *bar, int phase) -> bool {
      return __all_sync(0xffffffffu, wait_for(bar, phase & 1, abort_flag));
    };
    int kc = 0, vc = 0, n = 0;                 // K tiles, V tiles, items so far
    int pc[kQT] = {0, 0};                      // tiles of query tile g so far
    bool ok = true;
    auto issue_qk = [&](int g, int kslot) {
      const uint32_t qa = smem_u32(sm_q) + g * kQBytes, kb = smem_u32(sm_k) + kslot * kKBytes;
#pragma unroll
      for (int k = 0; k < kDq / 16; ++k)
        mma_ss(tmem + 256 * g, sdesc(qa + (k >> 2) * kBox + (k & 3) * 32, 16, 1024, kSwizzle128B),
               sdesc(kb + (k >> 2) * kBox + (k & 3) * 32, 16, 1024, kSwizzle128B), idesc_qk, k > 0, me);
      commit(&s_full[g], me);
    };
    auto issue_pv = [&](int g, bool first) {
      const uint32_t vb = smem_u32(sm_v);
#pragma unroll
      for (int k = 0; k < kBN / 16; ++k)       // (P of either half of the keys over its own scores)
        mma_ts(tmem + 256 * g + 128, tmem + 256 * g + 64 * (k >> 2) + 8 * (k & 3),
               sdesc(vb + k * 2048, kBox, 1024, kSwizzle128B), idesc_pv, first && k == 0 ? 0u : 1u, me);
      commit(&pv_done[g], me);
    };
    do {
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        Item it;
        if (!it.load(args, i) || it.ntiles == 0) continue;
        bool begun[kQT] = {false, false};
        if (!(ok = wait(q_full, n++))) break;
        // QK(0) of both; then per tile t: PV_A(t), QK_A(t+1), PV_B(t), QK_B(t+1).
        // QK_g(t+1) overwrites S_g after PV_g(t) has read P_g from the same
        // columns (the tensor core runs one thread's MMAs in order).
        if (!(ok = wait(&k_full[kc % kKStages], kc / kKStages))) break;
        tc_fence_after();
#pragma unroll
        for (int g = 0; g < kQT; ++g)
          if (it.takes(g, 0)) issue_qk(g, kc % kKStages);
        commit(&k_empty[kc % kKStages], me);
        ++kc;
        if (it.ntiles == 1) commit(q_empty, me);
        for (int t = 0; ok && t < it.ntiles; ++t) {
          if (!(ok = wait(v_full, vc))) break;
          ++vc;
          bool k_there = false;
#pragma unroll
          for (int g = 0; g < kQT; ++g) {
            if (!ok) break;
            if (it.takes(g, t)) {
              if (!(ok = wait(&p_full[g], pc[g]))) break;
              ++pc[g];
              tc_fence_after();
              issue_pv(g, !begun[g]);
              begun[g] = true;
            }
            if (g == kQT - 1) commit(v_empty, me);
            if (it.takes(g, t + 1)) {
              if (!k_there && !(ok = wait(&k_full[kc % kKStages], kc / kKStages))) break;
              tc_fence_after();
              k_there = true;
              issue_qk(g, kc % kKStages);
            }
          }
          if (!ok) break;
          if (t + 1 < it.ntiles) {
            commit(&k_empty[kc % kKStages], me);
            ++kc;
            if (t + 2 == it.ntiles) commit(q_empty, me);
          }
        }
      }
      if (*abort_flag) {
        commit(drain, me);
        volatile int no_abort = 0;
        mbar_wait(drain, 0, &no_abort);
      }
    } while (once_more(second) && (second = true));
  } else if (warp >= 4) {
    // -------------------------------------- softmax and results of tile g
    const int g = (warp - 4) >> 3, sub = ((warp - 4) >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane;           // query row of the tile
    const uint32_t lane_base = tmem + ((quarter * 32u) << 16);
    const uint32_t col_s = 256 * g + 64 * sub, col_o = 256 * g + 128 + 64 * sub;
    float *mine = xchg + 256 * sub + 128 * g + r, *its = xchg + 256 * (sub ^ 1) + 128 * g + r;
    const uint32_t bar_id = 1 + 4 * g + quarter;   // the two warps of the same rows
    // The hardware barrier has no limit, so neither warp may leave the other
    // in it: it takes along whether all is well, a warp whose wait ran out goes
    // through it once more before it leaves, and the other leaves behind it.
    bool told = false;
    auto exchange = [&](float v) -> float {
      *mine = v;
      told = !named_and(bar_id, true);
      return *its;
    };
    auto all_ok = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
    int c = 0, vc = 0;                           // tiles of query tile g, V tiles so far
    bool ok = true;
    uint32_t marks[6];                           // (second time) by columns: infinity, -infinity, NaN
    do {
      for (int i = blockIdx.x; ok && i < args.items; i += gridDim.x) {
        Item it;
        if (!it.load(args, i)) continue;
        const int vc0 = vc;
        vc += it.ntiles;
        // (selects: an index would put the arrays into local memory)
        const int nt = g ? it.nt[1] : it.nt[0], skip = g ? it.skip[1] : -1;
        const int rows = g ? it.rows[1] : it.rows[0];
        if (rows == 0) continue;
        const int q = it.row0 + g * kBM + r;       // query of the request
        const int lim = min(it.nk, q + it.nk - it.nq + 1);
        const int wlo = lim - args.window;         // the window's first key
        // sums of the probabilities, for the logarithm, and of their rounded values,
        // for the results: a large one's rounding is then in both parts of the quotient
        // (which counts where few keys have most of the weight)
        float m = -INFINITY, l = 0.f, lr = 0.f;
        bool any = false;
        if (second)
          for (uint32_t &w : marks) w = 0;
        for (int t = 0; t < nt; ++t) {
          if (t == skip) continue;
          const int key0 = it.tile(t) * kBN + 64 * sub;
          const bool masked = key0 + 64 > lim || (key0 < wlo && key0 + 64 > args.sinks);
          if (!(ok = all_ok(wait_for(&s_full[g], c & 1, abort_flag)))) break;
          tc_fence_after();
          // 32 scores at a time, read once for the maximum and once for the
          // exponentials: 64 at once would not fit the 96 registers that 20
          // warps have
          // (a bit for each of the 64 keys that this query sees: three compares
          // for each score made a masked tile cost twice an unmasked one)
          const uint64_t seen = masked ? low_bits(lim - key0) & (~low_bits(wlo - key0) | low_bits(args.sinks - key0))
                                       : ~uint64_t(0);
          auto load = [&](int h, float *x) {
            tmem_ld_x32(lane_base + col_s + 32 * h, reinterpret_cast<uint32_t *>(x));
            if (masked) {
              const uint32_t w = static_cast<uint32_t>(seen >> (32 * h));
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = w & (1u << k) ? x[k] : -INFINITY;
            }
          };
          // 32 rows by 32 keys that nobody sees need no exponentials: 6 of 16 of
          // the tiles on the diagonal and at the window's edge, 15 of a few sinks'
          const bool none[2] = {!__any_sync(0xffffffffu, static_cast<uint32_t>(seen) != 0),
                                !__any_sync(0xffffffffu, static_cast<uint32_t>(seen >> 32) != 0)};
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (none[h]) continue;
            float x[32];
            load(h, x);
#pragma unroll
            for (int k = 0; k < 32; k += 2) mx[(k >> 1) & 3] = fmax3(mx[(k >> 1) & 3], x[k], x[k + 1]);
          }
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * args.scale_log2;
          const float other = exchange(top);
          if (told) {
            ok = false;
            break;
          }
          top = fmaxf(top, other);
          const bool move = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
          float f = 1.f;
          if (move) {
            f = m == -INFINITY ? 0.f : ex2(m - top);
            m = top;
            l *= f;
            lr *= f;
          }
          const bool rescale = any && __any_sync(0xffffffffu, move);
          const float nm = m == -INFINITY ? 0.f : -m, sc = args.scale_log2;
          float ps[4] = {0.f, 0.f, 0.f, 0.f}, pr[2] = {0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];   // over scores that this thread has read: of the first half, then of both
            if (none[h]) {
#pragma unroll
              for (int k = 0; k < 16; ++k) pk[k] = 0;
              tmem_st_x16(lane_base + col_s + 16 * h, pk);
              continue;
            }
            float x[32];
            load(h, x);
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              fma_f32x2(x[k], x[k + 1], x[k], x[k + 1], sc, sc, nm, nm);
              fma_f32x2(x[k + 2], x[k + 3], x[k + 2], x[k + 3], sc, sc, nm, nm);
#pragma unroll
              for (int e = 0; e < 4; ++e) x[k + e] = ex2(x[k + e]);
              add_f32x2(ps[0], ps[1], ps[0], ps[1], x[k], x[k + 1]);
              add_f32x2(ps[2], ps[3], ps[2], ps[3], x[k + 2], x[k + 3]);
            }
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              pk[k] = bf16x2_rn(x[2 * k], x[2 * k + 1]);
              add_f32x2(pr[0], pr[1], pr[0], pr[1], __uint_as_float(pk[k] << 16),
                        __uint_as_float(pk[k] & 0xFFFF0000u));
            }
            tmem_st_x16(lane_base + col_s + 16 * h, pk);
          }
          l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
          lr += pr[0] + pr[1];
          if (rescale) {
            // O follows the maximum, now that the last P V is done (64 columns
            // for either thread of the row)
            if (!(ok = all_ok(wait_for(&pv_done[g], (c - 1) & 1, abort_flag)))) break;
            tc_fence_after();
#pragma unroll 1
            for (int o0 = 0; o0 < 64; o0 += 32) {
              uint32_t o[32];
              tmem_ld_x32(lane_base + col_o + o0, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st_x32(lane_base + col_o + o0, o);
            }
          }
          const int inside = it.nk - it.tile(t) * kBN;   // rows of the tile that are this request's
          if (inside < kBN && (g == 0 || !it.takes(0, t))) {   // (the first of the two to use it)
            // (its scores being there, the V tiles before it are: no parity is mistaken)
            if (!(ok = all_ok(wait_for(v_full, (vc0 + t) & 1, abort_flag)))) break;
            for (int u = ((warp - 4) & 7) * 32 + lane; u < (kBN - inside) * 16; u += 256)
              *reinterpret_cast<uint4 *>(sm_v + (u & 8 ? kBox : 0) + (inside + (u >> 4)) * 128 + (u & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          if (second && !(ok = look_again(args, i, t, g, sub, lim, wlo, marks, sm_v, v_full, (vc0 + t) & 1, abort_flag)))
            break;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[g]);
          any = true;
          ++c;
        }
        if (!ok) break;
        if (any && !(ok = all_ok(wait_for(&pv_done[g], (c - 1) & 1, abort_flag)))) break;
        tc_fence_after();
        {
          l += exchange(l);
          if (!told) {
            // the second sum goes into the slot that this thread has just read, and
            // the other's is in its own: what a thread writes next nobody reads any more
            *its = lr;
            told = !named_and(bar_id, true);
            lr += *mine;
          }
          if (told) {
            ok = false;
            break;
          }
        }
        const bool row_ok = r < rows;
        const int64_t orow = static_cast<int64_t>(it.q0 + q) * args.H + it.h;
        const bool empty = l == 0.f;
        const float inv = empty ? 0.f : 1.f / lr;
        float not_fin = 0.f;                       // NaN if a column is not finite
#pragma unroll 1
        for (int o0 = 0; o0 < 64; o0 += 32) {
          uint32_t o[32];
          if (any) tmem_ld_x32(lane_base + col_o + o0, o);
          if (__any_sync(0xffffffffu, empty)) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (empty) o[k] = 0;
          }
          float nan = 0.f, nan2 = 0.f;
#pragma unroll
          for (int k = 0; k < 32; k += 2)
            fma_f32x2(nan, nan2, __uint_as_float(o[k]), __uint_as_float(o[k + 1]), 0.f, 0.f, nan, nan2);
          nan += nan2;
          const int col = 64 * sub + o0;
          not_fin += nan;
          __syncwarp();
          // four lanes turn their rows' four 16-byte chunks round, so that a
          // store covers 64 bytes of eight rows and not 16 of 32 (which took
          // 4000 cycles an item)
          uint4 w[4];
          auto f = [&](int k) {
            float a, b;
            fma_f32x2(a, b, __uint_as_float(o[k]), __uint_as_float(o[k + 1]), inv, inv, -0.f, -0.f);
            return bf16x2_rn(a, b);
          };
#pragma unroll
          for (int ch = 0; ch < 4; ++ch)
            w[ch] = make_uint4(f(8 * ch), f(8 * ch + 2), f(8 * ch + 4), f(8 * ch + 6));
#pragma unroll
          for (int s = 1; s < 4; s <<= 1) {
            const bool up = lane & s;
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {
              if (ch & s) continue;
              uint4 give = up ? w[ch] : w[ch | s];
              give.x = __shfl_xor_sync(0xffffffffu, give.x, s);
              give.y = __shfl_xor_sync(0xffffffffu, give.y, s);
              give.z = __shfl_xor_sync(0xffffffffu, give.z, s);
              give.w = __shfl_xor_sync(0xffffffffu, give.w, s);
              if (up) w[ch] = give;
              else w[ch | s] = give;
            }
          }
          const int r0 = quarter * 32 + (lane & ~3);
          __nv_bfloat16 *dst = args.out + ((static_cast<int64_t>(it.q0) + it.row0 + g * kBM + r0) * args.H + it.h) * kDv +
                               col + 8 * (lane & 3);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (r0 + k < rows) *reinterpret_cast<uint4 *>(dst + static_cast<int64_t>(k) * args.H * kDv) = w[k];
        }
        // (a row whose own scores are not finite, l NaN, is as it should be)
        if (row_ok && l > 0.f && not_fin != 0.f) *unclean = 1;
        if (second) {
          __syncwarp();                            // (other lanes have stored the row)
          if (row_ok) put_back(args.out + orow * kDv + 64 * sub, marks);
        }
        if (row_ok && sub == 0)
          args.lse[orow] = empty ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        tc_fence_before();
      }
      if (!told) named_and(bar_id, ok && !*abort_flag);
    } while (once_more(second) && (second = true));
  } else {
    while (once_more(second)) second = true;
  }
  if (threadIdx.x == 0 && *abort_flag) raise_error(args.err, MLA_DEVERR_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_prefill_attn_window(const void *q, const void *k, const void *v,
                                       const int32_t *cu_q, const int32_t *cu_k, int B, int Tq,
                                       int Nk, int H, int max_q_len, int window, int sinks,
                                       float sm_scale, void *out, float *lse,
                                       mla_stream_t stream) {
  if (window < 1 || sinks < 0) return MLA_ERR_INVALID_ARG;
  if (B < 1 || Tq < 0 || Nk < 0 || H < 1 || H > 65535 || max_q_len < 0 || B > 65535)
    return MLA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !(sm_scale < INFINITY)) return MLA_ERR_INVALID_ARG;
  if (Tq == 0 || max_q_len == 0) return MLA_OK;
  if (!q || !k || !v || !cu_q || !cu_k || !out || !lse) return MLA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return MLA_ERR_INVALID_ARG;
  Args a{};
  a.err = device_error_word();
  if (!a.err) return MLA_ERR_CUDA;
  const uint32_t box[3] = {64, 1, 128};
  auto encode = [&](CUtensorMap *map, const void *base, int width, int64_t rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(width), static_cast<uint64_t>(H),
                              static_cast<uint64_t>(std::max<int64_t>(rows, 1))};
    const uint64_t strides[2] = {static_cast<uint64_t>(width) * 2,
                                 static_cast<uint64_t>(H) * width * 2};
    return make_tmap(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
  };
  CUtensorMap tq, tk, tv;
  if (!encode(&tq, q, kDq, Tq) || !encode(&tk, k, kDq, Nk) || !encode(&tv, v, kDv, Nk))
    return MLA_ERR_CUDA;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.B = B;
  a.H = H;
  a.Tq = Tq;
  a.Nk = Nk;
  a.nqp = (max_q_len - 1) / (kQT * kBM) + 1;
  const int64_t items = static_cast<int64_t>(a.nqp) * H * B;
  if (items > INT32_MAX - 1024) return MLA_ERR_INVALID_ARG;   // (and a grid's step on top)
  a.items = static_cast<int>(items);
  // (no request has 2^30 keys: sums with these stay within 32 bits)
  a.window = std::min(window, 1 << 30);
  a.sinks = std::min(sinks, 1 << 30);
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = static_cast<__nv_bfloat16 *>(out);
  a.lse = lse;
  a.v = static_cast<const __nv_bfloat16 *>(v);
  const int sms = device_sm_count();
  if (sms < 1 || cudaFuncSetAttribute(prefill_window_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      kSmemBytes) != cudaSuccess)
    return MLA_ERR_CUDA;
  const int grid = std::min(sms, a.items);
  return launch_pdl(prefill_window_kernel, dim3(grid), dim3(kThreads), kSmemBytes, stream, tq, tk, tv, a) ==
                 cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}
