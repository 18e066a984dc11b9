// The pages of a paged cache: copied, shared by sequences that go on from
// others, given to sequences that grow and taken from those that end, moved to
// the front of the pool, and the accepted rows of a drafted tree moved together
// (mla_cache_copy, _fork, _resize, _compact, _accept).
//
// State.  refs[page] counts the block-table entries that hold a page, 0 is a
// free one; with the table and the lengths that is all there is (no list of free
// pages, whose order would depend on the order of calls).  A call takes the
// lowest free pages, so what comes out depends on the state alone.
//
// Bookkeeping runs in one cluster of 8 CTAs: every CTA works out the calls'
// rows for itself (a prefix sum over them in shared memory), the cluster's
// warps count the free pages of a run of refs each, the CTAs' counts cross
// through distributed shared memory, and each free page then finds the row that
// it goes to by the number of free pages in front of it.  Latency is all it costs:
// two or three cluster barriers and as many rounds of loads.  On the device, calls
// behind one another: a resize 2.5 to 2.9 us that has nothing to do, 4.1 to 5.2 otherwise,
// in pools of up to 60000 pages; the bookkeeping of 64 forks of 100 pages each 6.9; a
// compaction of 48 sequences that finds nothing to move 4.9 with its empty copy.
//
// Copies take a list of pages from the bookkeeping kernel (or the caller) and
// go over all layers' caches in one launch: 500 pages of 12 e4m3 layers, 442 MB, in
// 69.4 us, 0.95 of a plain copy's rate; 6 pages of 4 bf16 layers in 3.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <algorithm>
#include <climits>

#include "common.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kMaxPools = 200;       // (their addresses and sizes are kernel arguments, of 4 KB at most)
constexpr int kMaxPairs = 1 << 16;   // of mla_cache_copy
constexpr int kMaxRows = 8192;       // sequences of a call, and forks: 5 words of shared memory for both
constexpr int kCtas = 8, kMaxThreads = 1024, kMaxWarps = kMaxThreads / 32;
static_assert(kMaxWarps <= 32 && kCtas <= 32, "a lane each");

// Threads of a CTA: few where there is little to count (64 forks of 8 sequences in a
// pool of 1500 pages, with the free in front of it and no copies, 256 / 512 / 1024 threads:
// 11.3 / 12.0 / 13.1 us; a resize of 8 sequences in one of 1500 pages 4.1 / 4.3 / 5.0, of
// 60000 5.2 / 5.2 / 5.7, of 140000 6.5 / 5.9 / 6.3, of 500000 11.0 / 8.4 / 7.7).
int threads_for(int num_blocks, int rows) {
  return num_blocks <= (1 << 14) && rows <= 512 ? 256 : num_blocks <= (1 << 17) && rows <= 1024 ? 512 : kMaxThreads;
}
__device__ __forceinline__ int warps_of() { return blockDim.x >> 5; }

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

__device__ __forceinline__ int warp_incl(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Sum over the CTA's threads in front of this one; total: over all of them.
__device__ __forceinline__ int block_excl(int x, int &total) {
  __shared__ int sums[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, incl = warp_incl(x);
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  const int of = warp_incl(lane < warps_of() ? sums[lane] : 0);
  total = __shfl_sync(0xffffffffu, of, 31);
  const int before = __shfl_sync(0xffffffffu, of, max(warp - 1, 0));
  return incl - x + (warp ? before : 0);
}

// The first of n ascending numbers that is over x.
__device__ __forceinline__ int first_over(const int *v, int n, int x) {
  int lo = 0;
  while (n > 0) {
    const int half = n >> 1;
    if (v[lo + half] <= x) {
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  return lo;
}

// A CTA writes into the others' shared memory only once all have started:
// arrive at the kernel's start, wait before the first such store.
__device__ __forceinline__ void cluster_started() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  sm100::cluster_sync();
}

// The pages that `is` says of their count, numbered in the order of the pages
// by the cluster's warps, which have a run of `per` pages each.
struct Scan {
  static constexpr int kHeld = 16;   // rounds of 128 pages that are kept from count() to each()
  const int32_t *refs;
  int num_blocks, per, first;
  uint64_t held;
  int before, all;

  __device__ Scan(const int32_t *r, int n, int rank) : refs(r), num_blocks(n), held(0) {
    const int all_warps = kCtas * warps_of();
    per = ((n + all_warps - 1) / all_warps + 127) / 128 * 128;
    first = min(static_cast<int64_t>(rank * warps_of() + (threadIdx.x >> 5)) * per, static_cast<int64_t>(n));
  }
  // Four pages' bits at a time (refs is written by other SMs in this launch: read from L2)
  template <typename Is>
  __device__ uint32_t four(int id, Is is) const {
    if (id + 3 < num_blocks) {
      const int4 v = __ldcg(reinterpret_cast<const int4 *>(refs + id));
      return is(v.x) | is(v.y) << 1 | is(v.z) << 2 | is(v.w) << 3;
    }
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (id + k < num_blocks) m |= is(__ldcg(refs + id + k)) << k;
    return m;
  }
  __device__ int end() const { return min(first + per, num_blocks); }
  // Of a lane's pages
  template <typename Is>
  __device__ int count_mine(Is is) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int id = first + 4 * lane, r = 0; id < end(); id += 512) {
      uint32_t m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = id + 128 * k < end() ? four(id + 128 * k, is) : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k, ++r) {
        n += __popc(m[k]);
        if (r < kHeld) held |= static_cast<uint64_t>(m[k]) << (4 * r);
      }
    }
    return n;
  }
  // (refs and sums of the cluster's CTAs; the barrier in it orders what they wrote before)
  template <typename Is>
  __device__ void count(Is is, int rank) {
    join(count_mine(is), rank);
  }
  __device__ void join(int n, int rank) {
    __shared__ int of_warp[kMaxWarps], of_cta[kCtas];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) of_warp[warp] = n;
    __syncthreads();
    if (warp == 0) {
      const int sum = __reduce_add_sync(0xffffffffu, lane < warps_of() ? of_warp[lane] : 0);
      if (lane < kCtas)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sm100::peer_smem(&of_cta[rank], lane)), "r"(sum)
                     : "memory");
    }
    cluster_barrier();
    before = __reduce_add_sync(0xffffffffu, lane < warp ? of_warp[lane] : 0);
    all = 0;
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
      if (c < rank) before += of_cta[c];
      all += of_cta[c];
    }
  }
  // emit(page, its number) for the pages whose number is below `most`
  template <typename Is, typename Emit>
  __device__ void each(Is is, int most, Emit emit) const {
    const int lane = threadIdx.x & 31;
    int at = before;
    for (int r = 0, id0 = first; id0 < end() && at < most; id0 += 128, ++r) {
      const int id = id0 + 4 * lane;
      uint32_t m = r < kHeld ? static_cast<uint32_t>(held >> (4 * r)) & 15u : id < end() ? four(id, is) : 0;
      const int n = __popc(m), incl = warp_incl(n);
      int number = at + incl - n;
      at += __shfl_sync(0xffffffffu, incl, 31);
      for (; m; m &= m - 1, ++number)
        if (number < most) emit(id + __ffs(m) - 1, number);
    }
  }
};

__device__ __forceinline__ uint32_t is_free(int refs) { return refs == 0; }
__device__ __forceinline__ uint32_t is_live(int refs) { return refs > 0; }

struct Seqs {
  int32_t *refs;
  int num_blocks;
  int32_t *table, *lens;
  int B, max_blocks;
  int *err;
};

// The rows' entries dealt out to the cluster's warps: where there are few rows
// several warps share one.
constexpr int kAtOnce = 4;             // entries of a lane on their way
struct Share {
  int first, step, lane0, lanes;
  __device__ Share(int rows, int wid) {
    const int all_warps = kCtas * warps_of(), per = rows >= all_warps ? 1 : 1 << (31 - __clz(all_warps / rows));
    first = wid / per;
    step = all_warps / per;
    lane0 = 32 * (wid % per);
    lanes = 32 * per;
  }
};

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kMaxThreads, 1)
resize_kernel(const __grid_constant__ Seqs s, const int32_t *__restrict__ new_lens) {
  extern __shared__ int rows[];
  // pages; needed ones up to and with this row; the new length (-1: it stays as it is)
  int *had = rows, *want = rows + s.B, *end = rows + 2 * s.B, *goal = rows + 3 * s.B;
  cluster_started();
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, rank = static_cast<int>(sm100::cluster_rank());
  const int wid = rank * warps_of() + (tid >> 5), most = s.max_blocks * kPage;
  const int per = (s.B + blockDim.x - 1) / blockDim.x, r0 = min(tid * per, s.B), r1 = min(r0 + per, s.B);
  auto ok = [&](int len) { return len >= 0 && len <= most; };
  int sum = 0;
  for (int b = r0; b < r1; ++b) {
    const int old = s.lens[b], now = new_lens[b];
    const bool valid = ok(old) && ok(now);
    if (!valid && rank == 0) raise_error(s.err, MLA_DEVERR_SEQ_LEN);
    const int h = valid ? pages_of(old) : 0, w = valid ? pages_of(now) : 0;
    had[b] = h;
    want[b] = w;
    goal[b] = valid ? now : -1;
    end[b] = sum += max(0, w - h);
  }
  int total;
  const int before = block_excl(sum, total);
  for (int b = r0; b < r1; ++b) end[b] += before;
  cluster_wait();
  __syncthreads();
  {
    const Share share(s.B, wid);
    for (int b = share.first; b < s.B; b += share.step) {
      int32_t *row = s.table + static_cast<int64_t>(b) * s.max_blocks;
      const int k1 = had[b];
      for (int k0 = want[b] + share.lane0 + lane; k0 < k1; k0 += kAtOnce * share.lanes) {
        int page[kAtOnce], was[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) page[i] = k0 + i * share.lanes < k1 ? row[k0 + i * share.lanes] : 0;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int k = k0 + i * share.lanes;
          was[i] = 1;
          if (k >= k1) continue;
          row[k] = -1;
          if (page[i] >= 0 && page[i] < s.num_blocks) was[i] = atomicSub(s.refs + page[i], 1);
          else raise_error(s.err, MLA_DEVERR_BLOCK_ID);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          if (was[i] > 0) continue;
          atomicAdd(s.refs + page[i], 1);          // it was free
          raise_error(s.err, MLA_DEVERR_PAGES);
        }
      }
    }
  }
  cluster_barrier();   // (whether or not there was anything: no CTA goes by what it alone has read)
  Scan scan(s.refs, s.num_blocks, rank);
  if (total == 0) scan.first = s.num_blocks;   // (nothing to count)
  scan.count(is_free, rank);
  // every CTA has read the lengths
  if (rank == 0) {
    for (int b = r0; b < r1; ++b) {
      if (goal[b] < 0) continue;
      if (want[b] > had[b] && end[b] > scan.all) raise_error(s.err, MLA_DEVERR_PAGES);
      else s.lens[b] = goal[b];
    }
  }
  scan.each(is_free, total, [&](int page, int number) {
    const int b = first_over(end, s.B, number), need = want[b] - had[b];
    if (end[b] > scan.all) return;
    s.table[static_cast<int64_t>(b) * s.max_blocks + had[b] + number - (end[b] - need)] = page;
    s.refs[page] = 1;
  });
}

// Pages to copy: from src[k] to dst[k] (dst < 0: none) the first rows[k] rows.
struct List {
  int32_t *src, *dst, *rows;
};

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kMaxThreads, 1)
fork_kernel(const __grid_constant__ Seqs s, const int32_t *__restrict__ parents,
            const int32_t *__restrict__ children, int n, const __grid_constant__ List list) {
  extern __shared__ int rows[];
  // first fork to a row; own pages up to and with this fork (before that: its parent's last
  // page); parent, child (-1: left out) and length
  int *first = rows, *end = rows + s.B, *from = end + n, *to = from + n, *length = to + n;
  cluster_started();
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, rank = static_cast<int>(sm100::cluster_rank());
  const int wid = rank * warps_of() + (tid >> 5), most = s.max_blocks * kPage;
  const int per = (n + blockDim.x - 1) / blockDim.x, i0 = min(tid * per, n), i1 = min(i0 + per, n);
  auto row_ok = [&](int b) { return b >= 0 && b < s.B; };
  auto len_ok = [&](int len) { return len >= 0 && len <= most; };
  auto entry = [&](int p, int e) { return s.table[static_cast<int64_t>(p) * s.max_blocks + e]; };
  // A page can be shared, or copied from, if somebody holds it: one that nobody does is
  // given away by this very call.  0, or the error (refs: read from L2, see Scan)
  auto fault_of = [&](int page) {
    if (page < 0 || page >= s.num_blocks) return static_cast<int>(MLA_DEVERR_BLOCK_ID);
    return __ldcg(s.refs + page) > 0 ? 0 : static_cast<int>(MLA_DEVERR_PAGES);
  };
  for (int b = tid; b < s.B; b += blockDim.x) first[b] = INT_MAX;
  for (int i = i0; i < i1; ++i) {
    from[i] = parents[i];
    to[i] = children[i];
  }
  __syncthreads();
  int child_len = 0;                        // of the last of this thread's forks (of several: read again)
  bool some = false;
  for (int i = i0; i < i1; ++i) {
    if (row_ok(to[i])) {
      atomicMin(first + to[i], i);
      child_len = s.lens[to[i]];
    }
    const int len = row_ok(from[i]) ? s.lens[from[i]] : 0;
    const bool part = len_ok(len) && len % kPage;
    length[i] = len;
    end[i] = part ? entry(from[i], len / kPage) : -1;
    some |= part;
  }
  some = __syncthreads_or(some);
  // The entries of the warp's first fork are asked for along with the pages' counts, and
  // then the counts of them, and of the last pages
  const Share share(n, wid);
  int page[kAtOnce], fault[kAtOnce];
  auto fetch = [&](int p, int len, int e0) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      page[i] = e0 + i * share.lanes < len / kPage ? entry(p, e0 + i * share.lanes) : -1;
  };
  auto look = [&] {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) fault[i] = fault_of(page[i]);
  };
  const int e_first = share.lane0 + lane, f = share.first;
  fetch(f < n ? from[f] : 0, f < n && row_ok(from[f]) && len_ok(length[f]) ? length[f] : 0, e_first);
  Scan scan(s.refs, s.num_blocks, rank);
  if (!some) scan.first = s.num_blocks;     // (nothing to count)
  const int mine = scan.count_mine(is_free);
  look();
  int sum = 0;
  for (int i = i0; i < i1; ++i) {
    const int p = from[i], c = to[i], len = length[i];
    int bits = 0;
    if (!row_ok(p) || !row_ok(c)) bits = MLA_DEVERR_RANGE;
    else if (first[c] != i || (per == 1 ? child_len : s.lens[c]) != 0) bits = MLA_DEVERR_PAGES;
    else if (!len_ok(len)) bits = MLA_DEVERR_SEQ_LEN;
    bool own = false;
    if (bits) {
      to[i] = -1;
    } else if (len % kPage) {
      // (a last page that is none: the child has a hole there too, and takes no page)
      bits = fault_of(end[i]);
      own = !bits;
    }
    if (bits && rank == 0) raise_error(s.err, bits);
    end[i] = sum += own;
  }
  int total;
  const int before = block_excl(sum, total);
  for (int i = i0; i < i1; ++i) end[i] += before;
  cluster_wait();
  __syncthreads();
  scan.join(mine, rank);
  for (int i = share.first; i < n; i += share.step) {
    const int len = length[i], p = from[i], c = to[i];
    const bool own = end[i] > (i > 0 ? end[i - 1] : 0), fails = own && end[i] > scan.all;
    const bool one = lane + share.lane0 == 0;
    if (one) {
      if (fails) raise_error(s.err, MLA_DEVERR_PAGES);
      if (!own || fails) list.dst[i] = -1;
    }
    if (c < 0 || fails) continue;
    int32_t *row = s.table + static_cast<int64_t>(c) * s.max_blocks;
    if (one) {
      s.lens[c] = len;
      if (own) {
        list.src[i] = entry(p, len / kPage);
        list.rows[i] = len % kPage;
      } else if (len % kPage) {
        row[len / kPage] = -1;
      }
    }
    for (int e0 = e_first; e0 < len / kPage; e0 += kAtOnce * share.lanes) {
      if (i != share.first || e0 != e_first) {
        fetch(p, len, e0);
        look();
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int e = e0 + j * share.lanes;
        if (e >= len / kPage) continue;
        row[e] = fault[j] ? -1 : page[j];
        if (fault[j]) raise_error(s.err, fault[j]);
        else atomicAdd(s.refs + page[j], 1);
      }
    }
  }
  // Free pages stay free until every entry has been looked at (in front of the counts'
  // barrier, where the rows' first batches are all that there may be)
  if (share.step < n || s.max_blocks > kAtOnce * share.lanes) cluster_barrier();
  scan.each(is_free, total, [&](int page, int number) {
    const int i = first_over(end, n, number);
    s.table[static_cast<int64_t>(to[i]) * s.max_blocks + length[i] / kPage] = page;
    s.refs[page] = 1;
    list.dst[i] = page;
  });
}

// Where the pages in use go: of n in use those from page n on, in their order, to
// the free ones below, in theirs.  head: {n, how many move, a counter}; number[page]: which
// of the list a page from n on is, -1 for one that is not in use.
__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kMaxThreads, 1)
compact_plan_kernel(const int32_t *__restrict__ refs, int num_blocks, int32_t *head, int32_t *n_live,
                    int32_t *src, int32_t *dst, int32_t *number) {
  __shared__ int below;                    // pages in use in front of page n
  cluster_started();
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int rank = static_cast<int>(sm100::cluster_rank()), lane = threadIdx.x & 31;
  Scan scan(refs, num_blocks, rank);
  if (threadIdx.x == 0) below = 0;
  cluster_wait();
  scan.count(is_live, rank);
  const int n = scan.all;
  // the warp that has page n tells all CTAs
  if (n < num_blocks && scan.first <= n && n < scan.end()) {
    int at = scan.before;
    for (int id0 = scan.first; id0 <= n; id0 += 128) {
      int c = 0;
      const int id = id0 + 4 * lane;
      if (id < scan.end()) {
        uint32_t m = scan.four(id, is_live);
        if (id + 4 > n) m &= n > id ? (1u << (n - id)) - 1 : 0;
        c = __popc(m);
      }
      at += __reduce_add_sync(0xffffffffu, c);
    }
    if (lane < kCtas)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(sm100::peer_smem(&below, lane)), "r"(at) : "memory");
  }
  cluster_barrier();
  const int kept = n < num_blocks ? below : n;
  if (rank == 0 && threadIdx.x == 0) {
    head[0] = n;
    head[1] = n - kept;
    head[2] = head[3] = 0;                 // items taken so far
    *n_live = n;
  }
  const int warp_end = scan.end();
  int at = scan.before;
  for (int id0 = scan.first; id0 < warp_end; id0 += 128) {
    const int id = id0 + 4 * lane;
    const uint32_t m = id < warp_end ? scan.four(id, is_live) : 0;
    const int c = __popc(m), incl = warp_incl(c);
    int live = at + incl - c;              // pages in use in front of this one
    at += __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int page = id + k;
      if (page >= warp_end) break;
      const bool in_use = m >> k & 1;
      if (page < n) {
        if (!in_use && page - live < n - kept) dst[page - live] = page;
      } else {
        number[page] = in_use ? live - kept : -1;
        if (in_use) src[live - kept] = page;
      }
      live += in_use;
    }
  }
}

// ------------------------------------------------------------------ copies
constexpr int kCopyThreads = 256;
constexpr int kChunk = 36864;        // of a page at a time: 9 words of 16 bytes a thread
constexpr int kLoads = kChunk / (16 * kCopyThreads);
constexpr int kMostCtas = 8192;
constexpr int kSmall = 1024;         // pages below this, or of no whole 16-byte words, go by 4-byte words, together

struct Pools {
  void *at[kMaxPools];
  uint32_t bytes[kMaxPools];         // of a page
  uint32_t first[kMaxPools];         // chunks of the large pools in front of this one
  uint32_t by_rows[(kMaxPools + 31) / 32];   // a bit each: a page is the rows of its 64 tokens
  int large, n, chunks, same;        // the large ones come first; same: chunks of each, 0 if they differ
  __device__ bool rows_of(int k) const { return by_rows[k >> 5] >> (k & 31) & 1; }
};
static_assert(sizeof(Pools) <= 3900, "kernel arguments");

enum CopyMode { kListed = 0, kForks = 1, kCompaction = 2 };

struct CopyArgs {
  const int32_t *src, *dst, *rows;
  int32_t *head;
  const int32_t *number;
  int n, few;                        // few: chunks below which they are cut
  Seqs s;
};

// Items are a chunk (or a third, or a ninth of one) of a pair of pages in one
// pool.  A CTA takes a run of them: one, up to kMostCtas items (500 pages of 12
// e4m3 layers, 442 MB, in 6000 CTAs 69 us; in 608 that stay, four to an SM, 76: some
// SMs are slower, and the last ones' runs are what is waited for).  Of a compaction
// only the device knows how many there are: 608 CTAs take them from a counter (48
// requests, 280 MB in 4 layers, with two resizes around it: 57.4 us; when this was chosen,
// 58.7, in runs 63.4, in 4096 CTAs 57.2, but then one that moves nothing 9.3 in place of
// 5.2, now 4.9).  A pair's ids are looked at while the first item's loads are on their way.
template <int MODE, int L>
__device__ __forceinline__ void copy_items(const CopyArgs &a, const Pools &p, int pairs) {
  constexpr int kParts = kLoads / L;
  const int per_pair = p.chunks * kParts + (p.n > p.large ? 1 : 0);
  const int64_t items = static_cast<int64_t>(pairs) * per_pair;
  int64_t item = MODE == kCompaction ? blockIdx.x : items * blockIdx.x / gridDim.x;
  const int64_t end_item = MODE == kCompaction ? items : items * (blockIdx.x + 1) / gridDim.x;
  __shared__ int64_t next;
  int64_t ahead = 0;
  int pair = -1, s = -1, d = -1, rows = kPage;
  auto page = [&](int id) { return id >= 0 && id < a.s.num_blocks; };
  auto advance = [&] {
    if constexpr (MODE == kCompaction) {
      if (threadIdx.x == 0) next = ahead;
      __syncthreads();
      item = next;
      __syncthreads();
    } else {
      ++item;
    }
  };
  for (; item < end_item; advance()) {
    if (MODE == kCompaction && threadIdx.x == 0)
      ahead = gridDim.x + static_cast<int64_t>(atomicAdd(reinterpret_cast<unsigned long long *>(a.head + 2), 1ull));
    const int now = static_cast<int>(item / per_pair);
    const int part = static_cast<int>(item - static_cast<int64_t>(now) * per_pair);
    const bool other = now != pair;
    if (other) {
      pair = now;
      s = a.src[pair];
      d = a.dst[pair];
      if constexpr (MODE == kForks) rows = a.rows[pair];
      if (MODE == kListed && threadIdx.x == 0 && (s >= a.s.num_blocks || d >= a.s.num_blocks))
        raise_error(a.s.err, MLA_DEVERR_BLOCK_ID);
      if (!page(s) || !page(d) || s == d) d = -1;
    }
    if (d < 0) continue;
    const bool small = part == p.chunks * kParts;
    uint4 v[L];
    uint8_t *to = nullptr;
    uint32_t bytes = 0;
    if (!small) {
      const int chunk = part / kParts, third = part - chunk * kParts;
      int k;
      if (p.same) {
        k = chunk / p.same;
      } else {
        int lo = 0, hi = p.large - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.first[mid] <= static_cast<uint32_t>(chunk)) lo = mid;
          else hi = mid - 1;
        }
        k = lo;
      }
      const uint32_t size = p.bytes[k], at = (chunk - p.first[k]) * kChunk + third * (L * 16 * kCopyThreads);
      const uint32_t end = MODE == kForks && p.rows_of(k) ? size / kPage * rows : size;
      if (at < end) bytes = end - at;
      const uint8_t *from = static_cast<const uint8_t *>(p.at[k]) + static_cast<int64_t>(s) * size + at;
      to = static_cast<uint8_t *>(p.at[k]) + static_cast<int64_t>(d) * size + at;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const uint32_t w = (i * kCopyThreads + threadIdx.x) * 16;
        if (w < bytes) v[i] = __ldcs(reinterpret_cast<const uint4 *>(from + w));
      }
    }
    if (MODE == kListed && other) {
      // of equal destinations the last one's source stays; a destination that is
      // another pair's source is refused: which of the two came first is not defined
      bool later = false, read = false;
      for (int k = threadIdx.x; k < a.n; k += kCopyThreads) {
        const int sk = __ldg(a.src + k), dk = __ldg(a.dst + k);
        if (!page(sk) || !page(dk) || sk == dk) continue;
        later |= dk == d && k > pair;
        read |= sk == d;
      }
      read = __syncthreads_or(read);
      if (read && threadIdx.x == 0) raise_error(a.s.err, MLA_DEVERR_PAGES);
      if (__syncthreads_or(later) || read) d = -1;
      if (d < 0) continue;
    }
    if (small) {
      // the small pools, 16 threads to a page
      for (int k = p.large + threadIdx.x / 16; k < p.n; k += kCopyThreads / 16) {
        const uint32_t words = p.bytes[k] / 4;
        const uint32_t *f = static_cast<const uint32_t *>(p.at[k]) + static_cast<int64_t>(s) * words;
        uint32_t *t = static_cast<uint32_t *>(p.at[k]) + static_cast<int64_t>(d) * words;
        const uint32_t end = MODE == kForks && p.rows_of(k) ? words / kPage * rows : words;
        for (uint32_t w = threadIdx.x % 16; w < end; w += 16) t[w] = f[w];
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const uint32_t w = (i * kCopyThreads + threadIdx.x) * 16;
      if (w < bytes) __stcs(reinterpret_cast<uint4 *>(to + w), v[i]);
    }
  }
}

template <int MODE>
__global__ void __launch_bounds__(kCopyThreads, 4)
copy_kernel(const __grid_constant__ CopyArgs a, const __grid_constant__ Pools p) {
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  int pairs = a.n;
  if constexpr (MODE == kCompaction) {
    // The rows' entries, a warp or several to a row, four entries a lane (looked at where
    // nothing moves, too: what is wrong with them is flagged whether or not there were free
    // pages in between)
    const int threads = gridDim.x * kCopyThreads, thread = blockIdx.x * kCopyThreads + threadIdx.x;
    const int warps = threads / 32, wid = thread / 32;
    const int per = max(1, min(warps / a.s.B, (a.s.max_blocks + 127) / 128)), step = warps / per;
    const int first = wid < step * per ? wid / per : a.s.B;
    const int len0 = first < a.s.B ? a.s.lens[first] : 0;
    const int live = a.head[0];
    pairs = a.head[1];
    for (int i = thread; i < pairs; i += threads) {
      a.s.refs[a.dst[i]] = a.s.refs[a.src[i]];
      a.s.refs[a.src[i]] = 0;
    }
    for (int b = first; b < a.s.B; b += step) {
      const int len = b == first ? len0 : a.s.lens[b], lane = thread % 32 + 32 * (wid % per);
      if (lane == 0 && (len < 0 || len > a.s.max_blocks * kPage)) raise_error(a.s.err, MLA_DEVERR_SEQ_LEN);
      int32_t *row = a.s.table + static_cast<int64_t>(b) * a.s.max_blocks;
      const int end = pages_of(min(len, a.s.max_blocks * kPage));
#pragma unroll 4
      for (int e = lane; e < end; e += 32 * per) {
        const int page = row[e];
        if (page < 0 || page >= a.s.num_blocks) {
          raise_error(a.s.err, MLA_DEVERR_BLOCK_ID);
        } else if (page >= live) {
          const int k = a.number[page];
          if (k >= 0) row[e] = a.dst[k];
          else raise_error(a.s.err, MLA_DEVERR_PAGES);
        }
      }
    }
  }
  // (as large a piece as leaves every SM some)
  const int64_t chunks = static_cast<int64_t>(pairs) * p.chunks;
  if (chunks >= a.few) copy_items<MODE, kLoads>(a, p, pairs);
  else if (chunks * 3 >= a.few) copy_items<MODE, kLoads / 3>(a, p, pairs);
  else copy_items<MODE, 1>(a, p, pairs);
}

// The first `by_rows` pools are copied by rows where a page is copied in part.
int gather_pools(void *const *pools, const int64_t *page_bytes, int n, Pools &p, int by_rows = 0) {
  if (n < 0 || n > kMaxPools || (n > 0 && (!pools || !page_bytes)) || by_rows < 0 || by_rows > n)
    return MLA_ERR_INVALID_ARG;
  p.n = n;
  p.large = p.chunks = 0;
  p.same = 0;
  for (uint32_t &w : p.by_rows) w = 0;
  for (int pass = 0, at = 0; pass < 2; ++pass) {
    for (int k = 0; k < n; ++k) {
      const int64_t bytes = page_bytes[k];
      if (!pools[k] || bytes < 4 || bytes % 4 || bytes > (1ll << 28) || (reinterpret_cast<uintptr_t>(pools[k]) & 3u))
        return MLA_ERR_INVALID_ARG;
      if (k < by_rows && bytes % (4 * kPage)) return MLA_ERR_INVALID_ARG;
      const bool large = bytes >= kSmall && bytes % (k < by_rows ? 16 * kPage : 16) == 0;
      if (large && !aligned16(pools[k])) return MLA_ERR_INVALID_ARG;
      if (large != (pass == 0)) continue;
      p.at[at] = pools[k];
      p.bytes[at] = static_cast<uint32_t>(bytes);
      p.first[at] = static_cast<uint32_t>(p.chunks);
      if (large) {
        const int c = static_cast<int>((bytes + kChunk - 1) / kChunk);
        p.same = p.large == 0 || p.same == c ? c : 0;
        if (p.large > 0 && static_cast<int>(p.first[at]) != p.large * c) p.same = 0;
        p.chunks += c;
        ++p.large;
      }
      if (k < by_rows) p.by_rows[at >> 5] |= 1u << (at & 31);
      ++at;
    }
  }
  return MLA_OK;
}

// most: pairs that there may be
template <int MODE>
int launch_copy(CopyArgs &a, const Pools &p, int64_t most, mla_stream_t stream) {
  const int sms = device_sm_count();
  if (sms == 0) return MLA_ERR_CUDA;
  a.few = 2 * sms;
  const int64_t chunks = most * p.chunks, cut = chunks >= a.few ? 1 : chunks * 3 >= a.few ? 3 : 9;
  const int64_t items = chunks * cut + (p.n > p.large ? most : 0);
  const int ctas = MODE == kCompaction ? 4 * sms : static_cast<int>(std::clamp<int64_t>(items, 1, kMostCtas));
  return launch_pdl(copy_kernel<MODE>, dim3(ctas), dim3(kCopyThreads), 0, stream, a, p) == cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}

// Shared memory of the bookkeeping kernels beyond the usual 48 KB (some of it is
// static): the most that there may be, so that calls of several threads do not take
// it from each other.
template <typename K>
bool allow_smem(K *kernel, size_t bytes) {
  return bytes <= 40 * 1024 || cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    5 * sizeof(int) * kMaxRows) == cudaSuccess;
}

int check_seqs(const Seqs &s) {
  if (s.num_blocks < 1 || s.num_blocks >= (1 << 25) || s.B < 1 || s.B > kMaxRows || s.max_blocks < 1 ||
      s.max_blocks > (1 << 24) || static_cast<int64_t>(s.B) * s.max_blocks > INT_MAX)   // (sums of pages)
    return MLA_ERR_INVALID_ARG;
  if (!s.refs || !aligned16(s.refs) || !s.table || !s.lens) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

// ------------------------------------------------------------------ accept
constexpr int kMaxTree = 64;

struct AcceptArgs {
  uint8_t *pools[kMaxPools];
  float *scales[kMaxPools];
  int n_pools, chunks;               // 16-byte words of a row
  int num_blocks, max_blocks, q_len, width, sb_shift;
  const int32_t *table, *lens, *tree_lens, *path, *path_lens;
  int32_t *new_lens;
  int *err;
};
static_assert(sizeof(AcceptArgs) <= 4000, "kernel arguments");

constexpr int kAcceptThreads = 256;

// The slots that a request's rows come from and go to.
struct Rows {
  int from[kMaxTree], to[kMaxTree];
  int base, count;
};

__device__ __forceinline__ void find_rows(const AcceptArgs &a, int b, bool tell, Rows &rows) {
  const int i = threadIdx.x, most = a.max_blocks * kPage;
  const int len = a.lens[b], k = a.path_lens[b], n = a.tree_lens ? a.tree_lens[b] : a.q_len;
  const int32_t *path = a.path + static_cast<int64_t>(b) * a.width;
  const bool mine = i < kMaxTree && i < k && i < a.width;
  const int node = mine ? path[i] : 0, before = mine && i > 0 ? path[i - 1] : -1;
  const int base = len - n;
  int bits = 0;
  if (len < 0 || len > most || n < 0 || n > a.q_len) {
    bits = MLA_DEVERR_SEQ_LEN;
  } else if (k < 0 || k > a.width || k > n || (k > 0 && base < 0) || (mine && (node <= before || node >= n))) {
    bits = MLA_DEVERR_RANGE;
  } else if (mine) {
    auto slot = [&](int pos) -> int {
      const int page = __ldg(a.table + static_cast<int64_t>(b) * a.max_blocks + pos / kPage);
      if (page < 0 || page >= a.num_blocks) bits = MLA_DEVERR_BLOCK_ID;
      return page * kPage + pos % kPage;
    };
    rows.from[i] = slot(base + node);
    rows.to[i] = slot(base + i);
  }
  const bool bad = __syncthreads_or(bits);   // the request stays as it is
  if (bits && tell) raise_error(a.err, bits);
  if (i == 0) {
    rows.base = base;
    rows.count = bad ? 0 : k;
    if (tell) a.new_lens[b] = bad || base < 0 ? len : base + k;
  }
  __syncthreads();
}

// 32 requests of 16 tokens, 30 bf16 layers: 4.2 us on the device, one request and
// layer 2.0, most of it the chain lengths, path, table, rows.
//
// Rows keep their bits.  Sources ascend and none is in front of its
// destination, so what a batch of loads leaves unread lies behind all that the
// batch's stores write.
__global__ void __launch_bounds__(kAcceptThreads)
accept_kernel(const __grid_constant__ AcceptArgs a) {
  constexpr int kBatch = 6;
  __shared__ Rows rows;
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  find_rows(a, blockIdx.x, blockIdx.y == 0, rows);
  const int total = rows.count * a.chunks;
  for (int p = blockIdx.y; p < a.n_pools; p += gridDim.y) {
    uint4 *pool = reinterpret_cast<uint4 *>(a.pools[p]);
    for (int c0 = 0; c0 < total; c0 += kBatch * kAcceptThreads) {
      uint4 v[kBatch];
      int64_t to[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int c = c0 + j * kAcceptThreads + threadIdx.x;
        to[j] = -1;
        if (c >= total) continue;
        const int i = c / a.chunks, at = c - i * a.chunks;
        if (rows.to[i] == rows.from[i]) continue;
        v[j] = pool[static_cast<int64_t>(rows.from[i]) * a.chunks + at];
        to[j] = static_cast<int64_t>(rows.to[i]) * a.chunks + at;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (to[j] >= 0) pool[to[j]] = v[j];
    }
  }
}

__device__ __forceinline__ float2 e4m3x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// four codes -> the codes of code * ratio
__device__ __forceinline__ uint32_t recode4(uint32_t v, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float2 f = e4m3x2(v >> (16 * k));
    f.x *= ratio;
    f.y *= ratio;
    o |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << (16 * k);
  }
  return o;
}
__device__ __forceinline__ uint4 recode16(uint4 v, float ratio) {
  return make_uint4(recode4(v.x, ratio), recode4(v.y, ratio), recode4(v.z, ratio), recode4(v.w, ratio));
}
// the largest of four codes' sizes, as a code; NaN counts as 0
__device__ __forceinline__ uint32_t top4(uint32_t v) {
  v &= 0x7F7F7F7Fu;
  const uint32_t nan = ((v + 0x01010101u) & 0x80808080u) >> 7;
  v &= ~(nan * 0xFFu);
  v = __vmaxu4(v, v >> 16);
  return max(v & 0xFFu, (v >> 8) & 0xFFu);
}
// Smallest 2^e, e >= -100, with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -100) + 127) << 23);
}

// Rows of a block-scaled cache go from block to block: they are appended to
// their new ones by the rule of mla_rope_cache_append.  A CTA has a request's
// rows of one layer, at most 9 words of 16 codes a thread, in registers between
// the maximum and the store.  16 requests, 8 layers: 3.5 us.
__global__ void __launch_bounds__(kAcceptThreads)
accept_scaled_kernel(const __grid_constant__ AcceptArgs a) {
  constexpr int kChunks = kDqk / 16, kPer = kMaxTree * kChunks / kAcceptThreads;
  constexpr int kBlocks = (kMaxTree - 1) / 16 + 2;   // that 64 tokens can touch
  __shared__ Rows rows;
  __shared__ uint32_t amax[kBlocks];
  __shared__ float olds[kBlocks], nows[kBlocks];
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  const int b = blockIdx.x, tid = threadIdx.x;
  find_rows(a, b, blockIdx.y == 0, rows);
  const int k = rows.count, base = rows.base, total = k * kChunks;
  if (k == 0) return;
  const int sb = 1 << a.sb_shift, block0 = base >> a.sb_shift;
  for (int p = blockIdx.y; p < a.n_pools; p += gridDim.y) {
    uint4 *pool = reinterpret_cast<uint4 *>(a.pools[p]);
    float *scales = a.scales[p];
    if (tid < kBlocks) amax[tid] = 0;
    __syncthreads();
    uint4 v[kPer];
    float scale[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = j * kAcceptThreads + tid, i = c / kChunks;
      if (c >= total) continue;
      v[j] = pool[static_cast<int64_t>(rows.from[i]) * kChunks + (c - i * kChunks)];
      scale[j] = scales[rows.from[i] >> a.sb_shift];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = j * kAcceptThreads + tid, i = c / kChunks;
      if (c >= total) continue;
      // (what is no scale: NaN)
      if (!(scale[j] >= 0.f && scale[j] <= 0x1p120f)) scale[j] = __uint_as_float(0x7FC00000u);
      const uint32_t top = max(max(top4(v[j].x), top4(v[j].y)), max(top4(v[j].z), top4(v[j].w)));
      const float size = e4m3x2(top).x * scale[j];
      if (size > 0.f) atomicMax(&amax[((base + i) >> a.sb_shift) - block0], __float_as_uint(size));
    }
    __syncthreads();
    const int first = max(0, ((block0 + tid) << a.sb_shift) - base);   // row that block `tid` gets
    if (tid < kBlocks && first < k) {
      const int g = rows.to[first] >> a.sb_shift;
      const float held = scales[g];
      // a block whose first row is written begins afresh
      const bool fresh = (block0 + tid) << a.sb_shift >= base;
      const float old = !fresh && held > 0.f && held <= 0x1p120f ? held : 0.f;
      const float now = fmaxf(old, scale_for(__uint_as_float(amax[tid])));
      olds[tid] = old;
      nows[tid] = now;
      scales[g] = now;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int c = j * kAcceptThreads + tid, i = c / kChunks;
      if (c >= total) continue;
      pool[static_cast<int64_t>(rows.to[i]) * kChunks + (c - i * kChunks)] =
          recode16(v[j], scale[j] / nows[((base + i) >> a.sb_shift) - block0]);
    }
    // rows that stay where they are follow a scale that grew: of the first block,
    // the only one that has some
    if (olds[0] > 0.f && nows[0] > olds[0]) {
      const int64_t g0 = static_cast<int64_t>(rows.to[0] >> a.sb_shift) << a.sb_shift;
      const int skip = base & (sb - 1), rest = sb - min(k, sb - skip);
      for (int c = tid; c < rest * kChunks; c += kAcceptThreads) {
        int row = c / kChunks;
        const int at = c - row * kChunks;
        if (row >= skip) row += sb - rest;
        uint4 *w = pool + (g0 + row) * kChunks + at;
        *w = recode16(*w, olds[0] / nows[0]);
      }
    }
    __syncthreads();
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_cache_copy(void *const *pools, const int64_t *page_bytes, int n_pools, int num_blocks,
                              const int32_t *src, const int32_t *dst, int n, mla_stream_t stream) {
  if (num_blocks < 1 || num_blocks >= (1 << 25) || n < 0 || n > kMaxPairs) return MLA_ERR_INVALID_ARG;
  Pools p;
  const int st = gather_pools(pools, page_bytes, n_pools, p);
  if (st != MLA_OK) return st;
  if (n == 0 || n_pools == 0) return MLA_OK;
  if (!src || !dst) return MLA_ERR_INVALID_ARG;
  CopyArgs a{};
  a.src = src;
  a.dst = dst;
  a.n = n;
  a.s.num_blocks = num_blocks;
  a.s.err = device_error_word();
  if (!a.s.err) return MLA_ERR_CUDA;
  return launch_copy<kListed>(a, p, n, stream);
}

extern "C" int mla_cache_resize(int32_t *refs, int num_blocks, int32_t *block_table, int32_t *seq_lens,
                                const int32_t *new_lens, int B, int max_blocks, mla_stream_t stream) {
  Seqs s{refs, num_blocks, block_table, seq_lens, B, max_blocks, nullptr};
  const int st = check_seqs(s);
  if (st != MLA_OK) return st;
  if (!new_lens) return MLA_ERR_INVALID_ARG;
  s.err = device_error_word();
  if (!s.err) return MLA_ERR_CUDA;
  const size_t smem = 4 * sizeof(int) * B;
  if (!allow_smem(resize_kernel, smem)) return MLA_ERR_CUDA;
  const dim3 threads(threads_for(num_blocks, B));
  return launch_pdl(resize_kernel, dim3(kCtas), threads, smem, stream, s, new_lens) == cudaSuccess ? MLA_OK
                                                                                                  : MLA_ERR_CUDA;
}

extern "C" int mla_cache_fork_workspace_size(int n, size_t *bytes) {
  if (!bytes || n < 0 || n > kMaxRows) return MLA_ERR_INVALID_ARG;
  *bytes = 3 * sizeof(int32_t) * static_cast<size_t>(n);
  return MLA_OK;
}

extern "C" int mla_cache_fork(void *const *pools, const int64_t *page_bytes, int n_pools, int n_by_rows,
                              int32_t *refs, int num_blocks, int32_t *block_table, int32_t *seq_lens, int B,
                              int max_blocks,
                              const int32_t *parents, const int32_t *children, int n, void *workspace,
                              size_t ws_bytes, mla_stream_t stream) {
  Seqs s{refs, num_blocks, block_table, seq_lens, B, max_blocks, nullptr};
  int st = check_seqs(s);
  if (st != MLA_OK) return st;
  if (n < 0 || n > kMaxRows) return MLA_ERR_INVALID_ARG;
  Pools p;
  if ((st = gather_pools(pools, page_bytes, n_pools, p, n_by_rows)) != MLA_OK) return st;
  if (n == 0) return MLA_OK;
  if (!parents || !children || (reinterpret_cast<uintptr_t>(workspace) & 3u)) return MLA_ERR_INVALID_ARG;
  size_t need = 0;
  mla_cache_fork_workspace_size(n, &need);
  if (!workspace || ws_bytes < need) return MLA_ERR_WORKSPACE;
  s.err = device_error_word();
  if (!s.err) return MLA_ERR_CUDA;
  int32_t *ws = static_cast<int32_t *>(workspace);
  const List list{ws, ws + n, ws + 2 * n};
  const size_t smem = sizeof(int) * (static_cast<size_t>(B) + 4 * n);
  if (!allow_smem(fork_kernel, smem)) return MLA_ERR_CUDA;
  const dim3 threads(threads_for(num_blocks, std::max(B, n)));
  if (launch_pdl(fork_kernel, dim3(kCtas), threads, smem, stream, s, parents, children, n, list) != cudaSuccess)
    return MLA_ERR_CUDA;
  if (n_pools == 0) return MLA_OK;
  CopyArgs a{};
  a.src = list.src;
  a.dst = list.dst;
  a.rows = list.rows;
  a.n = n;
  a.s = s;
  return launch_copy<kForks>(a, p, n, stream);
}

extern "C" int mla_cache_compact_workspace_size(int num_blocks, size_t *bytes) {
  if (!bytes || num_blocks < 1 || num_blocks >= (1 << 25)) return MLA_ERR_INVALID_ARG;
  *bytes = sizeof(int32_t) * (4 + 2 * (static_cast<size_t>(num_blocks) / 2 + 1) + num_blocks);
  return MLA_OK;
}

extern "C" int mla_cache_compact(void *const *pools, const int64_t *page_bytes, int n_pools, int32_t *refs,
                                 int num_blocks, int32_t *block_table, const int32_t *seq_lens, int B,
                                 int max_blocks, int32_t *n_live, void *workspace, size_t ws_bytes,
                                 mla_stream_t stream) {
  Seqs s{refs, num_blocks, block_table, const_cast<int32_t *>(seq_lens), B, max_blocks, nullptr};
  int st = check_seqs(s);
  if (st != MLA_OK) return st;
  Pools p;
  if ((st = gather_pools(pools, page_bytes, n_pools, p)) != MLA_OK) return st;
  if (!n_live || (reinterpret_cast<uintptr_t>(workspace) & 7u)) return MLA_ERR_INVALID_ARG;
  size_t need = 0;
  mla_cache_compact_workspace_size(num_blocks, &need);
  if (!workspace || ws_bytes < need) return MLA_ERR_WORKSPACE;
  s.err = device_error_word();
  if (!s.err) return MLA_ERR_CUDA;
  int32_t *head = static_cast<int32_t *>(workspace), *src = head + 4, *dst = src + num_blocks / 2 + 1,
          *number = dst + num_blocks / 2 + 1;
  const dim3 threads(threads_for(num_blocks, 0));
  if (launch_pdl(compact_plan_kernel, dim3(kCtas), threads, 0, stream, static_cast<const int32_t *>(refs), num_blocks,
                 head, n_live, src, dst, number) != cudaSuccess)
    return MLA_ERR_CUDA;
  CopyArgs a{};
  a.src = src;
  a.dst = dst;
  a.head = head;
  a.number = number;
  a.s = s;
  return launch_copy<kCompaction>(a, p, num_blocks / 2, stream);
}

extern "C" int mla_cache_accept(void *const *pools, int kv_dtype, float *const *kv_scales, int scale_block,
                                int n_pools, int num_blocks, const int32_t *block_table,
                                const int32_t *seq_lens, const int32_t *tree_lens, int q_len,
                                const int32_t *path, int path_width, const int32_t *path_lens, int B,
                                int max_blocks, int32_t *new_lens, mla_stream_t stream) {
  if (num_blocks < 1 || num_blocks >= (1 << 25) || B < 1 || max_blocks < 1 || max_blocks > (1 << 24) ||
      q_len < 1 || q_len > kMaxTree || path_width < 1 || path_width > kMaxTree || n_pools < 0 ||
      n_pools > kMaxPools || (kv_dtype != MLA_BF16 && kv_dtype != MLA_E4M3))
    return MLA_ERR_INVALID_ARG;
  if (kv_scales && (kv_dtype != MLA_E4M3 || (scale_block != 16 && scale_block != 32 && scale_block != 64)))
    return MLA_ERR_INVALID_ARG;
  if (!block_table || !seq_lens || !path || !path_lens || !new_lens || (n_pools > 0 && !pools))
    return MLA_ERR_INVALID_ARG;
  // (a request's CTAs all read these, and one of them writes its new length)
  auto meets = [&](const int32_t *p, int64_t n) {
    const auto at = reinterpret_cast<uintptr_t>(p), out = reinterpret_cast<uintptr_t>(new_lens);
    return p && at < out + sizeof(int32_t) * B && out < at + sizeof(int32_t) * n;
  };
  if (meets(seq_lens, B) || meets(tree_lens, B) || meets(path_lens, B) ||
      meets(path, static_cast<int64_t>(B) * path_width) || meets(block_table, static_cast<int64_t>(B) * max_blocks))
    return MLA_ERR_INVALID_ARG;
  AcceptArgs a{};
  for (int k = 0; k < n_pools; ++k) {
    if (!pools[k] || !aligned16(pools[k]) || (kv_scales && !kv_scales[k])) return MLA_ERR_INVALID_ARG;
    a.pools[k] = static_cast<uint8_t *>(pools[k]);
    if (kv_scales) a.scales[k] = kv_scales[k];
  }
  a.n_pools = n_pools;
  a.chunks = kDqk * (kv_dtype == MLA_BF16 ? 2 : 1) / 16;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks;
  a.q_len = q_len;
  a.width = path_width;
  a.sb_shift = scale_block == 64 ? 6 : scale_block == 32 ? 5 : 4;
  a.table = block_table;
  a.lens = seq_lens;
  a.tree_lens = tree_lens;
  a.path = path;
  a.path_lens = path_lens;
  a.new_lens = new_lens;
  a.err = device_error_word();
  const int sms = device_sm_count();
  if (!a.err || sms == 0) return MLA_ERR_CUDA;
  // a CTA goes over several layers of its request where there are many of both
  const int y = std::max(1, std::min(n_pools, (8 * sms + B - 1) / B));
  const cudaError_t e = kv_scales
                            ? launch_pdl(accept_scaled_kernel, dim3(B, y), dim3(kAcceptThreads), 0, stream, a)
                            : launch_pdl(accept_kernel, dim3(B, y), dim3(kAcceptThreads), 0, stream, a);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
