// Rotary embedding of the new tokens and their append to a block-scaled e4m3
// cache (mla_rope_cache_append).
//
// Angles without 64-bit floating point: the rotation by position * theta_i
// depends on the angle's fraction of a turn only, so the host hands over
// turns-per-position theta_i / 2pi as a 64-bit binary fraction, and the
// position times it, modulo 2^64, is the exact fraction of a turn (off by at
// most position * 2^-53 turns, the host's roundings of theta_i / 2pi).  Its
// upper 32 bits go through sincospi in fp32.  (The fp64 sine and cosine that
// mla_rope_cache_write takes cost more than the call's memory traffic once
// there are thousands of tokens: this GPU runs two fp64 FMAs a clock and SM.)
//
// Blocks of the cache: a block's new scale depends on all its new rows, and
// its old rows may have to follow it, so one CTA owns a block: that of the
// block's first token in the call.  It finds the other members by reading
// the slot list; most tokens are passed over on seeing that the token before
// them has the same block.  (Every block reads all slots: at 2048 tokens one
// round of loads, but the work grows with their square.)
//
// What bounds it: a step (32 tokens, 128 heads: 1 MB) is one chain of loads
// (slots, rows), arithmetic and stores, 4.0 us with the launch.  A chunk moves
// its queries, read and written: 63 MB in 15.3 us, 4.1 TB/s of the 6.8 that a
// copy reaches, the first 3 us of which pass until that rate is there.  Measured on the way there: a CTA for each token, that looks at the
// slots and leaves, 18.5 us; rows read again for their codes instead of kept,
// 15.8; three CTAs to an SM in 40 registers, 16.0 (spilled rows).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <climits>
#include <cmath>

#include "common.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kQueryRows = 256;     // (token, head) rows that a CTA rotates: four 16-byte chunks a thread
constexpr int kMinHeadShift = 4, kMaxHeadShift = 7, kMaxTokens = kQueryRows >> kMinHeadShift;
constexpr int kPairs = kRope / 2;
constexpr int kMinExp = -100;
// CTAs that look for blocks (under two to an SM): one for each token up to
// these, then as many tokens to a CTA as that takes
constexpr int kAppendCtas = 256, kMaxPerCta = 64;
constexpr int kAhead = 4;           // slots that a thread has on their way

// theta_i / 2pi as a fraction of 2^64
struct Turns {
  unsigned long long per_pos[kPairs];
};

struct AppendArgs {
  const uint8_t *q_pe;
  const uint8_t *k_pe;
  const uint8_t *kv_c;
  uint8_t *q_out, *k_out;
  int64_t q_st, q_sh, k_st, c_st;   // bytes
  int64_t qo_st, qo_sh, ko_st;      // bytes
  const int32_t *positions;
  const int32_t *slots;
  int T, H, half_layout;
  uint8_t *cache;
  float *scales;
  int sb_shift;                     // log2(scale_block)
  int64_t num_slots;
  unsigned append_ctas;             // CTAs for the cache rows, per_cta tokens each
  int per_cta;
  int groups, head_shift;           // query items: 2^head_shift heads of a few tokens
  int *err;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// sine and cosine of position * theta
__device__ __forceinline__ void turn(int pos, unsigned long long per_pos, float &s, float &c) {
  const unsigned long long f = static_cast<unsigned long long>(static_cast<long long>(pos)) * per_pos;
  // the signed fraction of a turn in [-1/2, 1/2), times two: sin(pi x)
  const float x = static_cast<float>(static_cast<int>(f >> 32)) * 0x1p-31f;
  sincospif(x, &s, &c);
}

__device__ __forceinline__ uint32_t rot_pair(float a, float b, float c, float s) {
  return sm100::bf16x2_rn(fmaf(a, c, -(b * s)), fmaf(a, s, b * c));
}

// Maxima of |x| over the finite values of both halves of bf16 words, as 16-bit
// integers 0x80 above their bits: that makes infinity and NaN negative.
constexpr uint32_t kMaxStart = 0x00800080u;
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t w) {
  return __vmaxs2(m, (w & 0x7FFF7FFFu) + kMaxStart);
}

// two bf16 values -> two e4m3 codes of value / scale.  inv: 1 / scale where
// that is exact and so is the same; a caller's scale may be no power of two
__device__ __forceinline__ uint32_t codes2(uint32_t w, float scale, float inv) {
  float2 f = make_float2(bf_lo(w), bf_hi(w));
  if (inv != 0.f) {
    f.x *= inv;
    f.y *= inv;
  } else {
    f.x /= scale;
    f.y /= scale;
  }
  return __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
}

// four e4m3 codes -> the codes of value * ratio
__device__ __forceinline__ uint32_t recode4(uint32_t v, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((v >> (16 * k)) & 0xFFFFu), __NV_E4M3);
    float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    f.x *= ratio;
    f.y *= ratio;
    o |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)) << (16 * k);
  }
  return o;
}

// Smallest 2^e, e >= kMinExp, with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, kMinExp);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Token t's k_pe as one warp holds it: lane i has pair i as (a, b) in the low
// and high half of a word.
__device__ __forceinline__ uint32_t load_k(const AppendArgs &p, int t, int lane) {
  const uint16_t *k = reinterpret_cast<const uint16_t *>(p.k_pe + t * p.k_st);
  if (!p.half_layout) return reinterpret_cast<const uint32_t *>(k)[lane];
  return k[lane] | (static_cast<uint32_t>(k[lane + kPairs]) << 16);
}

// Rotates it by the token's position and stores it to k_out; returns the pairs.
__device__ __forceinline__ uint32_t store_k(const AppendArgs &p, unsigned long long per_pos, int t,
                                            int pos, uint32_t w, int lane) {
  uint16_t *o = reinterpret_cast<uint16_t *>(p.k_out + t * p.ko_st);
  float s, c;
  turn(pos, per_pos, s, c);
  w = rot_pair(bf_lo(w), bf_hi(w), c, s);
  __syncwarp();   // in place: every lane has read its pair
  if (!p.half_layout) {
    reinterpret_cast<uint32_t *>(o)[lane] = w;
  } else {
    o[lane] = static_cast<uint16_t>(w);
    o[lane + kPairs] = static_cast<uint16_t>(w >> 16);
  }
  return w;
}

__device__ __forceinline__ void rotate_k(const AppendArgs &p, unsigned long long per_pos, int t,
                                         int lane) {
  store_k(p, per_pos, t, p.positions[t], load_k(p, t, lane), lane);
}

// The slots of tokens u, u + kThreads, ..
__device__ __forceinline__ void load_slots(const AppendArgs &p, int64_t u, int (&s)[kAhead]) {
#pragma unroll
  for (int i = 0; i < kAhead; ++i, u += kThreads) s[i] = u < p.T ? __ldg(p.slots + u) : -1;
}

// The block g of token t, whose token before is in another block.  A warp keeps
// its kRows rows in registers from the maximum to the store: every load of the
// block is on its way at once, and with the queries' traffic beside it a load
// takes microseconds.  ahead: the first kAhead slots of this thread.
template <int kRows>
__device__ __forceinline__ void append_block(const AppendArgs &p, unsigned long long per_pos, int t,
                                             int g, const int (&ahead)[kAhead]) {
  constexpr int kBlock = kRows * kWarps;
  __shared__ int row_t[kBlock];       // the token that a row gets, or -1
  __shared__ int first, members;
  __shared__ uint32_t amax_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto same = [&](int s) { return s >= 0 && s < p.num_slots && (s >> p.sb_shift) == g; };
  if (tid < kBlock) row_t[tid] = -1;
  if (tid == 0) {
    first = t;
    members = 0;
    amax_s = 0;
  }
  const float held = p.scales[g];
  __syncthreads();
  int s[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) s[i] = ahead[i];
  for (int64_t u0 = tid;;) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (!same(s[i])) continue;
      const int u = static_cast<int>(u0) + i * kThreads;
      if (u < t) first = 0;   // any member before t: its CTA, or another's, owns the block
      atomicMax(&row_t[s[i] & (kBlock - 1)], u);
      atomicAdd(&members, 1);
    }
    u0 += kAhead * kThreads;
    if (u0 >= p.T) break;
    load_slots(p, u0, s);
  }
  __syncthreads();
  if (first != t) return;

  uint4 c[kRows][2];
  uint32_t kp[kRows];
  int pos[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int u = row_t[warp + r * kWarps];
    if (u < 0) continue;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.kv_c + u * p.c_st) + lane;
    pos[r] = p.positions[u];
    kp[r] = load_k(p, u, lane);
    c[r][0] = __ldg(src);
    c[r][1] = __ldg(src + 32);
  }
  int kept = 0;
  uint32_t m2 = kMaxStart;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int u = row_t[warp + r * kWarps];
    if (u < 0) continue;
    ++kept;
    kp[r] = store_k(p, per_pos, u, pos[r], kp[r], lane);
    m2 = finite_max(m2, kp[r]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m2 = finite_max(m2, c[r][k].x);
      m2 = finite_max(m2, c[r][k].y);
      m2 = finite_max(m2, c[r][k].z);
      m2 = finite_max(m2, c[r][k].w);
    }
  }
  m2 = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
  if (lane == 0) {
    atomicMax(&amax_s, m2 - (kMaxStart & 0xFFFFu));
    atomicSub(&members, kept);
  }
  __syncthreads();   // and every thread has the old scale
  const float old = row_t[0] < 0 && held > 0.f && held <= 0x1p120f ? held : 0.f;
  const float now = fmaxf(old, scale_for(__uint_as_float(amax_s << 16)));
  uint8_t *block = p.cache + static_cast<int64_t>(g) * kBlock * kDqk;
  if (tid == 0) p.scales[g] = now;
  const bool grew = old > 0.f && now > old;
  const bool exact = (__float_as_uint(now) & 0x7FFFFFu) == 0 && now >= 0x1p-126f && now <= 0x1p126f;
  const float inv = exact ? 1.f / now : 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = warp + r * kWarps;
    uint8_t *dst = block + row * kDqk;
    if (row_t[row] >= 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 v = c[r][k];
        reinterpret_cast<uint2 *>(dst)[lane + 32 * k] =
            make_uint2(codes2(v.x, now, inv) | (codes2(v.y, now, inv) << 16),
                       codes2(v.z, now, inv) | (codes2(v.w, now, inv) << 16));
      }
      const uint32_t w = codes2(kp[r], now, inv);
      if (!p.half_layout) {
        reinterpret_cast<uint16_t *>(dst + kLatent)[lane] = static_cast<uint16_t>(w);
      } else {
        dst[kLatent + lane] = static_cast<uint8_t>(w);
        dst[kLatent + kPairs + lane] = static_cast<uint8_t>(w >> 8);
      }
    }
  }
  if (grew) {
    const float ratio = old / now;
#pragma unroll 1
    for (int row = warp; row < kBlock; row += kWarps) {
      if (row_t[row] >= 0) continue;
      uint32_t *d = reinterpret_cast<uint32_t *>(block + row * kDqk);
#pragma unroll
      for (int k = 0; k < 4; ++k) d[lane + 32 * k] = recode4(d[lane + 32 * k], ratio);
      if (lane < 16) d[lane + 128] = recode4(d[lane + 128], ratio);
    }
  }
  // tokens whose slot a later token took: their k_pe is rotated all the same
  if (members > 0) {
    for (int u0 = warp * 32; u0 < p.T; u0 += kThreads) {
      const int u = u0 + lane;
      const int s = u < p.T ? p.slots[u] : -1;
      uint32_t lost = __ballot_sync(0xffffffffu, same(s) && row_t[s & (kBlock - 1)] != u);
      for (; lost; lost &= lost - 1) rotate_k(p, per_pos, u0 + __ffs(lost) - 1, lane);
    }
  }
}

// The cache rows of p.per_cta tokens: few CTAs look at the slots, so that those
// of the queries start at once.
__device__ __forceinline__ void append_tokens(const AppendArgs &p, const Turns &turns) {
  __shared__ int slots[kMaxPerCta + 1];
  const int t0 = blockIdx.x * p.per_cta, n = min(p.per_cta, p.T - t0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int mine = tid <= n && t0 + tid > 0 ? p.slots[t0 + tid - 1] : -1;
  int ahead[kAhead];
  load_slots(p, tid, ahead);
  const unsigned long long per_pos = turns.per_pos[lane];
  if (tid <= n) slots[tid] = mine;
  __syncthreads();
  auto valid = [&](int s) { return s >= 0 && s < p.num_slots; };
  for (int i = warp; i < n; i += kWarps) {
    const int s = slots[i + 1];
    if (valid(s)) continue;            // nothing to store
    rotate_k(p, per_pos, t0 + i, lane);
    if (lane == 0 && s >= 0) raise_error(p.err, MLA_DEVERR_BLOCK_ID);
  }
  for (int i = 0; i < n; ++i) {
    const int s = slots[i + 1], before = slots[i];
    if (!valid(s)) continue;
    const int g = s >> p.sb_shift;
    if (valid(before) && before >> p.sb_shift == g) continue;
    if (p.sb_shift == 6) append_block<kPage / kWarps>(p, per_pos, t0 + i, g, ahead);
    else if (p.sb_shift == 5) append_block<32 / kWarps>(p, per_pos, t0 + i, g, ahead);
    else append_block<16 / kWarps>(p, per_pos, t0 + i, g, ahead);
    __syncthreads();                   // before the next block's shared words
  }
}

// The first CTAs take the cache rows, the others rotate 256 (token, head) rows.
__global__ void __launch_bounds__(kThreads, 2)
append_kernel(const __grid_constant__ AppendArgs p, const __grid_constant__ Turns turns) {
  sm100::grid_dep_wait();
  sm100::grid_dep_launch();
  if (blockIdx.x < p.append_ctas) {
    append_tokens(p, turns);
    return;
  }
  const int item = blockIdx.x - p.append_ctas;
  const int tokens = kQueryRows >> p.head_shift, span = item / p.groups;
  const int64_t t0 = static_cast<int64_t>(span) * tokens;
  const int h0 = (item - span * p.groups) << p.head_shift;
  const int nt = static_cast<int>(min(static_cast<int64_t>(tokens), p.T - t0));
  const int nh = min(1 << p.head_shift, p.H - h0);
  // every load of the thread goes out before the angles are there
  __shared__ __align__(16) float cs[kMaxTokens][kPairs], sn[kMaxTokens][kPairs];
  const int tid = threadIdx.x;
  const uint8_t *q = p.q_pe + t0 * p.q_st + h0 * p.q_sh;
  uint8_t *o = p.q_out + t0 * p.qo_st + h0 * p.qo_sh;
  auto angles = [&] {
    const int t = tid / kPairs, i = tid % kPairs;
    if (t < nt) turn(p.positions[t0 + t], turns.per_pos[i], sn[t][i], cs[t][i]);
    __syncthreads();
  };
  // row r of the item: token r >> head_shift, head r & (2^head_shift - 1)
  if (!p.half_layout) {                // 8 dims: pairs 4ch .. 4ch + 3
    constexpr int kPer = kQueryRows * 8 / kThreads;
    const int ch = tid & 7;
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (tid + i * kThreads) >> 3, t = r >> p.head_shift, h = r - (t << p.head_shift);
      if (t < nt && h < nh) v[i] = reinterpret_cast<const uint4 *>(q + t * p.q_st + h * p.q_sh)[ch];
    }
    angles();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (tid + i * kThreads) >> 3, t = r >> p.head_shift, h = r - (t << p.head_shift);
      if (t >= nt || h >= nh) continue;
      const float4 c = reinterpret_cast<const float4 *>(cs[t])[ch], sv = reinterpret_cast<const float4 *>(sn[t])[ch];
      reinterpret_cast<uint4 *>(o + t * p.qo_st + h * p.qo_sh)[ch] =
          make_uint4(rot_pair(bf_lo(v[i].x), bf_hi(v[i].x), c.x, sv.x),
                     rot_pair(bf_lo(v[i].y), bf_hi(v[i].y), c.y, sv.y),
                     rot_pair(bf_lo(v[i].z), bf_hi(v[i].z), c.z, sv.z),
                     rot_pair(bf_lo(v[i].w), bf_hi(v[i].w), c.w, sv.w));
    }
  } else {                             // dims 8ch .. and 32 + 8ch ..
    constexpr int kPer = kQueryRows * 4 / kThreads;
    const int ch = tid & 3;
    uint4 va[kPer], vb[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (tid + i * kThreads) >> 2, t = r >> p.head_shift, h = r - (t << p.head_shift);
      if (t < nt && h < nh) {
        const uint4 *row = reinterpret_cast<const uint4 *>(q + t * p.q_st + h * p.q_sh);
        va[i] = row[ch];
        vb[i] = row[ch + 4];
      }
    }
    angles();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int r = (tid + i * kThreads) >> 2, t = r >> p.head_shift, h = r - (t << p.head_shift);
      if (t >= nt || h >= nh) continue;
      uint32_t *a = reinterpret_cast<uint32_t *>(&va[i]), *b = reinterpret_cast<uint32_t *>(&vb[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 c = *reinterpret_cast<const float2 *>(&cs[t][8 * ch + 2 * k]);
        const float2 sv = *reinterpret_cast<const float2 *>(&sn[t][8 * ch + 2 * k]);
        const uint32_t r0 = rot_pair(bf_lo(a[k]), bf_lo(b[k]), c.x, sv.x);
        const uint32_t r1 = rot_pair(bf_hi(a[k]), bf_hi(b[k]), c.y, sv.y);
        a[k] = __byte_perm(r0, r1, 0x5410);
        b[k] = __byte_perm(r0, r1, 0x7632);
      }
      uint4 *dst = reinterpret_cast<uint4 *>(o + t * p.qo_st + h * p.qo_sh);
      dst[ch] = va[i];
      dst[ch + 4] = vb[i];
    }
  }
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" int mla_rope_cache_append(void *q_pe, int64_t q_stride_t, int64_t q_stride_h, void *k_pe,
                                     int64_t k_stride, const void *kv_c, int64_t c_stride,
                                     const int32_t *positions, const int32_t *slot_mapping, int T,
                                     int H, float rope_base, int rope_layout, void *q_out,
                                     void *k_out, void *kv_cache, float *kv_scales, int scale_block,
                                     int num_blocks, mla_stream_t stream) {
  if (T < 0 || (q_pe && (H < 1 || H > 4096)) || num_blocks < 1 || num_blocks >= (1 << 25))
    return MLA_ERR_INVALID_ARG;
  if (rope_layout != MLA_ROPE_INTERLEAVED && rope_layout != MLA_ROPE_HALF)
    return MLA_ERR_INVALID_ARG;
  if (!(rope_base > 1.f) || !(rope_base < INFINITY)) return MLA_ERR_INVALID_ARG;
  if (scale_block != 16 && scale_block != 32 && scale_block != 64) return MLA_ERR_INVALID_ARG;
  if (T == 0) return MLA_OK;
  if (!k_pe || !kv_c || !positions || !slot_mapping || !kv_cache || !kv_scales || (q_out && !q_pe))
    return MLA_ERR_INVALID_ARG;
  if (!aligned16(q_pe) || !aligned16(k_pe) || !aligned16(kv_c) || !aligned16(kv_cache) ||
      !aligned16(q_out) || !aligned16(k_out))
    return MLA_ERR_INVALID_ARG;
  // rows of one tensor start on 16 bytes and do not overlap
  if (k_stride % 8 || c_stride % 8 || (T > 1 && (k_stride < kRope || c_stride < kLatent)))
    return MLA_ERR_INVALID_ARG;
  if (q_pe) {
    const int64_t st = q_stride_t, sh = q_stride_h;
    if (st % 8 || sh % 8 || (T > 1 && st < kRope) || (H > 1 && sh < kRope)) return MLA_ERR_INVALID_ARG;
    if (T > 1 && H > 1 && st < (H - 1) * sh + kRope && sh < (T - 1) * st + kRope)
      return MLA_ERR_INVALID_ARG;
  }
  const int per_cta = min(kMaxPerCta, 1 + (T - 1) / kAppendCtas), append_ctas = 1 + (T - 1) / per_cta;
  int head_shift = kMinHeadShift;
  while (head_shift < kMaxHeadShift && (1 << head_shift) < H) ++head_shift;
  const int tokens = kQueryRows >> head_shift, groups = q_pe ? (H + (1 << head_shift) - 1) >> head_shift : 0;
  const int64_t ctas = append_ctas + static_cast<int64_t>(1 + (T - 1) / tokens) * groups;
  if (ctas > INT_MAX) return MLA_ERR_INVALID_ARG;
  AppendArgs p{};
  p.append_ctas = append_ctas;
  p.per_cta = per_cta;
  p.groups = groups;
  p.head_shift = head_shift;
  p.q_pe = static_cast<const uint8_t *>(q_pe);
  p.k_pe = static_cast<const uint8_t *>(k_pe);
  p.kv_c = static_cast<const uint8_t *>(kv_c);
  p.q_st = 2 * q_stride_t;
  p.q_sh = 2 * q_stride_h;
  p.k_st = 2 * k_stride;
  p.c_st = 2 * c_stride;
  p.q_out = static_cast<uint8_t *>(q_out ? q_out : q_pe);
  p.qo_st = q_out ? static_cast<int64_t>(H) * kRope * 2 : p.q_st;
  p.qo_sh = q_out ? kRope * 2 : p.q_sh;
  p.k_out = static_cast<uint8_t *>(k_out ? k_out : k_pe);
  p.ko_st = k_out ? kRope * 2 : p.k_st;
  p.positions = positions;
  p.slots = slot_mapping;
  p.T = T;
  p.H = H;
  p.half_layout = rope_layout == MLA_ROPE_HALF;
  p.cache = static_cast<uint8_t *>(kv_cache);
  p.scales = kv_scales;
  p.sb_shift = scale_block == 64 ? 6 : scale_block == 32 ? 5 : 4;
  p.num_slots = static_cast<int64_t>(num_blocks) * kPage;
  p.err = device_error_word();
  if (!p.err) return MLA_ERR_CUDA;
  // base^(-i/32) as products of base^(-1/2), base^(-1/4), ... by i's bits: at
  // most five roundings, where 32 calls of exp2 cost a microsecond
  Turns turns;
  double f[kPairs];
  f[0] = 0.15915494309189533577 * 0x1p64;   // 2^64 / 2 pi
  for (int bit = 1; bit < kPairs; bit <<= 1) {
    const double step = std::pow(static_cast<double>(rope_base), -static_cast<double>(bit) / kPairs);
    for (int i = 0; i < bit; ++i) f[bit + i] = f[i] * step;
  }
  for (int i = 0; i < kPairs; ++i) turns.per_pos[i] = static_cast<unsigned long long>(f[i]);
  return launch_pdl(append_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, p, turns) ==
                 cudaSuccess
             ? MLA_OK
             : MLA_ERR_CUDA;
}
