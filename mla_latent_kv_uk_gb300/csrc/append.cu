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
// the slot list; CTAs of other members leave at once, most of them on seeing
// that the token before them has the same block.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include <cmath>

#include "common.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kHeadsPerCta = 128;   // query heads that a CTA rotates: four 16-byte chunks a thread
constexpr int kPairs = kRope / 2;
constexpr int kMinExp = -100;

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

// largest |x| of a pair of bf16 values that is finite
__device__ __forceinline__ float finite_max(float m, uint32_t w) {
  const float a = fabsf(bf_lo(w)), b = fabsf(bf_hi(w));
  if (a < INFINITY) m = fmaxf(m, a);
  if (b < INFINITY) m = fmaxf(m, b);
  return m;
}

// two bf16 values -> two e4m3 codes of value / scale (a caller's scale may be
// no power of two, so this divides)
__device__ __forceinline__ uint32_t codes2(uint32_t w, float scale) {
  return __nv_cvt_float2_to_fp8x2(make_float2(bf_lo(w) / scale, bf_hi(w) / scale), __NV_SATFINITE,
                                  __NV_E4M3);
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

// One warp: token t's k_pe, rotated and stored to k_out; lane i returns its
// pair i as (a, b) in the low and high half of the word.
__device__ __forceinline__ uint32_t rotate_k(const AppendArgs &p, const Turns &turns, int t, int lane) {
  const uint16_t *k = reinterpret_cast<const uint16_t *>(p.k_pe + t * p.k_st);
  uint16_t *o = reinterpret_cast<uint16_t *>(p.k_out + t * p.ko_st);
  uint32_t w;
  if (!p.half_layout) w = reinterpret_cast<const uint32_t *>(k)[lane];
  else w = k[lane] | (static_cast<uint32_t>(k[lane + kPairs]) << 16);
  float s, c;
  turn(p.positions[t], turns.per_pos[lane], s, c);
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

// kRows: rows of a block that one warp keeps (scale_block / 8)
template <int kRows>
__device__ void append_block(const AppendArgs &p, const Turns &turns, int t) {
  constexpr int kBlock = kRows * kWarps;
  __shared__ int row_t[kBlock];       // the token that a row gets, or -1
  __shared__ int first, members;
  __shared__ uint32_t amax_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t slot = p.slots[t];
  if (slot < 0 || slot >= p.num_slots) {   // nothing to store
    if (warp == 0) rotate_k(p, turns, t, lane);
    if (tid == 0 && slot >= p.num_slots) raise_error(p.err, MLA_DEVERR_BLOCK_ID);
    return;
  }
  const int g = static_cast<int>(slot >> p.sb_shift);
  auto same = [&](int s) { return s >= 0 && s < p.num_slots && (s >> p.sb_shift) == g; };
  if (t > 0 && same(p.slots[t - 1])) return;
  if (tid < kBlock) row_t[tid] = -1;
  if (tid == 0) {
    first = t;
    members = 0;
    amax_s = 0;
  }
  __syncthreads();
  for (int u = tid; u < p.T; u += kThreads) {
    const int s = p.slots[u];
    if (same(s)) {
      if (u < t) first = 0;   // any member before t: its CTA, or another's, owns the block
      atomicMax(&row_t[s & (kBlock - 1)], u);
      atomicAdd(&members, 1);
    }
  }
  __syncthreads();
  if (first != t) return;

  // new rows: kept in registers from the maximum to the store
  uint4 c[kRows][2];
  uint32_t kp[kRows];
  int kept = 0;
  float m = 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int u = row_t[warp + r * kWarps];
    if (u < 0) continue;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.kv_c + u * p.c_st);
    c[r][0] = src[lane];
    c[r][1] = src[lane + 32];
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int u = row_t[warp + r * kWarps];
    if (u < 0) continue;
    ++kept;
    kp[r] = rotate_k(p, turns, u, lane);
    m = finite_max(m, kp[r]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m = finite_max(m, c[r][k].x);
      m = finite_max(m, c[r][k].y);
      m = finite_max(m, c[r][k].z);
      m = finite_max(m, c[r][k].w);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) {
    atomicMax(&amax_s, __float_as_uint(m));
    atomicSub(&members, kept);
  }
  __syncthreads();
  float old = row_t[0] >= 0 ? 0.f : p.scales[g];
  if (!(old > 0.f) || !(old < INFINITY)) old = 0.f;
  const float now = fmaxf(old, scale_for(__uint_as_float(amax_s)));
  uint8_t *block = p.cache + static_cast<int64_t>(g) * kBlock * kDqk;
  __syncthreads();   // every thread has the old scale
  if (tid == 0) p.scales[g] = now;
  const bool grew = old > 0.f && now > old;
  const float ratio = old / now;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int row = warp + r * kWarps;
    uint8_t *dst = block + static_cast<int64_t>(row) * kDqk;
    if (row_t[row] >= 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint4 v = c[r][k];
        reinterpret_cast<uint2 *>(dst)[lane + 32 * k] =
            make_uint2(codes2(v.x, now) | (codes2(v.y, now) << 16), codes2(v.z, now) | (codes2(v.w, now) << 16));
      }
      const uint32_t w = codes2(kp[r], now);
      if (!p.half_layout) {
        reinterpret_cast<uint16_t *>(dst + kLatent)[lane] = static_cast<uint16_t>(w);
      } else {
        dst[kLatent + lane] = static_cast<uint8_t>(w);
        dst[kLatent + kPairs + lane] = static_cast<uint8_t>(w >> 8);
      }
    } else if (grew) {
      uint32_t *d = reinterpret_cast<uint32_t *>(dst);
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
      for (; lost; lost &= lost - 1) rotate_k(p, turns, u0 + __ffs(lost) - 1, lane);
    }
  }
}

// Grid (T, 1 + head groups): the first CTA of a token takes its cache row,
// the others rotate 128 heads each.
__global__ void __launch_bounds__(kThreads)
append_kernel(const __grid_constant__ AppendArgs p, const __grid_constant__ Turns turns) {
  const int t = blockIdx.x;
  if (blockIdx.y == 0) {
    if (p.sb_shift == 6) append_block<8>(p, turns, t);
    else if (p.sb_shift == 5) append_block<4>(p, turns, t);
    else append_block<2>(p, turns, t);
    return;
  }
  // every load of the thread goes out before the angles are there
  __shared__ __align__(16) float cs[kPairs], sn[kPairs];
  const int tid = threadIdx.x;
  const int h0 = (blockIdx.y - 1) * kHeadsPerCta, nh = min(kHeadsPerCta, p.H - h0);
  const uint8_t *q = p.q_pe + t * p.q_st + h0 * p.q_sh;
  uint8_t *o = p.q_out + t * p.qo_st + h0 * p.qo_sh;
  if (!p.half_layout) {                // 8 dims: pairs 4ch .. 4ch + 3
    constexpr int kPer = kHeadsPerCta * 8 / kThreads;
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int h = (tid + i * kThreads) >> 3;
      if (h < nh) v[i] = reinterpret_cast<const uint4 *>(q + h * p.q_sh)[tid & 7];
    }
    if (tid < kPairs) turn(p.positions[t], turns.per_pos[tid], sn[tid], cs[tid]);
    __syncthreads();
    const int ch = tid & 7;
    const float4 c = reinterpret_cast<const float4 *>(cs)[ch], sv = reinterpret_cast<const float4 *>(sn)[ch];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int h = (tid + i * kThreads) >> 3;
      if (h < nh)
        reinterpret_cast<uint4 *>(o + h * p.qo_sh)[ch] =
            make_uint4(rot_pair(bf_lo(v[i].x), bf_hi(v[i].x), c.x, sv.x),
                       rot_pair(bf_lo(v[i].y), bf_hi(v[i].y), c.y, sv.y),
                       rot_pair(bf_lo(v[i].z), bf_hi(v[i].z), c.z, sv.z),
                       rot_pair(bf_lo(v[i].w), bf_hi(v[i].w), c.w, sv.w));
    }
  } else {                             // dims 8ch .. and 32 + 8ch ..
    constexpr int kPer = kHeadsPerCta * 4 / kThreads;
    uint4 va[kPer], vb[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int h = (tid + i * kThreads) >> 2;
      if (h < nh) {
        const uint4 *row = reinterpret_cast<const uint4 *>(q + h * p.q_sh);
        va[i] = row[tid & 3];
        vb[i] = row[(tid & 3) + 4];
      }
    }
    if (tid < kPairs) turn(p.positions[t], turns.per_pos[tid], sn[tid], cs[tid]);
    __syncthreads();
    const int ch = tid & 3;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int h = (tid + i * kThreads) >> 2;
      if (h >= nh) continue;
      uint32_t *a = reinterpret_cast<uint32_t *>(&va[i]), *b = reinterpret_cast<uint32_t *>(&vb[i]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 8 * ch + 2 * k;
        const uint32_t r0 = rot_pair(bf_lo(a[k]), bf_lo(b[k]), cs[j], sn[j]);
        const uint32_t r1 = rot_pair(bf_hi(a[k]), bf_hi(b[k]), cs[j + 1], sn[j + 1]);
        a[k] = __byte_perm(r0, r1, 0x5410);
        b[k] = __byte_perm(r0, r1, 0x7632);
      }
      uint4 *dst = reinterpret_cast<uint4 *>(o + h * p.qo_sh);
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
  AppendArgs p{};
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
  const dim3 grid(T, 1 + (q_pe ? (H + kHeadsPerCta - 1) / kHeadsPerCta : 0));
  append_kernel<<<grid, kThreads, 0, stream>>>(p, turns);
  return launch_status();
}
