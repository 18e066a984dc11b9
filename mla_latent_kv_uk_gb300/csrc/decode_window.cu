// Paged latent decode with a sliding window and sinks, over a bf16, an e4m3
// or a block-scaled e4m3 cache (mla_decode_paged_window, _scaled).
//
// One warp per (request, query token, head): 18 of the 576 dims per lane,
// one visible key after the other with an online softmax.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;

struct WindowArgs {
  const uint8_t *q, *kv;
  const float *scales;          // nullptr: k_scale
  int sb_shift;
  float k_scale, scale_log2;    // sm_scale * log2(e) * q_scale
  const int32_t *block_table, *seq_lens;
  int B, q_len, H, max_blocks, num_blocks, window, sinks;
  void *out;
  int out_f32;
  float *lse;
  int *err;
};

template <bool FP8>
__device__ __forceinline__ float load1(const uint8_t *p, int i) {
  if constexpr (FP8) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half *>(&h));
  } else {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kWarps * 32) window_kernel(WindowArgs a) {
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y * kWarps + (threadIdx.x >> 5);
  if (h >= a.H) return;
  const int b = blockIdx.x / a.q_len, i = blockIdx.x % a.q_len;
  int len = a.seq_lens[b];
  if (len < 0 || len > a.max_blocks * kPage) {
    raise_error(a.err, MLA_DEVERR_SEQ_LEN);
    len = min(max(len, 0), a.max_blocks * kPage);
  }
  constexpr int kRow = kDqk * (FP8 ? 1 : 2);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * a.H + h;
  float q[18], o[16];
#pragma unroll
  for (int k = 0; k < 18; ++k) q[k] = load1<FP8>(a.q + row * kRow, lane + 32 * k);
#pragma unroll
  for (int k = 0; k < 16; ++k) o[k] = 0.f;
  const int p = len - a.q_len + i;
  const int lo = a.window ? max(0, p - a.window + 1) : 0;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j <= p; ++j) {
    if (j >= a.sinks && j < lo) {
      j = lo - 1;
      continue;
    }
    const int blk = a.block_table[static_cast<int64_t>(b) * a.max_blocks + j / kPage];
    float kv[18], sc = a.k_scale;
    if (blk < 0 || blk >= a.num_blocks) {
      raise_error(a.err, MLA_DEVERR_BLOCK_ID);
#pragma unroll
      for (int k = 0; k < 18; ++k) kv[k] = 0.f;
    } else {
      const int64_t slot = static_cast<int64_t>(blk) * kPage + j % kPage;
      if (a.scales) sc = a.scales[slot >> a.sb_shift];
#pragma unroll
      for (int k = 0; k < 18; ++k) kv[k] = load1<FP8>(a.kv + slot * kRow, lane + 32 * k) * sc;
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 18; ++k) s = fmaf(q[k], kv[k], s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2;
    if (s > m) {
      const float f = exp2f(m - s);
      l *= f;
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] *= f;
      m = s;
    }
    const float w = exp2f(s - m);
    l += w;
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = fmaf(w, kv[k], o[k]);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int64_t at = row * kLatent + lane + 32 * k;
    if (a.out_f32) static_cast<float *>(a.out)[at] = o[k] * inv;
    else static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(o[k] * inv);
  }
  if (lane == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

bool shape_ok(int B, int q_len, int H) {
  if (B < 1 || q_len < 1 || q_len > 64 || H < 1 || H > 4096) return false;
  return static_cast<int64_t>(B) * q_len * ((H + 127) / 128) <= (1 << 22);
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
  if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(out)) return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

size_t ws_bytes_for(int, int, int, int, int) { return 256; }

int launch_window(const void *q, bool fp8, float q_scale, const void *kv_cache, float k_scale,
                  const float *scales, int sb_shift, const int32_t *block_table,
                  const int32_t *seq_lens, int B, int q_len, int H, int max_blocks, int num_blocks,
                  float sm_scale, int window, int sinks, int split_tiles, void *out, int out_dtype,
                  float *lse, void *workspace, size_t ws_bytes, mla_stream_t stream) {
  if (!aligned16(workspace)) return MLA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < ws_bytes_for(B, q_len, H, max_blocks * kPage, split_tiles))
    return MLA_ERR_WORKSPACE;
  WindowArgs a{};
  a.err = device_error_word();
  if (!a.err) return MLA_ERR_CUDA;
  a.q = static_cast<const uint8_t *>(q);
  a.kv = static_cast<const uint8_t *>(kv_cache);
  a.scales = scales;
  a.sb_shift = sb_shift;
  a.k_scale = fp8 ? k_scale : 1.f;
  a.scale_log2 = sm_scale * 1.4426950408889634f * (fp8 ? q_scale : 1.f);
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.B = B;
  a.q_len = q_len;
  a.H = H;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.window = window < (1 << 30) ? window : 1 << 30;
  a.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
  a.out = out;
  a.out_f32 = out_dtype == MLA_F32;
  a.lse = lse;
  const dim3 grid(B * q_len, (H + kWarps - 1) / kWarps);
  if (fp8) window_kernel<true><<<grid, kWarps * 32, 0, stream>>>(a);
  else window_kernel<false><<<grid, kWarps * 32, 0, stream>>>(a);
  return launch_status();
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
  *bytes = ws_bytes_for(B, q_len, H, max_seq_len, split_tiles);
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
