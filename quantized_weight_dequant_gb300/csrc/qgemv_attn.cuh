// Attention of one new token per request over a paged key-value cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_ptx.cuh"

namespace qg {

__device__ __forceinline__ float kv_to_float(const void* p, int64_t i, int type) {
  if (type == QGEMV_KV_F16) return __half2float(static_cast<const __half*>(p)[i]);
  if (type == QGEMV_KV_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  const __nv_fp8_e4m3 v = static_cast<const __nv_fp8_e4m3*>(p)[i];
  return static_cast<float>(v);
}

// The definition, one warp per request and query head: lanes over the head's elements, tokens
// one after another with a running maximum m and sum l; the sum and the output are scaled by
// exp(m_old - m_new) when the maximum moves.
template <int D>
__global__ void __launch_bounds__(128) attn_decode_kernel(const qgemv_attn_decode_t p, int* err) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (unit >= static_cast<int64_t>(p.requests) * p.q_heads) return;
  const int r = static_cast<int>(unit / p.q_heads), g = static_cast<int>(unit % p.q_heads);
  const int P = p.cache.page_size, head = g / (p.q_heads / p.cache.kv_heads);
  const int64_t end = static_cast<int64_t>(p.table_width) * P;
  int64_t len = p.lens[r];
  if (len < 0 || len > end) {
    if (lane == 0) atomicOr(err, kDevErrIndex);
    len = len < 0 ? 0 : end;
  }
  float q[E], o[E] = {};
  for (int e = 0; e < E; ++e) q[e] = kv_to_float(p.q, r * p.q_stride + static_cast<int64_t>(g) * D + lane + 32 * e, p.type);
  const float neg = __int_as_float(0xff800000);
  float m = neg, l = 0.f;
  for (int64_t t = p.window ? max(len - p.window, int64_t{0}) : 0; t < len; ++t) {
    const int page = p.table[r * p.table_stride + t / P];
    if (page < 0 || page >= p.cache.pages) {
      if (lane == 0) atomicOr(err, kDevErrIndex);
      continue;
    }
    const int64_t line = static_cast<int64_t>(head) * P + t % P, at = page * p.cache.page_stride + line * D;
    const int64_t sat = page * p.cache.scale_stride + line;
    const bool coded = p.cache.type == QGEMV_KV_E4M3;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * kv_to_float(p.cache.k, at + lane + 32 * e, p.cache.type);
    s = warp_sum(s) * p.scale;
    if (coded) s *= p.cache.k_scale[sat];
    const float mn = fmaxf(m, s), base = mn == neg ? 0.f : mn;
    const float keep = expf(m - base), w = expf(s - base);
    m = mn;
    l = l * keep + w;
    const float wv = coded ? w * p.cache.v_scale[sat] : w;
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * keep + (w != 0.f ? wv * kv_to_float(p.cache.v, at + lane + 32 * e, p.cache.type) : 0.f);
  }
  for (int e = 0; e < E; ++e) {
    const float v = l != 0.f ? o[e] / l : 0.f;
    const int64_t at = r * p.out_stride + static_cast<int64_t>(g) * D + lane + 32 * e;
    if (p.type == QGEMV_OUT_F16)
      static_cast<__half*>(p.out)[at] = __float2half_rn(v);
    else
      static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
  }
  if (p.lse && lane == 0) p.lse[static_cast<int64_t>(r) * p.q_heads + g] = l != 0.f ? m + logf(l) : neg;
}

}  // namespace qg
