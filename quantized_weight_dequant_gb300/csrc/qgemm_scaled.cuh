// Projection of e4m3 rows by e4m3 weights, each with a scale for blocks of 128:
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] W[n, k].
#pragma once
#include <cuda_fp8.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_elems.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kFp8Block = 128;

__device__ __forceinline__ void e4m3x4(uint32_t c, float (&f)[4]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> (16 * j) & 0xffff), __NV_E4M3);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * j] = v.x, f[2 * j + 1] = v.y;
  }
}

__device__ __forceinline__ void fp8_store(void* y, int64_t at, int type, float v) {
  if (type == QGEMV_OUT_F32)
    static_cast<float*>(y)[at] = v;
  else if (type == QGEMV_OUT_F16)
    static_cast<__half*>(y)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
}

// A warp per weight row and eight rows of x.
constexpr int kFp8SimpleRows = 8;
__global__ void __launch_bounds__(256) fp8_simple_kernel(const __grid_constant__ qgemv_scaled_t p, unsigned row_sets) {
  const int lane = threadIdx.x & 31;
  const int64_t n = static_cast<int64_t>(blockIdx.x / row_sets) * 8 + threadIdx.x / 32;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x % row_sets) * kFp8SimpleRows;
  pdl_launch_dependents();
  pdl_wait();
  if (n >= p.N) return;
  const int64_t blocks = (p.K + kFp8Block - 1) / kFp8Block;
  float sum[kFp8SimpleRows] = {};
  for (int64_t b = 0; b < blocks; ++b) {
    const int64_t k = b * kFp8Block + lane * 4;
    float w[4] = {};
    if (k < p.K) e4m3x4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.W) + n * p.K + k), w);
    const float ws = p.w_scale[n / kFp8Block * blocks + b];
#pragma unroll
    for (int r = 0; r < kFp8SimpleRows; ++r) {
      const int64_t m = m0 + r;
      if (m >= p.M) break;
      float x[4] = {};
      if (k < p.K) e4m3x4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.x) + m * p.x_stride + k), x);
      float d = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) d = fmaf(x[j], w[j], d);
      sum[r] = fmaf(warp_sum(d), p.x_scale[m * p.x_scale_stride + b] * ws, sum[r]);
    }
  }
  for (int r = 0; r < kFp8SimpleRows && m0 + r < p.M; ++r)
    if (lane == r) fp8_store(p.y, (m0 + r) * p.y_stride + n, p.out, sum[r]);
}

}  // namespace qg
