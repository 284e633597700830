// Low-rank adapters of many requests beside a shared projection.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_epilogue.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kLoraMaxRank = 128;

__device__ __forceinline__ float lora_elem(const void* p, int64_t i, int type) {
  return type == QGEMV_OUT_F16 ? __half2float(static_cast<const __half*>(p)[i])
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float lora_base(const void* p, int64_t i, int out) {
  return out == QGEMV_OUT_F32 ? static_cast<const float*>(p)[i] : lora_elem(p, i, out);
}

// The definition, one CTA per row: its warps form the inner sums, its threads the outputs.
__global__ void __launch_bounds__(256) lora_kernel(const qgemv_lora_t p, int* err) {
  __shared__ float low[kLoraMaxRank];
  const int64_t m = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int a = p.ids[m];
  if (a < -1 || a >= p.adapters) {
    if (threadIdx.x == 0) atomicOr(err, kDevErrIndex);
    a = -1;
  }
  const int r = a < 0 ? 0 : p.ranks ? min(max(p.ranks[a], 0), p.rank) : p.rank;
  const float scale = a >= 0 && p.scales ? p.scales[a] : 1.f;
  for (int j = warp; j < r; j += 8) {
    float s = 0.f;
    for (int64_t k = lane; k < p.K; k += 32)
      s += lora_elem(p.A, (static_cast<int64_t>(a) * p.rank + j) * p.K + k, p.type) * lora_elem(p.x, m * p.x_stride + k, p.type);
    s = warp_sum(s);
    if (lane == 0) low[j] = s;
  }
  __syncthreads();
  for (int64_t n = threadIdx.x; n < p.N; n += 256) {
    float s = 0.f;
    for (int j = 0; j < r; ++j) s += lora_elem(p.B, (static_cast<int64_t>(a) * p.N + n) * p.rank + j, p.type) * low[j];
    const float b = p.base ? lora_base(p.base, m * p.y_stride + n, p.out) : 0.f;
    const float y = r ? b + scale * s : b;
    if (p.out == QGEMV_OUT_F32)
      static_cast<float*>(p.y)[m * p.y_stride + n] = y;
    else if (p.out == QGEMV_OUT_F16)
      static_cast<__half*>(p.y)[m * p.y_stride + n] = __float2half_rn(y);
    else
      static_cast<__nv_bfloat16*>(p.y)[m * p.y_stride + n] = __float2bfloat16_rn(y);
  }
}

}  // namespace qg
