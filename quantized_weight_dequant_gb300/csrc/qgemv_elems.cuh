// Elements of rows in memory and in fp32, eight at a time, and their e4m3 codes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "../../include/qgemv.h"

namespace qg {

// Eight consecutive elements of a row, as they are in memory and in fp32.
template <int T>
struct Raw8 {
  uint4 v[T == QGEMV_OUT_F32 ? 2 : 1];
};
template <int T>
__device__ __forceinline__ Raw8<T> load_raw(const uint8_t* at) {
  Raw8<T> r;
  const uint4* p = reinterpret_cast<const uint4*>(at);
  r.v[0] = p[0];
  if constexpr (T == QGEMV_OUT_F32) r.v[1] = p[1];
  return r;
}
template <int T>
__device__ __forceinline__ void to_float(const Raw8<T>& r, float (&v)[8]) {
  if constexpr (T == QGEMV_OUT_F32) {
    const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (T == QGEMV_OUT_F16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
      } else {
        v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ uint32_t pack2(int type, float a, float b) {
  uint32_t u;
  if (type == QGEMV_OUT_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    u = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    u = *reinterpret_cast<const uint32_t*>(&h);
  }
  return u;
}

__device__ __forceinline__ uint4 pack8(int type, const float (&v)[8]) {
  return make_uint4(pack2(type, v[0], v[1]), pack2(type, v[2], v[3]), pack2(type, v[4], v[5]), pack2(type, v[6], v[7]));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
// The larger magnitude of two, with either sign; NaN where one is.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
  float m;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// The scale of values whose largest magnitude is `top`: top / 448, the largest code; 1 where that is 0 or not finite.
__device__ __forceinline__ float e4m3_scale(float top) {
  float scale = __fdiv_rn(top, 448.f);
  if (!(scale > 0.f && scale < __int_as_float(0x7f800000))) scale = 1.f;
  return fmaxf(scale, 1.17549435e-38f);  // its reciprocal stays finite
}

// e4m3 codes of x / scale, infinities as +-448.
// x / scale rounded once: the product with the reciprocal, then its remainder's share (Markstein, IBM J. Res.
// Dev. 34, 1990).  The product alone sends some quotients halfway between two codes to the other one; a division
// each costs the cache store 3 us of 36.7 (8191 tokens).
__device__ __forceinline__ uint2 e4m3_codes(float (&x)[8], float top, float scale) {
  const float by = __frcp_rn(scale);
  const bool finite = top < __int_as_float(0x7f800000);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float y = x[j] * by;
    x[j] = finite ? fmaf(fmaf(-y, scale, x[j]), by, y) : y;
  }
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float* y = x + 4 * j;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    w[j] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace qg
