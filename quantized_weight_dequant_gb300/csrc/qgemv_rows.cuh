// Row operators of a layer with projections in 8 bits: the root-mean-square norm with the residual's
// addition, and the quantisation of rows (or of the MLP's gated product) to e4m3 with a scale per 128.
#pragma once
#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_elems.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

// Eight elements of a row at a time: a group of 128, which shares a scale, is 16 neighbouring lanes.
constexpr int kGroupLanes = 16;

// Eight elements whose type is known when the kernel runs: WIDE fp32, else fp16 or bf16 by `type`.
template <bool WIDE>
struct Elems8 {
  uint4 v[WIDE ? 2 : 1];
};
template <bool WIDE>
__device__ __forceinline__ Elems8<WIDE> load_elems(const void* row, int64_t at) {
  Elems8<WIDE> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + at * (WIDE ? 4 : 2));
  r.v[0] = p[0];
  if constexpr (WIDE) r.v[1] = p[1];
  return r;
}
template <bool WIDE>
__device__ __forceinline__ void elems_float(const Elems8<WIDE>& r, int type, float (&f)[8]) {
  if constexpr (WIDE) {
    to_float<QGEMV_OUT_F32>(Raw8<QGEMV_OUT_F32>{{r.v[0], r.v[1]}}, f);
  } else if (type == QGEMV_OUT_F16) {
    to_float<QGEMV_OUT_F16>(Raw8<QGEMV_OUT_F16>{{r.v[0]}}, f);
  } else {
    to_float<QGEMV_OUT_BF16>(Raw8<QGEMV_OUT_BF16>{{r.v[0]}}, f);
  }
}
__device__ __forceinline__ void store_elems(void* row, int64_t at, int type, const float (&f)[8]) {
  if (type == QGEMV_OUT_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + at);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(row) + at * 2) = pack8(type, f);
  }
}

// Codes of this lane's P times eight elements, which are neighbours, and their group's scale from its first lane.  All 32 lanes come
// here together; `in`: the row has them.
template <int P>
__device__ __forceinline__ void store_codes(float (*f)[8], bool in, int first, uint8_t* codes, float* scale) {
  constexpr int L = kGroupLanes / P;  // lanes of a group
  float top = 0.f;                    // NaN where one of them is
#pragma unroll
  for (int j = 0; j < 8 * P; ++j) top = max_abs_nan(top, f[j / 8][j % 8]);
  top = in ? fabsf(top) : 0.f;
#pragma unroll
  for (int k = L / 2; k > 0; k >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, k));
  const float s = e4m3_scale(top);
  if (!in) return;
  const uint2 c = e4m3_codes(f[0], top, s);
  if constexpr (P == 1) {
    *reinterpret_cast<uint2*>(codes + first) = c;
  } else {
    const uint2 d = e4m3_codes(f[1], top, s);
    *reinterpret_cast<uint4*>(codes + first) = make_uint4(c.x, c.y, d.x, d.y);
  }
  if (first % (8 * kGroupLanes) == 0) scale[first / (8 * kGroupLanes)] = s;
}

// y = s / sqrt(mean(s^2) + eps) * (offset + weight), s = x + res.  A row is held in registers, V times eight elements a
// thread, by one warp (kNormWarps rows in a CTA) or by a whole CTA, so that every byte is read once and the norm of a row
// may overwrite it.  Memory bounds it: 8191 rows of 4096 in bf16 with the sum written back and codes, 235 MB, take 40.0 us
// (5.9 TB/s); 8191 of 2048 22.3; 64 of 4096 2.9 and one row 2.7, which is the launch and one trip to memory.  (Rows of more than 16384
// columns are partly kept in local memory: 1024 threads have 64 registers each.)
constexpr int kNormWarps = 4;  // rows of a CTA where a warp has a row

template <bool WIDE, int RES, int V, bool WARP>  // RES: 0 none, 1 of 16 bits, 2 fp32
__global__ void __launch_bounds__(WARP ? 32 * kNormWarps : 1024) norm_kernel(const __grid_constant__ qgemv_norm_t p) {
  __shared__ float part[2][32];
  const int threads = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * kNormWarps : gridDim.x;
  int64_t m = WARP ? static_cast<int64_t>(blockIdx.x) * kNormWarps + threadIdx.x / 32 : blockIdx.x;
  constexpr int kEl = WIDE ? 4 : 2, kResEl = RES == 2 ? 4 : 2;
  // pieces of eight side by side, whose group's scale is worked out once (8191 x 4096 42.1 us for 44.8; of fp32 rows with an fp32
  // residual, 64 bytes apart then, 91 for 83)
  constexpr int P = V == 1 || WIDE || RES == 2 ? 1 : 2;
  auto place = [&](int j) { return ((j / P * threads + tid) * P + j % P) * 8; };
  Elems8<WIDE> a[V];
  Elems8<RES == 2> b[RES ? V : 1];
  auto read = [&] {
    const uint8_t* x = static_cast<const uint8_t*>(p.x) + m * p.x_stride * kEl;
    const uint8_t* res = static_cast<const uint8_t*>(p.res) + m * p.res_stride * kResEl;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = place(j);
      if (at < p.N) {
        a[j] = load_elems<WIDE>(x, at);
        if constexpr (RES != 0) b[j] = load_elems<RES == 2>(res, at);
      }
    }
  };
  pdl_launch_dependents();
  pdl_wait();
  if (m >= p.rows) return;
  read();
  int turn = 0;
  do {
    float s[V][8];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = place(j);
      if (at < p.N) {
        elems_float<WIDE>(a[j], p.in, s[j]);
        if constexpr (RES != 0) {
          float r[8];
          elems_float<RES == 2>(b[j], p.res_type, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[j][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(s[j][i], s[j][i], sum);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] = 0.f;
      }
    }
    const int64_t row = m;
    m += step;
    if (m < p.rows) read();  // the next row is on its way while this one is finished
    sum = warp_sum(sum);
    if constexpr (!WARP) {
      if (tid % 32 == 0) part[turn][tid / 32] = sum;
      __syncthreads();  // and every element of the row has been read
      sum = warp_sum((tid & 31) < threads / 32 ? part[turn][tid & 31] : 0.f);
      turn ^= 1;
    }
    const float by = 1.f / sqrtf(sum / static_cast<float>(p.N) + p.eps);
    void* res_out = p.res_out ? static_cast<uint8_t*>(p.res_out) + row * p.res_out_stride * (p.res_type == QGEMV_OUT_F32 ? 4 : 2) : nullptr;
    void* y = p.y ? static_cast<uint8_t*>(p.y) + row * p.y_stride * (p.out == QGEMV_OUT_F32 ? 4 : 2) : nullptr;
    uint8_t* codes = p.codes ? static_cast<uint8_t*>(p.codes) + row * p.codes_stride : nullptr;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int at = place(j);
      const bool in = at < p.N;
      if (in && res_out) store_elems(res_out, at, p.res_type, s[j]);
      if (p.weight) {
        float w[8] = {};
        if (in) {
          if (p.weight_type == QGEMV_OUT_F32)
            elems_float<true>(load_elems<true>(p.weight, at), p.weight_type, w);
          else
            elems_float<false>(load_elems<false>(p.weight, at), p.weight_type, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] = s[j][i] * by * (p.offset + w[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) s[j][i] = s[j][i] * by;
      }
      if (in && y) store_elems(y, at, p.out, s[j]);
      // (codes come in whole sixteens: both pieces are in the row or neither)
      if (codes && j % P == P - 1) store_codes<P>(&s[j + 1 - P], in, place(j + 1 - P), codes, p.scale + row * p.scale_stride);
    }
  } while (m < p.rows);
}

// g / (1 + e^-g) to 2^-20: e^-g as 2^t with the rest of the product t = -g log2 e put back by its first-order term.  The bounds of
// -g keep t and e^-g finite; below g = -87.4 the quotient's divisor passes 2^126 and the result is 0 (of -inf NaN).
__device__ __forceinline__ float silu(float g) {
  constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596303e-8f, kLn2 = 0.693147182f;
  const float x = fminf(fmaxf(-g, -120.f), 88.f), t = x * kLog2e;
  const float rest = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -t));
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  return __fdividef(g, 1.f + fmaf(e, rest * kLn2, e));
}

// Codes of rows: a scale top / 448 and quotients per 128.  A thread has 16 elements, an eighth of a group, so that the group's scale is worked out for 16 at a
// time, and a CTA 2048 of its row.  Instructions bound it next to memory: 8191 rows of 4096 in bf16 take 18.9 us (15.0 at
// the copy's rate; with eight elements a thread 22.3; with CTAs of 64 threads 33.6, of 256 17.9), the gated
// product of 14336 117 (86; with expf and a division 144; with 64 threads 119, with 256 121), 64 rows of it 2.9, one of 4096 1.6.
constexpr int kQuantThreads = 128;

template <bool WIDE, bool GATED>
__global__ void __launch_bounds__(kQuantThreads) quant_kernel(const __grid_constant__ qgemv_quant_t p, int chunks) {
  const int64_t m = blockIdx.x;
  const uint8_t* x = static_cast<const uint8_t*>(p.x) + m * p.x_stride * (WIDE ? 4 : 2);
  const uint8_t* up = static_cast<const uint8_t*>(p.up) + m * p.up_stride * (WIDE ? 4 : 2);
  uint8_t* codes = static_cast<uint8_t*>(p.codes) + m * p.codes_stride;
  float* scale = p.scale + m * p.scale_stride;
  pdl_launch_dependents();
  pdl_wait();
  for (int c = blockIdx.y; c < chunks; c += gridDim.y) {
    const int at = (c * kQuantThreads + threadIdx.x) * 16;
    const bool in = at < p.N;
    float f[2][8] = {};
    if (in) {
      const Elems8<WIDE> a[2] = {load_elems<WIDE>(x, at), load_elems<WIDE>(x, at + 8)};
      Elems8<WIDE> b[2];
      if constexpr (GATED) b[0] = load_elems<WIDE>(up, at), b[1] = load_elems<WIDE>(up, at + 8);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        elems_float<WIDE>(a[j], p.in, f[j]);
        if constexpr (GATED) {
          float u[8];
          elems_float<WIDE>(b[j], p.in, u);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[j][i] = silu(f[j][i]) * u[i];
        }
      }
    }
    store_codes<2>(f, in, at, codes, scale);
  }
}

}  // namespace qg
