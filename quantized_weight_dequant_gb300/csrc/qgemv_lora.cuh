// Low-rank adapters of many requests beside a shared projection:
//   t = A_a x_m  (rank r_a),   y_m = base_m + s_a B_a t
//
// With a few rows per adapter the kernel is bound by the bytes of A and B, with many rows by those of
// base and y; a row's own work is 2 r (K + N) operations.  One launch does both products:
//  * A cluster of eight CTAs takes the rows of one adapter among 32 neighbouring rows of the batch.
//    Each CTA forms the inner sums over its eighth of K; the eight partial sums meet through
//    distributed shared memory (each CTA adds all of them in rank order), and each CTA writes its
//    eighth of N.  So the inner sums never leave the chip, and a single row still uses eight SMs.
//  * While the first product runs, the cluster's rows of B are brought into L2 by bulk prefetches.
//  * Both products run on mma.sync m16n8k16 with the adapter's rows as its 16 and the tokens as its 8.
//    A lane's operands are 16 consecutive bytes of its row: the order of k within a 32-wide block is the
//    same permutation on both sides, so no shared memory or ldmatrix is needed for A, B or x.
//  * The inner sums (fp32) enter the second product as two fp16 parts scaled by a power of two per row
//    (the row's largest in [2^14, 2^15)), or three bf16 parts: at least 21 bits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_mma.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraRows = 32;      // rows of the batch per cluster: one warp finds the rows of an adapter
constexpr int kLoraCluster = 8;
constexpr int kLoraLd = kLoraMaxRank + 4;  // floats per token of the sums in shared memory

struct LoraSmem {
  float part[kLoraWarps][kLoraRows][36];     // first product: per warp, 32 ranks at a time
  float own[kLoraRows][kLoraLd];             // this CTA's sums over its part of K
  float sum[kLoraRows][kLoraLd];             // over all of K
  uint4 frag[kLoraRows / 8][kLoraMaxRank / 32][3][32];  // 16-bit parts of the sums, as the B operand of a lane
  float factor[kLoraRows];                   // of a token: the adapter's scale over the parts' power of two
  int row[kLoraRows];                        // rows of the adapter in hand
};

__device__ __forceinline__ float4 cluster_ld4(uint32_t a, uint32_t rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(r) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 ld_stream(const void* p) {  // read once
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ float lora_load(const void* p, int64_t i, int type) {
  if (type == QGEMV_OUT_F32) return static_cast<const float*>(p)[i];
  if (type == QGEMV_OUT_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void lora_store(void* p, int64_t i, int type, float v) {
  if (type == QGEMV_OUT_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == QGEMV_OUT_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// First product over the 32-wide blocks b0 .. b1 of K for ranks j0 .. j0 + 16 RT - 1 and 8 TG tokens, the
// blocks dealt to the warps in turn; the warps' sums go to sm.part.  Lane (g, c) = (lane / 4, lane % 4).
template <bool BF, int RT, int TG>
__device__ __forceinline__ void lora_shrink(const qgemv_lora_t& p, LoraSmem& sm, const uint16_t* A, int r, int j0, int n_tok, int64_t b0, int64_t b1) {
  constexpr int U = TG == 1 ? 2 : 1;  // blocks in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  float acc[RT][TG][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int t = 0; t < TG; ++t) acc[i][t][0] = acc[i][t][1] = acc[i][t][2] = acc[i][t][3] = 0.f;
  const uint16_t* xr[TG];
#pragma unroll
  for (int t = 0; t < TG; ++t)
    xr[t] = 8 * t + g < n_tok ? static_cast<const uint16_t*>(p.x) + sm.row[8 * t + g] * p.x_stride + 8 * c : nullptr;
  const uint16_t* a0 = A + static_cast<int64_t>(j0 + g) * p.K + 8 * c;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int64_t b = b0 + warp; b < b1; b += kLoraWarps * U) {
    uint4 a[U][RT][2], x[U][TG];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = 32 * (b + kLoraWarps * u);
      const bool in = b + kLoraWarps * u < b1 && k + 8 * c < p.K;
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          a[u][i][h] = in && j0 + 16 * i + 8 * h + g < r ? *reinterpret_cast<const uint4*>(a0 + static_cast<int64_t>(16 * i + 8 * h) * p.K + k) : zero;
#pragma unroll
      for (int t = 0; t < TG; ++t) x[u][t] = in && xr[t] ? *reinterpret_cast<const uint4*>(xr[t] + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int t = 0; t < TG; ++t) {
          mma16816<BF>(acc[i][t], a[u][i][0].x, a[u][i][1].x, a[u][i][0].y, a[u][i][1].y, x[u][t].x, x[u][t].y);
          mma16816<BF>(acc[i][t], a[u][i][0].z, a[u][i][1].z, a[u][i][0].w, a[u][i][1].w, x[u][t].z, x[u][t].w);
        }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int t = 0; t < TG; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) sm.part[warp][8 * t + 2 * c + (e & 1)][16 * i + g + 8 * (e >> 1)] = acc[i][t][e];
  __syncthreads();
  for (int e = threadIdx.x; e < 8 * TG * 16 * RT; e += kLoraThreads) {
    const int tok = e / (16 * RT), j = e % (16 * RT);
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kLoraWarps; ++w) s += sm.part[w][tok][j];
    sm.own[tok][j0 + j] = s;
  }
  __syncthreads();
}

// The sums of 8 TG tokens as operands of the second product: lane (g, c) of block b takes ranks
// 32 b + 8 c .. + 7 of token 8 t + g.
template <bool BF>
__device__ __forceinline__ void lora_parts(LoraSmem& sm, int t, int blocks, float scale) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const float* s = &sm.sum[8 * t + g][8 * c];
  float by = 1.f, back = 1.f;
  if constexpr (!BF) {
    float top = 0.f;
    for (int b = 0; b < blocks; ++b)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(s[32 * b + e]));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int ex = __float_as_int(top) >> 23 & 0xff;
    if (ex >= 15 && ex < 255) {  // 2^(141 - ex) takes 1.x 2^(ex - 127) to 1.x 2^14
      by = __int_as_float((127 + 141 - ex) << 23);
      back = __int_as_float((127 - 141 + ex) << 23);
    }
  }
  for (int b = 0; b < blocks; ++b) {
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float u = s[32 * b + 2 * e] * by, v = s[32 * b + 2 * e + 1] * by;
      hi[e] = pair16<BF>(u, v);
      float2 f = unpair16<BF>(hi[e]);
      u -= f.x, v -= f.y;
      mid[e] = pair16<BF>(u, v);
      f = unpair16<BF>(mid[e]);
      lo[e] = pair16<BF>(u - f.x, v - f.y);
    }
    sm.frag[t][b][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    sm.frag[t][b][1][lane] = make_uint4(mid[0], mid[1], mid[2], mid[3]);
    if (BF) sm.frag[t][b][2][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  if (c == 0) sm.factor[8 * t + g] = scale * back;
}

// Second product: outputs of the 16-row tiles t0 .. t1 of N, dealt to the warps in turn, for 8 TG tokens.
template <bool BF, int TG, int OUT>
__device__ __forceinline__ void lora_expand(const qgemv_lora_t& p, const LoraSmem& sm, const uint16_t* B, int r, int n_tok, int64_t t0, int64_t t1) {
  constexpr int U = TG == 1 ? 4 : 2;  // tiles in flight
  constexpr int kParts = BF ? 3 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int blocks = (r + 31) / 32;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  int64_t at[TG][2];
  float factor[TG][2];
#pragma unroll
  for (int t = 0; t < TG; ++t)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int tok = 8 * t + 2 * c + e;
      at[t][e] = tok < n_tok ? sm.row[tok] * p.y_stride + g : -1;
      factor[t][e] = tok < n_tok ? sm.factor[tok] : 0.f;
    }
  for (int64_t tile = t0 + warp; tile < t1; tile += kLoraWarps * U) {
    float acc[U][TG][4], base[U][TG][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t n = 16 * (tile + kLoraWarps * u) + 8 * (e >> 1);
          acc[u][t][e] = 0.f;
          base[u][t][e] = p.base && tile + kLoraWarps * u < t1 && n + g < p.N && at[t][e & 1] >= 0 ? lora_load(p.base, at[t][e & 1] + n, OUT) : 0.f;
        }
    for (int b = 0; b < blocks; ++b) {
      const int j = 32 * b + 8 * c;
      uint4 w[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t n = 16 * (tile + kLoraWarps * u) + 8 * h + g;
          w[u][h] = tile + kLoraWarps * u < t1 && n < p.N && j < r ? ld_stream(B + n * p.rank + j) : zero;
          if (j < r && j + 8 > r) {  // what lies past the adapter's rank does not count
            uint32_t* q = reinterpret_cast<uint32_t*>(&w[u][h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] &= j + 2 * e >= r ? 0u : j + 2 * e + 1 >= r ? 0xffffu : 0xffffffffu;
          }
        }
#pragma unroll
      for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          const uint4 s = sm.frag[t][b][q][lane];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            mma16816<BF>(acc[u][t], w[u][0].x, w[u][1].x, w[u][0].y, w[u][1].y, s.x, s.y);
            mma16816<BF>(acc[u][t], w[u][0].z, w[u][1].z, w[u][0].w, w[u][1].w, s.z, s.w);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < TG; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t n = 16 * (tile + kLoraWarps * u) + 8 * (e >> 1);
          if (tile + kLoraWarps * u < t1 && n + g < p.N && at[t][e & 1] >= 0)
            lora_store(p.y, at[t][e & 1] + n, OUT, base[u][t][e] + factor[t][e & 1] * acc[u][t][e]);
        }
  }
}

template <bool BF, int OUT>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_kernel(const qgemv_lora_t p, int slots, int* err) {
  extern __shared__ __align__(16) uint8_t dyn[];
  LoraSmem& sm = *reinterpret_cast<LoraSmem*>(dyn);
  __shared__ uint32_t rows_of[kLoraRows];  // of each distinct adapter among the rows: their mask
  __shared__ int count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(blockIdx.x) % kLoraCluster;
  const int64_t cluster = blockIdx.x / kLoraCluster;
  const int64_t chunk = cluster / slots;
  const int slot = static_cast<int>(cluster % slots);
  const int64_t m0 = chunk * kLoraRows;
  if (warp == 0) {
    const int64_t m = m0 + lane;
    int id = -2;  // past the rows
    if (m < p.rows) {
      id = p.ids[m];
      if (id < -1 || id >= p.adapters) {
        if (slot == 0 && rank == 0) atomicOr(err, kDevErrIndex);
        id = -1;
      }
    }
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    const bool first = id != -2 && __ffs(same) - 1 == lane;
    const uint32_t firsts = __ballot_sync(0xffffffffu, first);
    if (first) rows_of[__popc(firsts & ((1u << lane) - 1))] = same;
    if (lane == 0) count = __popc(firsts);
  }
  __syncthreads();
  const int64_t blocks = (p.K + 31) / 32, tiles = (p.N + 15) / 16;
  const int64_t b0 = blocks * rank / kLoraCluster, b1 = blocks * (rank + 1) / kLoraCluster;
  const int64_t t0 = tiles * rank / kLoraCluster, t1 = tiles * (rank + 1) / kLoraCluster;
  for (int i = slot; i < count; i += slots) {
    const uint32_t mask = rows_of[i];
    const int n_tok = __popc(mask);
    const int id = p.ids[m0 + __ffs(mask) - 1];
    const int a = id >= 0 && id < p.adapters ? id : -1;
    const int r = a < 0 ? 0 : p.ranks ? min(max(p.ranks[a], 0), p.rank) : p.rank;
    if (warp == 0 && (mask >> lane & 1)) sm.row[__popc(mask & ((1u << lane) - 1))] = static_cast<int>(m0) + lane;
    __syncthreads();
    if (r == 0) {  // no adapter: the base itself
      if (p.base != p.y) {
        const int64_t n0 = 16 * t0, n1 = min(16 * t1, p.N);
        for (int t = 0; t < n_tok; ++t)
          for (int64_t n = n0 + threadIdx.x; n < n1; n += kLoraThreads) {
            const int64_t at = sm.row[t] * p.y_stride + n;
            lora_store(p.y, at, OUT, p.base ? lora_load(p.base, at, OUT) : 0.f);
          }
      }
      __syncthreads();
      continue;
    }
    const uint16_t* A = static_cast<const uint16_t*>(p.A) + static_cast<int64_t>(a) * p.rank * p.K;
    const uint16_t* B = static_cast<const uint16_t*>(p.B) + static_cast<int64_t>(a) * p.N * p.rank;
    {  // this CTA's rows of B on their way to L2, 16 KB a thread
      const int64_t from = 16 * t0 * p.rank * 2, to = min(16 * t1, p.N) * p.rank * 2;
      for (int64_t o = from + threadIdx.x * int64_t{16384}; o < to; o += kLoraThreads * int64_t{16384})
        prefetch_l2(reinterpret_cast<const uint8_t*>(B) + o, static_cast<uint32_t>(min(int64_t{16384}, to - o)));
    }
    if (n_tok <= 8) {
      for (int j = 0; j < r; j += 32) lora_shrink<BF, 2, 1>(p, sm, A, r, j, n_tok, b0, b1);
    } else {
      for (int j = 0; j < r; j += 32) lora_shrink<BF, 2, 4>(p, sm, A, r, j, n_tok, b0, b1);
    }
    cluster_barrier();
    const int r4 = (r + 31) / 32 * 8;  // float4 per token; past the rank the sums are zeros
    for (int e = threadIdx.x; e < (n_tok + 7) / 8 * 8 * r4; e += kLoraThreads) {
      const int tok = e / r4, j = e % r4 * 4;
      const uint32_t at = smem_u32(&sm.own[tok][j]);
      float4 v[kLoraCluster];
#pragma unroll
      for (int q = 0; q < kLoraCluster; ++q) v[q] = cluster_ld4(at, q);
      float4 s = v[0];
#pragma unroll
      for (int q = 1; q < kLoraCluster; ++q) s.x += v[q].x, s.y += v[q].y, s.z += v[q].z, s.w += v[q].w;
      *reinterpret_cast<float4*>(&sm.sum[tok][j]) = s;
    }
    cluster_barrier();  // the sums are here, and no CTA reads another's any more
    const int groups = (n_tok + 7) / 8;
    if (warp < groups) lora_parts<BF>(sm, warp, (r + 31) / 32, p.scales ? p.scales[a] : 1.f);
    __syncthreads();
    if (n_tok <= 8)
      lora_expand<BF, 1, OUT>(p, sm, B, r, n_tok, t0, t1);
    else
      lora_expand<BF, 4, OUT>(p, sm, B, r, n_tok, t0, t1);
    __syncthreads();  // sm is used again
  }
}

}  // namespace qg
