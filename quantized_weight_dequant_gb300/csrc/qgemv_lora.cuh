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
//  * Both products run on mma.sync m16n8k16, the first with A's rows as its 16 and the tokens as its 8, the
//    second with the tokens as its 16 and B's rows as its 8.  A lane's operands are 16 consecutive bytes of
//    its row: the order of k within a 32-wide block is the same permutation on both sides, so no shared
//    memory or ldmatrix is needed for A, B or x.  B's rows are dealt to the two 8-wide halves of a 16-row
//    tile so that a lane ends up with four consecutive outputs of a token.
//  * The inner sums (fp32) enter the second product as two fp16 parts scaled by a power of two per row
//    (the row's largest in [2^14, 2^15)), or three bf16 parts: at least 21 bits.  Up to eight tokens have
//    their first two parts in the upper and the lower eight rows of one instruction.
//  * Two shapes: up to 8 tokens at a time in CTAs of 4 warps, four on an SM (a few rows per adapter: the
//    whole batch is resident at once), and up to 32 in CTAs of 8 warps (many rows: A and B are read once
//    per 32 rows).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_mma.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraRows = 32;      // rows of the batch per cluster: one warp finds the rows of an adapter
constexpr int kLoraFewRows = 256;  // up to here eight tokens at a time
constexpr int kLoraCluster = 8;
constexpr int kLoraLd = kLoraMaxRank + 4;  // floats per token of the sums in shared memory

// TG: groups of eight tokens taken at a time.
template <int TG>
struct LoraShape {
  static constexpr int kWarps = TG == 1 ? 4 : 8, kThreads = 32 * kWarps, kCtasPerSm = TG == 1 ? 4 : 2;
  static constexpr int kRT = TG == 1 ? 4 : 2;  // 16-row tiles of A taken at a time
  static constexpr int kTokens = 8 * TG;
};

template <int TG>
struct LoraSmem {
  static constexpr int kT = LoraShape<TG>::kTokens;
  float part[LoraShape<TG>::kWarps][kT][16 * LoraShape<TG>::kRT + 4];  // first product: per warp
  float own[kT][kLoraLd];                           // this CTA's sums over its part of K
  float sum[kT][kLoraLd];                           // over all of K
  uint4 frag[TG][kLoraMaxRank / 32][3][32];         // 16-bit parts of the sums, as a lane's operand
  float factor[kT];                                 // of a token: the adapter's scale over the parts' power of two
  int row[kLoraRows];                               // rows of the adapter in hand
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

// Outputs i .. i + 3 of the flat array p, the first n of them (vec: 16- or 8-byte accesses are aligned).
template <int OUT>
__device__ __forceinline__ float4 lora_load4(const void* p, int64_t i, int n, bool vec) {
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (vec && n >= 4) {
    if constexpr (OUT == QGEMV_OUT_F32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    const float2 a = unpair16<OUT == QGEMV_OUT_BF16>(u.x), b = unpair16<OUT == QGEMV_OUT_BF16>(u.y);
    return make_float4(a.x, a.y, b.x, b.y);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) {
      if constexpr (OUT == QGEMV_OUT_F32)
        v[e] = static_cast<const float*>(p)[i + e];
      else
        v[e] = unpair16<OUT == QGEMV_OUT_BF16>(static_cast<const uint16_t*>(p)[i + e]).x;
    }
  return make_float4(v[0], v[1], v[2], v[3]);
}
template <int OUT>
__device__ __forceinline__ void lora_store4(void* p, int64_t i, int n, bool vec, float4 v) {
  constexpr bool kBF = OUT == QGEMV_OUT_BF16;
  if (vec && n >= 4) {
    if constexpr (OUT == QGEMV_OUT_F32)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(pair16<kBF>(v.x, v.y), pair16<kBF>(v.z, v.w));
    return;
  }
  const float w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n) {
      if constexpr (OUT == QGEMV_OUT_F32)
        static_cast<float*>(p)[i + e] = w[e];
      else
        static_cast<uint16_t*>(p)[i + e] = static_cast<uint16_t>(pair16<kBF>(w[e], 0.f));
    }
}

// First product over the 32-wide blocks b0 .. b1 of K for ranks j0 .. j0 + 16 RT - 1 and 8 TG tokens, the
// blocks dealt to the warps in turn; the warps' sums go to sm.part.  Lane (g, c) = (lane / 4, lane % 4).
template <bool BF, int TG>
__device__ __forceinline__ void lora_shrink(const qgemv_lora_t& p, LoraSmem<TG>& sm, const int* rows, const uint16_t* A, int r, int j0, int n_tok, int64_t b0, int64_t b1) {
  constexpr int RT = LoraShape<TG>::kRT, kLoraWarps = LoraShape<TG>::kWarps, kLoraThreads = LoraShape<TG>::kThreads;
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
    xr[t] = 8 * t + g < n_tok ? static_cast<const uint16_t*>(p.x) + rows[8 * t + g] * p.x_stride + 8 * c : nullptr;
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
template <bool BF, int TG>
__device__ __forceinline__ void lora_parts(LoraSmem<TG>& sm, int t, int blocks, float scale) {
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
__device__ __forceinline__ void lora_expand(const qgemv_lora_t& p, const LoraSmem<TG>& sm, const int* rows, const uint16_t* B, int r, int n_tok, int64_t t0, int64_t t1) {
  constexpr int kLoraWarps = LoraShape<TG>::kWarps;
  constexpr int U = TG == 1 ? 4 : 2;            // tiles in flight
  constexpr int TM = TG == 1 ? 1 : TG / 2;      // 16-token tiles
  constexpr int R = TG == 1 ? 1 : 2;            // rows of a lane in each: tokens g, and g + 8
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int blocks = (r + 31) / 32;
  const bool vec = p.y_stride % 4 == 0;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  int64_t at[TM][R];
  float factor[TM][R];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int h = 0; h < R; ++h) {
      const int tok = 16 * t + 8 * h + g;
      at[t][h] = tok < n_tok ? rows[tok] * p.y_stride + 4 * c : -1;
      factor[t][h] = tok < n_tok ? sm.factor[tok] : 0.f;
    }
  const int64_t my_row = 4 * (g >> 1) + (g & 1);  // of B in a tile; its second half begins two rows on
  for (int64_t tile = t0 + warp; tile < t1; tile += kLoraWarps * U) {
    float acc[U][TM][2][4];
    float4 base[U][TM][R];
    int left[U];  // outputs from this lane's first on
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tl = tile + kLoraWarps * u, n = 16 * tl + 4 * c;
      left[u] = tl < t1 ? static_cast<int>(min(p.N - n, int64_t{4})) : 0;
#pragma unroll
      for (int t = 0; t < TM; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[u][t][h][0] = acc[u][t][h][1] = acc[u][t][h][2] = acc[u][t][h][3] = 0.f;
#pragma unroll
        for (int h = 0; h < R; ++h)
          base[u][t][h] = p.base && left[u] > 0 && at[t][h] >= 0 ? lora_load4<OUT>(p.base, at[t][h] + 16 * tl, left[u], vec) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    for (int b = 0; b < blocks; ++b) {
      const int j = 32 * b + 8 * c;
      uint4 w[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t tl = tile + kLoraWarps * u, n = 16 * tl + my_row + 2 * h;
          w[u][h] = tl < t1 && n < p.N && j < r ? ld_stream(B + n * p.rank + j) : zero;
        }
      if (j < r && j + 8 > r) {  // what lies past the adapter's rank does not count
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t* q = reinterpret_cast<uint32_t*>(&w[u][h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] &= j + 2 * e >= r ? 0u : j + 2 * e + 1 >= r ? 0xffffu : 0xffffffffu;
          }
      }
      if constexpr (TG == 1) {
        const uint4 s0 = sm.frag[0][b][0][lane], s1 = sm.frag[0][b][1][lane];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mma16816<BF>(acc[u][0][h], s0.x, s1.x, s0.y, s1.y, w[u][h].x, w[u][h].y);
            mma16816<BF>(acc[u][0][h], s0.z, s1.z, s0.w, s1.w, w[u][h].z, w[u][h].w);
          }
        if constexpr (BF) {
          const uint4 s2 = sm.frag[0][b][2][lane];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              mma16816<BF>(acc[u][0][h], s2.x, 0u, s2.y, 0u, w[u][h].x, w[u][h].y);
              mma16816<BF>(acc[u][0][h], s2.z, 0u, s2.w, 0u, w[u][h].z, w[u][h].w);
            }
        }
      } else {
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          if (16 * t >= n_tok) break;
#pragma unroll
          for (int q = 0; q < (BF ? 3 : 2); ++q) {
            const uint4 s0 = sm.frag[2 * t][b][q][lane], s1 = sm.frag[2 * t + 1][b][q][lane];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                mma16816<BF>(acc[u][t][h], s0.x, s1.x, s0.y, s1.y, w[u][h].x, w[u][h].y);
                mma16816<BF>(acc[u][t][h], s0.z, s1.z, s0.w, s1.w, w[u][h].z, w[u][h].w);
              }
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int h = 0; h < R; ++h) {
          if (left[u] <= 0 || at[t][h] < 0) continue;
          const float f = factor[t][h];
          const float4 d = base[u][t][h];
          float4 v;
          if constexpr (TG == 1) {
            v = make_float4(acc[u][t][0][0] + acc[u][t][0][2], acc[u][t][0][1] + acc[u][t][0][3],
                            acc[u][t][1][0] + acc[u][t][1][2], acc[u][t][1][1] + acc[u][t][1][3]);
          } else {
            v = make_float4(acc[u][t][0][2 * h], acc[u][t][0][2 * h + 1], acc[u][t][1][2 * h], acc[u][t][1][2 * h + 1]);
          }
          lora_store4<OUT>(p.y, at[t][h] + 16 * (tile + kLoraWarps * u), left[u], vec, make_float4(d.x + f * v.x, d.y + f * v.y, d.z + f * v.z, d.w + f * v.w));
        }
  }
}

template <bool BF, int OUT, int TG>
__global__ void __launch_bounds__(LoraShape<TG>::kThreads, LoraShape<TG>::kCtasPerSm) lora_kernel(const qgemv_lora_t p, int slots, int* err) {
  using Sh = LoraShape<TG>;
  constexpr int kLoraThreads = Sh::kThreads;
  extern __shared__ __align__(16) uint8_t dyn[];
  LoraSmem<TG>& sm = *reinterpret_cast<LoraSmem<TG>*>(dyn);
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
        const bool vec = p.y_stride % 4 == 0;
        for (int t = 0; t < n_tok; ++t)
          for (int64_t n = 16 * t0 + 4 * threadIdx.x; n < min(16 * t1, p.N); n += 4 * kLoraThreads) {
            const int64_t at = sm.row[t] * p.y_stride + n;
            const int left = static_cast<int>(min(p.N - n, int64_t{4}));
            lora_store4<OUT>(p.y, at, left, vec, p.base ? lora_load4<OUT>(p.base, at, left, vec) : make_float4(0.f, 0.f, 0.f, 0.f));
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
    for (int k0 = 0; k0 < n_tok; k0 += Sh::kTokens) {  // up to kTokens of its rows at a time
      const int* rows = sm.row + k0;
      const int n = min(n_tok - k0, Sh::kTokens);
      for (int j = 0; j < r; j += 16 * Sh::kRT) lora_shrink<BF, TG>(p, sm, rows, A, r, j, n, b0, b1);
      cluster_barrier();
      const int r4 = (r + 31) / 32 * 8;  // float4 per token; past the rank the sums are zeros
      for (int e = threadIdx.x; e < (n + 7) / 8 * 8 * r4; e += kLoraThreads) {
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
      if (warp < (n + 7) / 8) lora_parts<BF, TG>(sm, warp, (r + 31) / 32, p.scales ? p.scales[a] : 1.f);
      __syncthreads();
      lora_expand<BF, TG, OUT>(p, sm, rows, B, r, n, t0, t1);
      __syncthreads();  // sm is used again
    }
  }
}

}  // namespace qg
