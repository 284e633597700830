// Low-rank adapters of many requests beside a shared projection:
//   t = A_a x_m  (rank r_a),   y_m = base_m + s_a B_a t
//
// With a few rows per adapter the kernel is bound by the bytes of A and B, with many rows by those of
// base and y; a row's own work is 2 r (K + N) operations.  One launch does both products:
//  * A cluster of eight CTAs takes the rows of one adapter among 16 or 32 neighbouring rows of the batch.
//    Each CTA forms the inner sums over its eighth of K; the eight partial sums meet through
//    distributed shared memory (each CTA adds all of them in rank order), and each CTA writes its
//    eighth of N.  So the inner sums never leave the chip, and a single row still uses eight SMs.
//  * Every lane fetches what it will multiply itself, B's rows and the base, through a ring of cp.async
//    in shared memory, and its first stages before the first product begins: no barrier, no registers.
//  * Both products run on mma.sync m16n8k16, the first with A's rows as its 16 and the tokens as its 8, the
//    second with the tokens as its 16 and B's rows as its 8.  A lane's operands are 16 consecutive bytes of
//    its row: the order of k within a 32-wide block is the same permutation on both sides, so no shared
//    memory or ldmatrix is needed for A, B or x.  B's rows are dealt to the two 8-wide halves of a 16-row
//    tile so that a lane ends up with four consecutive outputs of a token.
//  * The inner sums (fp32) enter the second product as two fp16 parts scaled by a power of two per row
//    (the row's largest in [2^14, 2^15)), or three bf16 parts: at least 21 bits.  Up to eight tokens have
//    their first two parts in the upper and the lower eight rows of one instruction.
//  * Two shapes, both of CTAs of 4 warps: up to 8 tokens at a time of an adapter's rows among 32 (a few
//    rows per adapter), and up to 16 among 16 (many rows: more clusters than run at once, so that they
//    even out over the SMs).  Where the rows are few, several clusters share an adapter's N; each forms
//    the inner sums for itself.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_mma.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kLoraMaxRank = 128;
constexpr int kLoraFewRows = 256;  // up to here eight tokens at a time
constexpr int kLoraCluster = 8;
constexpr int kLoraLd = kLoraMaxRank + 4;  // floats per token of the sums in shared memory

constexpr int kLoraWarps = 4;
constexpr int kLoraThreads = 32 * kLoraWarps;

// TG: groups of eight tokens taken at a time.
template <int TG>
struct LoraShape {
  static constexpr int kTokens = 8 * TG;
  static constexpr int kRows = TG == 1 ? 32 : 16;   // neighbouring rows of the batch per cluster
  static constexpr int kRT = 4;                     // 16-row tiles of A taken at a time
  static constexpr int kCtasPerSm = TG == 1 ? 4 : 3;
  static constexpr int kDepth = TG == 1 ? 3 : 2;    // stages of a lane's ring
  static constexpr int kPieces = 4 + 2 * TG;        // 16-byte pieces of a stage: four of B, two of the base per token
};

template <int TG>
struct LoraSmem {
  using Sh = LoraShape<TG>;
  uint4 ring[kLoraWarps][Sh::kDepth][Sh::kPieces][32];
  float own[Sh::kTokens][kLoraLd];                  // this CTA's sums over its part of K
  union {
    float part[kLoraWarps][Sh::kTokens][16 * Sh::kRT + 4];  // first product: per warp
    struct {
      float sum[Sh::kTokens][kLoraLd];                      // over all of K
      uint4 frag[TG][kLoraMaxRank / 32][3][32];             // 16-bit parts of the sums, as a lane's operand
    };
  };
  float factor[Sh::kTokens];                        // of a token: the adapter's scale over the parts' power of two
  int row[Sh::kRows];                               // rows of the adapter in hand
};

__device__ __forceinline__ float4 cluster_ld4(uint32_t a, uint32_t rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(r) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// `bytes` (8 or 16) of cp.async, of which `in` are read and the rest are zeros.
template <int BYTES>
__device__ __forceinline__ void cp_async_fill(uint32_t dst, const void* src, int in) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
  constexpr int RT = LoraShape<TG>::kRT;
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

// Second product: outputs of the 32-row tiles t0 .. t1 of N, dealt to the warps in turn, for up to 8 TG
// tokens.  A stage of a lane's ring is one 32-wide block of ranks of a tile: 16 bytes of four rows of B and,
// with a tile's first block, the base of its outputs.  Lane (g, c), half k of a tile (16 rows): rows
// 4 (g / 2) + g % 2 and two further; outputs 4 c .. 4 c + 3 of tokens g and g + 8.
template <bool BF, int TG, int OUT>
struct LoraExpand {
  using Sh = LoraShape<TG>;
  static constexpr int D = Sh::kDepth;
  static constexpr int kBytes = OUT == QGEMV_OUT_F32 ? 16 : 8;  // of four outputs
  const qgemv_lora_t& p;
  LoraSmem<TG>& sm;
  const int N, r, blocks, t1;
  int ask_tile, ask_b, ask_s, ask_n;  // ask_n: first row of the lane in the tile to be asked for
  const uint16_t* ask_row;            // its 16 bytes
  const uint8_t* base[TG];            // this lane's outputs of its tokens, in the tile to be asked for and
  uint8_t* y[TG];                     // in the tile in hand; null: no such token
  int64_t to_second, to_tile;         // elements from a row to the lane's second; from the last block of a tile to the next tile
  uint32_t mine;                      // this lane's first piece of its warp's ring
  bool vec;
  static constexpr int kStep = 32 * kLoraWarps;  // outputs from a warp's tile to its next

  __device__ __forceinline__ LoraExpand(const qgemv_lora_t& p_, LoraSmem<TG>& sm_, const int* rows, const uint16_t* B, int r_, int n_tok, int t0, int t1_)
      : p(p_), sm(sm_), N(static_cast<int>(p_.N)), r(r_), blocks((r_ + 31) / 32), t1(t1_), ask_b(0), ask_s(0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    ask_tile = t0 + warp;
    ask_n = 32 * ask_tile + 4 * (g >> 1) + (g & 1);
    ask_row = B + static_cast<int64_t>(ask_n) * p.rank + 8 * c;
    to_second = 2 * p.rank;
    to_tile = static_cast<int64_t>(kStep) * p.rank - 32 * (blocks - 1);
    mine = smem_u32(&sm.ring[warp][0][0][lane]);
    vec = p.y_stride % 4 == 0;
#pragma unroll
    for (int h = 0; h < TG; ++h) {
      const bool there = 8 * h + g < n_tok;
      const int64_t at = there ? (rows[8 * h + g] * p.y_stride + 4 * c + 32 * ask_tile) * (kBytes / 4) : 0;
      base[h] = there && p.base ? static_cast<const uint8_t*>(p.base) + at : nullptr;
      y[h] = there ? static_cast<uint8_t*>(p.y) + at : nullptr;
    }
  }
  __device__ __forceinline__ void ask() {  // the next stage
    if (ask_tile < t1) {
      const uint32_t to = mine + ask_s * (Sh::kPieces * 512);
      const int c8 = 8 * (threadIdx.x & 3);
      const bool in = 32 * ask_b + c8 < r;
#pragma unroll
      for (int h = 0; h < 4; ++h)  // rows 0, 2, 16, 18 from the lane's first
        cp_async_fill<16>(to + h * 512, ask_row + (h & 1) * to_second + (h >> 1) * 8 * to_second, in && ask_n + 2 * (h & 1) + 16 * (h >> 1) < N ? 16 : 0);
      if (ask_b == 0 && vec) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (32 * ask_tile + 16 * k + c8 / 2 + 4 <= N) {
#pragma unroll
            for (int h = 0; h < TG; ++h)
              if (base[h]) cp_async_fill<kBytes>(to + (4 + 2 * h + k) * 512, base[h] + 4 * k * kBytes, kBytes);
          }
      }
      if (++ask_b < blocks) {
        ask_row += 32;
      } else {
        ask_b = 0;
        ask_tile += kLoraWarps;
        ask_n += kStep;
        ask_row += to_tile;
#pragma unroll
        for (int h = 0; h < TG; ++h)
          if (base[h]) base[h] += kStep * (kBytes / 4);
      }
    }
    cp_async_commit();
    if (++ask_s == D) ask_s = 0;
  }
  __device__ __forceinline__ void begin() {
#pragma unroll 1
    for (int i = 0; i < D; ++i) ask();
  }
  __device__ __forceinline__ void run(int t0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    float factor[TG];
#pragma unroll
    for (int h = 0; h < TG; ++h) factor[h] = sm.factor[8 * h + g];
    int s = 0;
#pragma unroll 1
    for (int tile = t0 + warp; tile < t1; tile += kLoraWarps) {
      float acc[2][2][4] = {};
      uint4 old[TG][2];
#pragma unroll 1
      for (int b = 0; b < blocks; ++b) {
        cp_async_wait<D - 1>();
        const uint32_t from = mine + s * (Sh::kPieces * 512);
        uint4 w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) w[h] = lds_v4(from + h * 512);
        if (b == 0) {
#pragma unroll
          for (int h = 0; h < 2 * TG; ++h) old[h >> 1][h & 1] = lds_v4(from + (4 + h) * 512);
        }
        ask();
        if (++s == D) s = 0;
        const int j = 32 * b + 8 * c;
        if (j < r && j + 8 > r) {  // what lies past the adapter's rank does not count
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t* q = reinterpret_cast<uint32_t*>(&w[h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] &= j + 2 * e >= r ? 0u : j + 2 * e + 1 >= r ? 0xffffu : 0xffffffffu;
          }
        }
        auto add = [&](const uint4& s0, const uint4& s1) {  // operand rows 0..7 and 8..15
#pragma unroll
          for (int h = 0; h < 4; ++h) mma16816<BF>(acc[h >> 1][h & 1], s0.x, s1.x, s0.y, s1.y, w[h].x, w[h].y);
#pragma unroll
          for (int h = 0; h < 4; ++h) mma16816<BF>(acc[h >> 1][h & 1], s0.z, s1.z, s0.w, s1.w, w[h].z, w[h].w);
        };
        if constexpr (TG == 1) {
          add(sm.frag[0][b][0][lane], sm.frag[0][b][1][lane]);
          if constexpr (BF) add(sm.frag[0][b][2][lane], make_uint4(0, 0, 0, 0));
        } else {
#pragma unroll
          for (int q = 0; q < (BF ? 3 : 2); ++q) add(sm.frag[0][b][q][lane], sm.frag[1][b][q][lane]);
        }
      }
#pragma unroll
      for (int h = 0; h < TG; ++h) {
        if (!y[h]) continue;
        const float f = factor[h];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int n_left = N - 32 * tile - 16 * k - 4 * c;
          uint8_t* to = y[h] + 4 * k * kBytes;
          float4 v;
          if constexpr (TG == 1)
            v = make_float4(acc[k][0][0] + acc[k][0][2], acc[k][0][1] + acc[k][0][3], acc[k][1][0] + acc[k][1][2], acc[k][1][1] + acc[k][1][3]);
          else
            v = make_float4(acc[k][0][2 * h], acc[k][0][2 * h + 1], acc[k][1][2 * h], acc[k][1][2 * h + 1]);
          v = make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
          if (vec && n_left >= 4) {
            if (p.base) {
              const uint4 d = old[h][k];
              if constexpr (OUT == QGEMV_OUT_F32) {
                v.x += __uint_as_float(d.x), v.y += __uint_as_float(d.y), v.z += __uint_as_float(d.z), v.w += __uint_as_float(d.w);
              } else {
                const float2 a = unpair16<OUT == QGEMV_OUT_BF16>(d.x), e = unpair16<OUT == QGEMV_OUT_BF16>(d.y);
                v.x += a.x, v.y += a.y, v.z += e.x, v.w += e.y;
              }
            }
            lora_store4<OUT>(to, 0, 4, true, v);
          } else if (n_left > 0) {
            if (p.base) {
              const int64_t back = static_cast<const uint8_t*>(p.base) - static_cast<const uint8_t*>(p.y);
              const float4 d = lora_load4<OUT>(to + back, 0, n_left, false);
              v.x += d.x, v.y += d.y, v.z += d.z, v.w += d.w;
            }
            lora_store4<OUT>(to, 0, n_left, false, v);
          }
        }
        y[h] += kStep * (kBytes / 4);
      }
    }
    cp_async_wait<0>();  // the ring is used again
  }
};

template <bool BF, int OUT, int TG>
__global__ void __launch_bounds__(kLoraThreads, LoraShape<TG>::kCtasPerSm) lora_kernel(const qgemv_lora_t p, int slots, int shares, int* err) {
  using Sh = LoraShape<TG>;
  constexpr int kLoraRows = Sh::kRows;
  extern __shared__ __align__(16) uint8_t dyn[];
  LoraSmem<TG>& sm = *reinterpret_cast<LoraSmem<TG>*>(dyn);
  __shared__ uint32_t rows_of[kLoraRows];  // of each distinct adapter among the rows: their mask
  __shared__ int count;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(blockIdx.x) % kLoraCluster;
  const int cluster = static_cast<int>(blockIdx.x) / kLoraCluster, share = cluster % shares;
  const int slot = cluster / shares % slots;
  const int64_t chunk = cluster / shares / slots;
  const int64_t m0 = chunk * kLoraRows;
  if (warp == 0) {
    const int64_t m = m0 + lane;
    int id = -2;  // past the rows
    if (lane < kLoraRows && m < p.rows) {
      id = p.ids[m];
      if (id < -1 || id >= p.adapters) {
        if (slot == 0 && share == 0 && rank == 0) atomicOr(err, kDevErrIndex);
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
  const int64_t blocks = (p.K + 31) / 32, tiles = (p.N + 31) / 32, parts = shares * kLoraCluster, part = share * kLoraCluster + rank;
  const int64_t b0 = blocks * rank / kLoraCluster, b1 = blocks * (rank + 1) / kLoraCluster;
  const int t0 = static_cast<int>(tiles * part / parts), t1 = static_cast<int>(tiles * (part + 1) / parts);
  for (int i = slot; i < count; i += slots) {
    const uint32_t mask = rows_of[i];
    const int n_tok = __popc(mask);
    const int id = p.ids[m0 + __ffs(mask) - 1];
    const int a = id >= 0 && id < p.adapters ? id : -1;
    const int r = a < 0 ? 0 : p.ranks ? min(max(p.ranks[a], 0), p.rank) : p.rank;
    const float scale = a >= 0 && p.scales ? p.scales[a] : 1.f;
    if (warp == 0 && (mask >> lane & 1)) sm.row[__popc(mask & ((1u << lane) - 1))] = static_cast<int>(m0) + lane;
    __syncthreads();
    if (r == 0) {  // no adapter: the base itself
      if (p.base != p.y) {
        const bool vec = p.y_stride % 4 == 0;
        for (int t = 0; t < n_tok; ++t)
          for (int64_t n = int64_t{32} * t0 + 4 * threadIdx.x; n < min(int64_t{32} * t1, p.N); n += 4 * kLoraThreads) {
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
    for (int k0 = 0; k0 < n_tok; k0 += Sh::kTokens) {  // up to kTokens of its rows at a time
      const int* rows = sm.row + k0;
      const int n = min(n_tok - k0, Sh::kTokens);
      LoraExpand<BF, TG, OUT> expand(p, sm, rows, B, r, n, t0, t1);
      expand.begin();
      for (int j = 0; j < r; j += 16 * Sh::kRT) lora_shrink<BF, TG>(p, sm, rows, A, r, j, n, b0, b1);
      cluster_arrive();
      cluster_wait();
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
      cluster_arrive();  // this CTA reads the others' sums no more
      __syncthreads();
      if (warp < (n + 7) / 8) lora_parts<BF, TG>(sm, warp, (r + 31) / 32, scale);
      __syncthreads();
      expand.run(t0);
      cluster_wait();  // no CTA reads this one's sums: they are used again, or the CTA ends
      __syncthreads();
    }
  }
}

}  // namespace qg
