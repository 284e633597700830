// Low-rank adapters of many requests beside a shared projection:
//   t = A_a x_m  (rank r_a),   y_m = base_m + s_a B_a t
//
// With a few rows per adapter the work is bound by the bytes of A and B, with many rows by those of base
// and y; a row's own work is 2 r (K + N) operations.  Two launches, the second a dependent one: it starts
// while the first runs, fetches its first rows of B and the base, and waits for t only then.
//  * Sums (lora_sums_kernel).  A cluster of eight CTAs takes the rows of one adapter among 32
//    neighbouring rows of the batch, each CTA an eighth of K; the partial sums meet through distributed
//    shared memory, where each CTA adds those of its own tokens in rank order.  The sums (fp32) are left in
//    the workspace as what the second product multiplies: two fp16 parts scaled by a power of two per row
//    (the row's largest in [2^14, 2^15)), or three bf16 parts: at least 21 bits of each sum.  fp16's steps end
//    at 2^-24, so where one of a row's 32 neighbouring sums is below 2^-4 (2^-18 of the row's largest; of random
//    ones, one in some ten thousand) what the two parts leave of the 32 stays in fp32, and the outputs add three
//    bf16 parts of it times two of B, which hold fp16's 11 bits.
//  * Outputs of few rows (lora_few_kernel): the rows of one adapter stay, its B streams by, through a
//    ring of cp.async in which every lane fetches what it will multiply itself (no barrier, no
//    registers).  All CTAs run at once and have equal shares of the tiles of all rows.
//  * Outputs of many rows (lora_many_kernel): 32 rows of B stay in a warp's registers, the tokens stream
//    by, 16 at a time.
//  * All products run on mma.sync m16n8k16, the first with A's rows as its 16 and the tokens as its 8, the
//    second with the tokens as its 16 and B's rows as its 8.  A lane's operands are 16 consecutive bytes of
//    its row: the order of k within a 32-wide block is the same permutation on both sides, so no shared
//    memory or ldmatrix is needed for A, B or x.  B's rows are dealt to the two 8-wide halves of a 16-row
//    tile so that a lane ends up with four consecutive outputs of a token.
// Measured: one row of rank 16, K 4096, N 6144: 6.7 us, the latency of two launches; 64 rows of 48 adapters of
// ranks up to 64, K 4096, N 12288: 24.9 us (7 of them the sums; the outputs' CTAs take 4 us to begin, and rows
// of short ranks cost whole 64-byte pieces of memory); 2048 rows of 4, rank 32, N 14336: 49.8 us (sums 12,
// outputs 37 at 6.3 TB/s).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_mma.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kLoraMaxRank = 128;
// Up to here eight tokens of an adapter at a time, and B streams by; past it B is held and the rows stream by.  256 and
// 257 rows, rank 32, N 12288, of 1 / 16 / 64 / as many adapters as rows, shuffled: 24 / 43 / 49 / 62 and 13 / 47 / 71 /
// 92 us; 16 in runs: 19 and 17.  Many rows are mostly prompts, whose rows of one adapter follow one another; where
// they do not, B is fetched again at every change.
constexpr int kLoraFewRows = 256;
constexpr int kLoraCluster = 8;
constexpr int kLoraChunk = 32;     // neighbouring rows of the batch whose adapters one warp finds
constexpr int kLoraLd = kLoraMaxRank + 4;  // floats per token of the sums in shared memory
constexpr int kLoraWarps = 4;
constexpr int kLoraThreads = 32 * kLoraWarps;

// What a launch keeps of a row beside its sums: its adapter (-1: none, or one of rank 0), the adapter's scale over
// the sums' power of two, and a bit for each block of 32 whose parts leave a rest (fp16).
struct __align__(16) LoraRow {
  int adapter;
  float factor;
  uint32_t rests, pad;
};
// The rows of a launch in the workspace: per row, the parts of its sums (blocks of 32 ranks, kParts, four
// lanes of 16 bytes).
struct LoraWork {
  uint4* parts;
  LoraRow* row;
  float* rest;  // [rows][blocks][32], only where a row has the block's bit
  int blocks;  // 32-wide blocks of the largest rank
};
__host__ __device__ constexpr int lora_parts(bool bf) { return bf ? 3 : 2; }

// TG: groups of eight tokens taken at a time.
template <int TG>
struct LoraShape {
  static constexpr int kTokens = 8 * TG;
  static constexpr int kRT = TG == 1 ? 4 : 2;       // 16-row tiles of A taken at a time
};

template <int TG>
struct LoraSmem {
  float own[8 * TG][kLoraLd];                                             // this CTA's sums over its part of K
  float part[kLoraWarps][8 * TG][16 * LoraShape<TG>::kRT + 4];            // those of a warp
};

// The rows of one adapter among kLoraChunk neighbouring ones: n of them, from `first` on in the chunk's list.
struct LoraGroup {
  int n, first, adapter, rank;  // rank 0: no adapter, or one of rank 0
};
struct LoraChunk {
  LoraGroup group[kLoraChunk];  // in order of first appearance
  int row[kLoraChunk];          // rows, group by group
  int count;
};

__device__ __forceinline__ int lora_rank(const qgemv_lora_t& p, int a) {
  return a < 0 ? 0 : p.ranks ? min(max(p.ranks[a], 0), p.rank) : p.rank;
}

// One warp looks at the kLoraChunk rows from m0 on, a lane at one: its adapter (-2: past the rows) and rank, how
// many of them have that adapter, its place among those, and where those begin in a list of the rows by adapter.
struct LoraLane {
  int id, rank, n, place, first;
};
__device__ __forceinline__ LoraLane lora_lane(const qgemv_lora_t& p, int64_t m0, int* err) {
  const int lane = threadIdx.x & 31;
  LoraLane out;
  out.id = -2;
  if (m0 + lane < p.rows) {
    out.id = p.ids[m0 + lane];
    if (out.id < -1 || out.id >= p.adapters) {
      if (err) atomicOr(err, kDevErrIndex);
      out.id = -1;
    }
  }
  out.rank = lora_rank(p, out.id);
  const uint32_t same = __match_any_sync(0xffffffffu, out.id);
  out.n = __popc(same);
  out.place = __popc(same & ((1u << lane) - 1));
  int upto = out.id != -2 && out.place == 0 ? out.n : 0;
  const int own = upto;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  out.first = __shfl_sync(0xffffffffu, upto - own, __ffs(same) - 1);
  return out;
}

// Groups the rows from m0 on by their adapters.
__device__ __forceinline__ void lora_groups(const qgemv_lora_t& p, int64_t m0, LoraChunk& out, int* err) {
  const int lane = threadIdx.x & 31;
  const LoraLane me = lora_lane(p, m0, err);
  const bool there = me.id != -2, leads = there && me.place == 0;
  if (there) out.row[me.first + me.place] = static_cast<int>(m0) + lane;
  const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
  if (leads) out.group[__popc(leaders & ((1u << lane) - 1))] = LoraGroup{me.n, me.first, me.id, me.rank};
  if (lane == 0) out.count = __popc(leaders);
}

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

template <int OUT>
__device__ __forceinline__ float4 lora_four(const uint4& d) {  // four outputs in the first 16 or 8 bytes
  if constexpr (OUT == QGEMV_OUT_F32) return make_float4(__uint_as_float(d.x), __uint_as_float(d.y), __uint_as_float(d.z), __uint_as_float(d.w));
  const float2 a = unpair16<OUT == QGEMV_OUT_BF16>(d.x), b = unpair16<OUT == QGEMV_OUT_BF16>(d.y);
  return make_float4(a.x, a.y, b.x, b.y);
}

// Zeros in place of what lies past rank r in four rows' ranks j .. j + 7 (those are read where j < r).
__device__ __forceinline__ void lora_mask(uint4 (&w)[4], int j, int r) {
  if (j >= r || j + 8 <= r) return;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t* q = reinterpret_cast<uint32_t*>(&w[h]);
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] &= j + 2 * e >= r ? 0u : j + 2 * e + 1 >= r ? 0xffffu : 0xffffffffu;
  }
}

// What the parts left of the sums of rows m0 (operand rows 0..7) and m1 (8..15), in the blocks of r0 and r1, times
// the 32 rows of B from n0 on, added to acc: three bf16 parts times two of B (the third times the first only, the
// other is at 2^-24).  Rarely called, so it is a function of its own that reads B again: in line it took registers and
// instruction cache from the loops around it.  2048 rows, N 14336, without such a row / with one / with two: rank 32
// 49.6 / 51.1 / -, rank 64 59.5 / 61.5 / 63.5, rank 128 - / 117.5 / 119.5 us (4 us a row with one load after another).
__device__ __noinline__ void lora_rests(const qgemv_lora_t& p, const LoraWork& work, int a, int n0, int64_t m0, int64_t m1, uint32_t r0, uint32_t r1,
                                        float4* acc) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, r = lora_rank(p, a);
#pragma unroll 1
  for (int e = 0; e < 2 * work.blocks; ++e) {  // a block and a half of the rows at a time
    const int b = e >> 1, k = e & 1, j = 32 * b + 8 * c;
    const bool there = (k ? r1 : r0) >> b & 1;
    if (!__any_sync(0xffffffffu, there)) continue;
    // all that is read is asked for before the first is used
    const float4* at = reinterpret_cast<const float4*>(work.rest + ((k ? m1 : m0) * work.blocks + b) * 32 + 8 * c);
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f), x = there ? __ldcg(at) : none, y = there ? __ldcg(at + 1) : none;
    uint4 w[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int n = n0 + 4 * (g >> 1) + (g & 1) + 2 * (h & 1) + 16 * (h >> 1);
      w[h] = j < r && n < p.N ? *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.B) + (static_cast<int64_t>(a) * p.N + n) * p.rank + j)
                              : make_uint4(0, 0, 0, 0);
    }
    lora_mask(w, j, r);
    float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    uint32_t part[3][4];
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part[q][i] = pair16<true>(v[2 * i], v[2 * i + 1]);
        const float2 f = unpair16<true>(part[q][i]);
        v[2 * i] -= f.x, v[2 * i + 1] -= f.y;
      }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const uint32_t u[4] = {w[h].x, w[h].y, w[h].z, w[h].w};
      float d[4] = {k ? acc[h].z : acc[h].x, k ? acc[h].w : acc[h].y, 0.f, 0.f};  // eight rows of the product, and their second parts'
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const float2 f = unpair16<false>(u[i + o]);
          split16<true>(f.x, f.y, hi[o], lo[o]);
        }
        mma16816<true>(d, part[0][i], part[1][i], part[0][i + 1], part[1][i + 1], hi[0], hi[1]);
        mma16816<true>(d, part[0][i], part[1][i], part[0][i + 1], part[1][i + 1], lo[0], lo[1]);
        mma16816<true>(d, part[2][i], 0u, part[2][i + 1], 0u, hi[0], hi[1]);
      }
      if (k)
        acc[h].z = d[0] + d[2], acc[h].w = d[1] + d[3];
      else
        acc[h].x = d[0] + d[2], acc[h].y = d[1] + d[3];
    }
  }
}
__device__ __forceinline__ void lora_add_rests(const qgemv_lora_t& p, const LoraWork& work, int a, int n0, int64_t m0, int64_t m1, uint32_t r0, uint32_t r1,
                                               float (&acc)[2][2][4]) {
  float4 d[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) d[h] = make_float4(acc[h >> 1][h & 1][0], acc[h >> 1][h & 1][1], acc[h >> 1][h & 1][2], acc[h >> 1][h & 1][3]);
  lora_rests(p, work, a, n0, m0, m1, r0, r1, d);
#pragma unroll
  for (int h = 0; h < 4; ++h)
    acc[h >> 1][h & 1][0] = d[h].x, acc[h >> 1][h & 1][1] = d[h].y, acc[h >> 1][h & 1][2] = d[h].z, acc[h >> 1][h & 1][3] = d[h].w;
}

// First product over the 32-wide blocks b0 .. b1 of K for ranks j0 .. j0 + 16 RT - 1 and 8 TG tokens, the
// blocks dealt to the warps in turn; the warps' sums go to sm.part.  Lane (g, c) = (lane / 4, lane % 4).
template <bool BF, int TG>
__device__ __forceinline__ void lora_shrink(const qgemv_lora_t& p, LoraSmem<TG>& sm, const int* rows, const uint16_t* A, int r, int j0, int n_tok, int64_t b0, int64_t b1) {
  constexpr int RT = LoraShape<TG>::kRT;
  constexpr int U = 2;  // blocks in flight
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

// A finite value past bf16's largest would round to infinity: its first part ends there, the next hold the rest.
__device__ __forceinline__ float lora_bf16_end(float v) {
  const float end = __int_as_float(0x7f7f0000);
  return fabsf(v) < __int_as_float(0x7f800000) ? fminf(fmaxf(v, -end), end) : v;
}

template <bool BF, int TG>
__global__ void __launch_bounds__(kLoraThreads, 4) lora_sums_kernel(const __grid_constant__ qgemv_lora_t p, const LoraWork work, int slots, int* err) {
  using Sh = LoraShape<TG>;
  constexpr int kParts = lora_parts(BF);
  __shared__ __align__(16) LoraSmem<TG> sm;
  __shared__ LoraChunk chunk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(blockIdx.x) % kLoraCluster, cluster = static_cast<int>(blockIdx.x) / kLoraCluster;
  const int chunks = static_cast<int>((p.rows + kLoraChunk - 1) / kLoraChunk), slot = cluster / chunks;  // those without an adapter come last
  // The second launch may start once the launch before this one has ended (the base may be its); it waits for
  // this one's end before it reads the sums.
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) lora_groups(p, static_cast<int64_t>(cluster % chunks) * kLoraChunk, chunk, slot == 0 && rank == 0 ? err : nullptr);
  __syncthreads();
  const int64_t blocks = (p.K + 31) / 32;
  const int64_t b0 = blocks * rank / kLoraCluster, b1 = blocks * (rank + 1) / kLoraCluster;
  for (int i = slot; i < chunk.count; i += slots) {
    const LoraGroup group = chunk.group[i];
    const int n_tok = group.n, a = group.adapter, r = group.rank;
    const int* all = chunk.row + group.first;
    if (rank == 0 && static_cast<int>(threadIdx.x) < n_tok) work.row[all[threadIdx.x]].adapter = r ? a : -1;
    if (r == 0) continue;
    const float scale = p.scales ? p.scales[a] : 1.f;
    const uint16_t* A = static_cast<const uint16_t*>(p.A) + static_cast<int64_t>(a) * p.rank * p.K;
    for (int k0 = 0; k0 < n_tok; k0 += Sh::kTokens) {  // up to kTokens of its rows at a time
      const int n = min(n_tok - k0, Sh::kTokens);
      for (int j = 0; j < r; j += 16 * Sh::kRT) lora_shrink<BF, TG>(p, sm, all + k0, A, r, j, n, b0, b1);
      cluster_arrive();
      cluster_wait();
      // a warp per token of this CTA, four ranks a lane
      for (int tok = rank + kLoraCluster * warp; tok < n; tok += kLoraCluster * kLoraWarps) {
        const int j = 4 * lane;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (j < r) {
          const uint32_t at = smem_u32(&sm.own[tok][j]);
          float4 q[kLoraCluster];
#pragma unroll
          for (int c = 0; c < kLoraCluster; ++c) q[c] = cluster_ld4(at, c);
#pragma unroll
          for (int c = 0; c < kLoraCluster; ++c) v[0] += q[c].x, v[1] += q[c].y, v[2] += q[c].z, v[3] += q[c].w;
        }
        float by = 1.f, back = 1.f;
        uint32_t tiny = 0;  // lanes with a sum too small for its parts
        if constexpr (!BF) {
          float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const int ex = __float_as_int(top) >> 23 & 0xff;
          if (ex >= 15 && ex < 255) {  // 2^(141 - ex) takes 1.x 2^(ex - 127) to 1.x 2^14
            by = __int_as_float((127 + 141 - ex) << 23);
            back = __int_as_float((127 - 141 + ex) << 23);
          }
          bool small = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) small |= v[e] != 0.f && fabsf(v[e]) * by < 0.0625f;
          tiny = __ballot_sync(0xffffffffu, small);
        }
        const int64_t m = all[k0 + tok];
        if (lane < 8 * work.blocks) {
          uint2* to = reinterpret_cast<uint2*>(work.parts + (m * work.blocks + lane / 8) * (4 * kParts) + lane % 8 / 2) + lane % 2;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] *= by;
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = BF && q == 0 ? lora_bf16_end(v[e]) : v[e];
            const uint32_t u0 = pair16<BF>(w[0], w[1]), u1 = pair16<BF>(w[2], w[3]);
            to[8 * q] = make_uint2(u0, u1);
            const float2 f0 = unpair16<BF>(u0), f1 = unpair16<BF>(u1);
            v[0] -= f0.x, v[1] -= f0.y, v[2] -= f1.x, v[3] -= f1.y;
          }
          if (tiny >> (lane & 24) & 0xff)
            *reinterpret_cast<float4*>(work.rest + (m * work.blocks + lane / 8) * 32 + lane % 8 * 4) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (lane == 0) {
          work.row[m].factor = scale * back;
          work.row[m].rests = (tiny & 0xffu ? 1 : 0) | (tiny & 0xff00u ? 2 : 0) | (tiny & 0xff0000u ? 4 : 0) | (tiny >> 24 ? 8 : 0);
        }
      }
      cluster_arrive();
      cluster_wait();  // no CTA reads this one's sums: they are used again, or the CTA ends
    }
  }
}

// ------------------------------------------------------------------------- outputs of few rows
// A stage of a lane's ring is one 32-wide block of ranks of a 32-row tile of N: 16 bytes of four rows of B and,
// with a tile's first block, the base of its outputs.  Lane (g, c), half k of a tile (16 rows): rows
// 4 (g / 2) + g % 2 and two further; outputs 4 c .. 4 c + 3 of token g.  The tokens are the instruction's first
// eight rows, and their second parts the other eight (the third of bf16 another instruction).
constexpr int kLoraDepth = 2;   // stages of a lane's ring
constexpr int kLoraPieces = 6;  // 16-byte pieces of a stage

struct LoraFewSmem {
  uint4 ring[kLoraWarps][kLoraDepth][kLoraPieces][32];
  uint4 parts[kLoraMaxRank / 32][3][32];  // of the tokens in hand, as a lane's operand
  float factor[8];
  uint32_t rests[8];
};

template <bool BF, int OUT>
struct LoraStream {
  static constexpr int kBytes = OUT == QGEMV_OUT_F32 ? 16 : 8;  // of four outputs
  static constexpr int kStep = 32 * kLoraWarps;                 // outputs from a warp's tile to its next
  const qgemv_lora_t& p;
  LoraFewSmem& sm;
  const int N, r, blocks, t1;
  int ask_tile, ask_b, ask_s, ask_n;  // ask_n: first row of the lane in the tile to be asked for
  const uint16_t* ask_row;            // its 16 bytes
  const uint8_t* base;                // this lane's outputs of its token, in the tile to be asked for and
  uint8_t* y;                         // in the tile in hand; null: no such token
  int64_t to_second, to_tile;         // elements from a row to the lane's second; from the last block of a tile to the next tile
  uint32_t mine;                      // this lane's first piece of its warp's ring
  bool vec;

  __device__ __forceinline__ LoraStream(const qgemv_lora_t& p_, LoraFewSmem& sm_, const int* rows, const uint16_t* B, int r_, int n_tok, int t0, int t1_)
      : p(p_), sm(sm_), N(static_cast<int>(p_.N)), r(r_), blocks((r_ + 31) / 32), t1(t1_), ask_b(0), ask_s(0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    ask_tile = t0 + warp;
    ask_n = 32 * ask_tile + 4 * (g >> 1) + (g & 1);
    ask_row = B + static_cast<int64_t>(ask_n) * p.rank + 8 * c;
    to_second = 2 * p.rank;
    to_tile = static_cast<int64_t>(kStep) * p.rank - 32 * (blocks - 1);
    mine = smem_u32(&sm.ring[warp][0][0][lane]);
    vec = p.y_stride % 4 == 0;
    const int64_t at = g < n_tok ? (rows[g] * p.y_stride + 4 * c + 32 * ask_tile) * (kBytes / 4) : 0;
    base = g < n_tok && p.base ? static_cast<const uint8_t*>(p.base) + at : nullptr;
    y = g < n_tok ? static_cast<uint8_t*>(p.y) + at : nullptr;
  }
  __device__ __forceinline__ void ask() {  // the next stage
    if (ask_tile < t1) {
      const uint32_t to = mine + ask_s * (kLoraPieces * 512);
      const int c8 = 8 * (threadIdx.x & 3), in = 32 * ask_b + c8 < r ? 16 : 0;
      if (32 * ask_tile + 32 <= N) {
#pragma unroll
        for (int h = 0; h < 4; ++h)  // rows 0, 2, 16, 18 from the lane's first
          cp_async_fill<16>(to + h * 512, ask_row + (h & 1) * to_second + (h >> 1) * 8 * to_second, in);
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          cp_async_fill<16>(to + h * 512, ask_row + (h & 1) * to_second + (h >> 1) * 8 * to_second, ask_n + 2 * (h & 1) + 16 * (h >> 1) < N ? in : 0);
      }
      if (ask_b == 0 && vec && base) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (32 * ask_tile + 16 * k + c8 / 2 + 4 <= N) cp_async_fill<kBytes>(to + (4 + k) * 512, base + 4 * k * kBytes, kBytes);
      }
      if (++ask_b < blocks) {
        ask_row += 32;
      } else {
        ask_b = 0;
        ask_tile += kLoraWarps;
        ask_n += kStep;
        ask_row += to_tile;
        if (base) base += kStep * (kBytes / 4);
      }
    }
    cp_async_commit();
    if (++ask_s == kLoraDepth) ask_s = 0;
  }
  __device__ __forceinline__ void begin() {
#pragma unroll 1
    for (int i = 0; i < kLoraDepth; ++i) ask();
  }
  __device__ __forceinline__ void run(const LoraWork& work, const int* rows, int adapter, int t0) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const float f = sm.factor[g];
    const uint32_t rests = BF ? 0 : sm.rests[g], any_rests = BF ? 0 : __reduce_or_sync(0xffffffffu, rests);
    int s = 0;
#pragma unroll 1
    for (int tile = t0 + warp; tile < t1; tile += kLoraWarps) {
      float acc[2][2][4] = {};
      uint4 old[2];
#pragma unroll 1
      for (int b = 0; b < blocks; ++b) {
        cp_async_wait<kLoraDepth - 1>();
        const uint32_t from = mine + s * (kLoraPieces * 512);
        uint4 w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) w[h] = lds_v4(from + h * 512);
        if (b == 0) old[0] = lds_v4(from + 4 * 512), old[1] = lds_v4(from + 5 * 512);
        ask();
        if (++s == kLoraDepth) s = 0;
        lora_mask(w, 32 * b + 8 * c, r);
        auto add = [&](const uint4& s0, const uint4& s1) {  // operand rows 0..7 and 8..15
#pragma unroll
          for (int h = 0; h < 4; ++h) mma16816<BF>(acc[h >> 1][h & 1], s0.x, s1.x, s0.y, s1.y, w[h].x, w[h].y);
#pragma unroll
          for (int h = 0; h < 4; ++h) mma16816<BF>(acc[h >> 1][h & 1], s0.z, s1.z, s0.w, s1.w, w[h].z, w[h].w);
        };
        add(sm.parts[b][0][lane], sm.parts[b][1][lane]);
        if constexpr (BF) add(sm.parts[b][2][lane], make_uint4(0, 0, 0, 0));
      }
      if (any_rests) lora_add_rests(p, work, adapter, 32 * tile, rests ? rows[g] : 0, 0, rests, 0, acc);
      if (!y) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int n_left = N - 32 * tile - 16 * k - 4 * c;
        uint8_t* to = y + 4 * k * kBytes;
        float4 v = make_float4(f * (acc[k][0][0] + acc[k][0][2]), f * (acc[k][0][1] + acc[k][0][3]), f * (acc[k][1][0] + acc[k][1][2]),
                               f * (acc[k][1][1] + acc[k][1][3]));
        if (n_left <= 0) continue;
        const bool whole = vec && n_left >= 4;
        if (p.base) {
          const int64_t back = static_cast<const uint8_t*>(p.base) - static_cast<const uint8_t*>(p.y);
          const float4 d = whole ? lora_four<OUT>(old[k]) : lora_load4<OUT>(to + back, 0, n_left, false);
          v.x += d.x, v.y += d.y, v.z += d.z, v.w += d.w;
        }
        lora_store4<OUT>(to, 0, n_left, whole, v);
      }
      y += kStep * (kBytes / 4);
    }
    cp_async_wait<0>();  // the ring is used again
  }
};

// Up to eight rows of one adapter among kLoraChunk neighbouring ones, from `first` on in their list, whose outputs
// cost `cost` units a tile (`at`: units of the chunk's items before).
struct LoraItem {
  int64_t at;
  int n, first, adapter, rank, cost;
};
struct LoraItems {
  int64_t total;
  LoraItem item[kLoraChunk];
  int row[kLoraChunk];
  int count;
};
__device__ __forceinline__ int64_t lora_div(int64_t a, int b) {  // 32-bit arithmetic where a allows it
  return a >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}
__device__ __forceinline__ void lora_items(const qgemv_lora_t& p, int64_t m0, int tiles, LoraItems& out) {
  const int lane = threadIdx.x & 31;
  const LoraLane me = lora_lane(p, m0, nullptr);
  const bool there = me.id != -2;
  if (there) out.row[me.first + me.place] = static_cast<int>(m0) + lane;
  const int n = min(me.n - me.place, 8);
  // by the bytes: a block of 32 ranks of a tile of B is 2 KB, a row's base and outputs 256 bytes, which alone
  // (no adapter) take longer, four copies of a thread at a time
  int cost = me.rank ? 8 * ((me.rank + 31) / 32) + n : p.base != p.y ? 3 * n : 0;
  if (!there || me.place % 8) cost = 0;
  const int64_t units = static_cast<int64_t>(cost) * tiles;
  int64_t upto = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  const uint32_t items = __ballot_sync(0xffffffffu, cost > 0);
  if (cost) out.item[__popc(items & ((1u << lane) - 1))] = LoraItem{upto - units, n, me.first + me.place, me.id, me.rank, cost};
  if (lane == 31) out.total = upto, out.count = __popc(items);
}

// All tiles of all items are cut into equal shares, one per CTA, all of which run at once: every CTA looks at all
// rows and finds its share.  Against CTAs that divide each adapter's tiles, in two rounds: 64 rows of 48 adapters of
// ranks up to 64, N 12288: 27.0 -> 24.5 us; 128 rows of 16, rank 128: 48 -> 34; 256 rows of one, rank 64, N 6144:
// 74 -> 22; 16 rows of 16, rank 16, N 6144: 8.1 -> 8.6.
template <bool BF, int OUT>
__global__ void __launch_bounds__(kLoraThreads, 4) lora_few_kernel(const __grid_constant__ qgemv_lora_t p, const __grid_constant__ LoraWork work) {
  constexpr int kParts = lora_parts(BF);
  extern __shared__ __align__(16) uint8_t dyn[];
  LoraFewSmem& sm = *reinterpret_cast<LoraFewSmem*>(dyn);
  __shared__ LoraItems list[kLoraFewRows / kLoraChunk];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int tiles = static_cast<int>((p.N + 31) / 32), chunks = static_cast<int>((p.rows + kLoraChunk - 1) / kLoraChunk);
  for (int q = warp; q < chunks; q += kLoraWarps) lora_items(p, static_cast<int64_t>(q) * kLoraChunk, tiles, list[q]);
  __syncthreads();
  int64_t total = 0;
  for (int q = 0; q < chunks; ++q) total += list[q].total;
  const int cta = static_cast<int>(blockIdx.x);
  const int64_t each = lora_div(total, static_cast<int>(gridDim.x)), more = total - each * gridDim.x;
  int64_t lo = each * cta + min(static_cast<int64_t>(cta), more), hi = lo + each + (cta < more ? 1 : 0);  // from the chunk's first unit
  bool waited = false;
  for (int q = 0; q < chunks && hi > 0; lo -= list[q].total, hi -= list[q].total, ++q) {
    const LoraItems& chunk = list[q];
    if (lo >= chunk.total) continue;
    const LoraItem& own = chunk.item[lane];
    int i = __popc(__ballot_sync(0xffffffffu, lane < chunk.count && own.at + static_cast<int64_t>(own.cost) * tiles <= lo));
    for (; i < chunk.count && chunk.item[i].at < hi; ++i) {
      const LoraItem item = chunk.item[i];
      auto tile_at = [&](int64_t unit) {  // the first that begins at or after it
        const int64_t in = unit - item.at;
        return in <= 0 ? 0 : static_cast<int>(min(lora_div(in + item.cost - 1, item.cost), static_cast<int64_t>(tiles)));
      };
      const int t0 = tile_at(lo), t1 = tile_at(hi);
      if (t0 >= t1) continue;
      const int n = item.n, r = item.rank;
      const int* rows = chunk.row + item.first;
      if (r == 0) {  // no adapter: the base itself
        const bool vec = p.y_stride % 4 == 0;
        const int64_t end = min(int64_t{32} * t1, p.N);
        for (int t = 0; t < n; ++t)
          for (int64_t e0 = int64_t{32} * t0 + 4 * threadIdx.x; e0 < end; e0 += 4 * 4 * kLoraThreads) {
            float4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int64_t e = e0 + 4 * kLoraThreads * u;
              v[u] = p.base && e < end ? lora_load4<OUT>(p.base, rows[t] * p.y_stride + e, static_cast<int>(min(p.N - e, int64_t{4})), vec) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int64_t e = e0 + 4 * kLoraThreads * u;
              if (e < end) lora_store4<OUT>(p.y, rows[t] * p.y_stride + e, static_cast<int>(min(p.N - e, int64_t{4})), vec, v[u]);
            }
          }
        continue;
      }
      LoraStream<BF, OUT> stream(p, sm, rows, static_cast<const uint16_t*>(p.B) + static_cast<int64_t>(item.adapter) * p.N * p.rank, r, n, t0, t1);
      stream.begin();
      if (!waited) pdl_wait();  // for the sums
      waited = true;
      const int blocks = (r + 31) / 32;
      uint4 v[kParts];  // at most 4 kParts operands of four warps
      const uint4* parts = work.parts + static_cast<int64_t>(rows[g < n ? g : 0]) * work.blocks * (4 * kParts) + c;
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        const int e = warp + kLoraWarps * u;
        v[u] = g < n && e < blocks * kParts ? __ldcg(parts + 4 * e) : make_uint4(0, 0, 0, 0);
      }
      if (threadIdx.x < 8) {
        const int4 row = static_cast<int>(threadIdx.x) < n ? __ldcg(reinterpret_cast<const int4*>(&work.row[rows[threadIdx.x]])) : make_int4(0, 0, 0, 0);
        sm.factor[threadIdx.x] = __int_as_float(row.y);
        sm.rests[threadIdx.x] = static_cast<uint32_t>(row.z);
      }
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        const int e = warp + kLoraWarps * u;
        if (e < blocks * kParts) sm.parts[e / kParts][e % kParts][lane] = v[u];
      }
      __syncthreads();
      stream.run(work, rows, item.adapter, t0);
      __syncthreads();
    }
  }
  pdl_launch_dependents();
  if (!waited) pdl_wait();  // the launch ends after the one before it
}

// ------------------------------------------------------------------------- outputs of many rows
// A warp keeps 32 rows of B (NB blocks of 32 ranks) and walks over tiles of 16 rows of the batch.  What a tile
// needs is asked for kLoraAhead tiles ahead, through a ring of cp.async: a lane's own 64 bytes of the base, and for
// all warps of the CTA together the rows' adapters, factors and sums.  2048 rows, N 14336, rank 32: 49.8 us with the
// inner sums (60.6 with the sums read from L2 by each warp when it needs them), rank 64: 60, rank 128: 117; with
// three tiles ahead, as it was first, 51.2 for 50.4, 84 for 60 and 113 for 113.
constexpr int kLoraAhead = 2;
template <bool BF, int NB>
struct LoraManyStage {
  uint4 sums[NB * lora_parts(BF)][2][32];  // block and part, row half
  uint4 base[kLoraWarps][4][32];           // row half and half of the outputs
  LoraRow row[16];
};
template <bool BF, int OUT, int NB>
__global__ void __launch_bounds__(kLoraThreads, NB == 1 ? 4 : NB == 2 ? 3 : 2)
    lora_many_kernel(const __grid_constant__ qgemv_lora_t p, const __grid_constant__ LoraWork work, int splits) {
  using Stage = LoraManyStage<BF, NB>;
  constexpr int kParts = lora_parts(BF);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  constexpr int kBytes = OUT == QGEMV_OUT_F32 ? 16 : 8;  // of four outputs
  const int split = static_cast<int>(blockIdx.x) % splits;
  const int n0 = (static_cast<int>(blockIdx.x) / splits * kLoraWarps + warp) * 32;
  const int64_t tiles = (p.rows + 15) / 16;
  const int t0 = static_cast<int>(tiles * split / splits), t1 = static_cast<int>(tiles * (split + 1) / splits);
  const int N = static_cast<int>(p.N);
  const bool vec = p.y_stride % 4 == 0;
  const int left[2] = {N - n0 - 4 * c, N - n0 - 16 - 4 * c};  // outputs from the lane's first in each half
  const bool whole = vec && n0 + 32 <= N;                     // all lanes' outputs are there, four at once
  extern __shared__ __align__(16) uint8_t dyn[];
  Stage* ring = reinterpret_cast<Stage*>(dyn);
  const int m_first = 16 * t0 + g, m_end = static_cast<int>(min(p.rows, int64_t{16} * t1));
  const int64_t row8 = 8 * p.y_stride * (kBytes / 4), lane_at = (m_first * p.y_stride + n0 + 4 * c) * (kBytes / 4);
  const int part_row = 4 * kParts * work.blocks;
  // of row g of the next tile to be asked for
  const uint8_t* base_at = p.base ? static_cast<const uint8_t*>(p.base) + lane_at : nullptr;
  const uint4* part_at = work.parts + static_cast<int64_t>(m_first) * part_row + c;
  int m_base = m_first, m_sums = m_first;
  // of the tile in hand
  const uint8_t* old_at = base_at;
  uint8_t* y_at = static_cast<uint8_t*>(p.y) + lane_at;
  auto ask_base = [&](Stage& st) {
    if (!whole || !base_at) return;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (m_base + 8 * h < m_end) {
#pragma unroll
        for (int k = 0; k < 2; ++k) cp_async_fill<kBytes>(smem_u32(&st.base[warp][2 * h + k][lane]), base_at + h * row8 + k * 4 * kBytes, kBytes);
      }
    base_at += 2 * row8;
    m_base += 16;
  };
  auto ask_sums = [&](Stage& st) {  // a fourth of the CTA's
    for (int q = warp; q < kParts * work.blocks; q += kLoraWarps)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (m_sums + 8 * h < m_end) cp_async_fill<16>(smem_u32(&st.sums[q][h][lane]), part_at + h * 8 * part_row + q * 4, 16);
    if (warp == kLoraWarps - 1 && c < 2 && m_sums + 8 * c < m_end) cp_async_fill<16>(smem_u32(&st.row[g + 8 * c]), work.row + m_sums + 8 * c, 16);
    part_at += 16 * part_row;
    m_sums += 16;
    cp_async_commit();
  };
  uint4 w[NB][4];
  int cur = -1;
  auto hold = [&](int a) {  // the rows of B of adapter a
    cur = a;
    const int r = lora_rank(p, a);
    const uint16_t* at = static_cast<const uint16_t*>(p.B) + (static_cast<int64_t>(a) * p.N + n0 + 4 * (g >> 1) + (g & 1)) * p.rank + 8 * c;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int row = 2 * (h & 1) + 16 * (h >> 1);
        w[b][h] = 32 * b + 8 * c < r && n0 + 4 * (g >> 1) + (g & 1) + row < N ? *reinterpret_cast<const uint4*>(at + row * p.rank + 32 * b) : make_uint4(0, 0, 0, 0);
      }
      lora_mask(w[b], 32 * b + 8 * c, r);
    }
  };
#pragma unroll 1
  for (int i = 0; i < kLoraAhead; ++i) ask_base(ring[i]);
  pdl_wait();  // for the sums; the base is not theirs
#pragma unroll 1
  for (int i = 0; i < kLoraAhead; ++i) ask_sums(ring[i]);
  int s = 0;
#pragma unroll 1
  for (int tile = t0, m = m_first; tile < t1; ++tile, m += 16) {
    const Stage& st = ring[s];
    cp_async_wait<kLoraAhead - 1>();
    __syncthreads();  // every warp's copies are there, and every warp is through with the tile before
    Stage& next = ring[s == 0 ? kLoraAhead : s - 1];
    ask_base(next);
    ask_sums(next);
    LoraRow row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) row[h] = m + 8 * h < m_end ? st.row[g + 8 * h] : LoraRow{-1, 0.f, 0u, 0u};
    // One adapter after another, and the rows without one: mostly a single pass, as rows of one adapter follow
    // one another.  A pass has its own sums, of which it writes its rows': an adapter with infinities or NaN
    // makes NaN of the others' rows.
    bool todo[2] = {m < m_end, m + 8 < m_end};
#pragma unroll 1
    for (;;) {
      const uint32_t has0 = __ballot_sync(0xffffffffu, todo[0]), has1 = __ballot_sync(0xffffffffu, todo[1]);
      if (!(has0 | has1)) break;
      const int a = __shfl_sync(0xffffffffu, has0 ? row[0].adapter : row[1].adapter, __ffs(has0 ? has0 : has1) - 1);
      const bool in[2] = {todo[0] && row[0].adapter == a, todo[1] && row[1].adapter == a};
      float acc[2][2][4] = {};
      if (a >= 0) {
        if (a != cur) hold(a);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (NB == 4 && b == 3 && work.blocks == 3) break;
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            const uint4 s0 = in[0] ? st.sums[b * kParts + q][0][lane] : zero, s1 = in[1] ? st.sums[b * kParts + q][1][lane] : zero;
#pragma unroll
            for (int h = 0; h < 4; ++h) mma16816<BF>(acc[h >> 1][h & 1], s0.x, s1.x, s0.y, s1.y, w[b][h].x, w[b][h].y);
#pragma unroll
            for (int h = 0; h < 4; ++h) mma16816<BF>(acc[h >> 1][h & 1], s0.z, s1.z, s0.w, s1.w, w[b][h].z, w[b][h].w);
          }
        }
        if constexpr (!BF) {
          const uint32_t rests[2] = {in[0] ? row[0].rests : 0u, in[1] ? row[1].rests : 0u}, any_rests = __reduce_or_sync(0xffffffffu, rests[0] | rests[1]);
          if (any_rests) lora_add_rests(p, work, a, n0, m, m + 8, rests[0], rests[1], acc);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!in[h]) continue;
        todo[h] = false;
        const float f = a >= 0 ? row[h].factor : 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (left[k] <= 0) continue;
          float4 v = make_float4(f * acc[k][0][2 * h], f * acc[k][0][2 * h + 1], f * acc[k][1][2 * h], f * acc[k][1][2 * h + 1]);
          const int64_t off = h * row8 + k * 4 * kBytes;
          if (old_at) {
            const float4 d = whole ? lora_four<OUT>(st.base[warp][2 * h + k][lane]) : lora_load4<OUT>(old_at + off, 0, left[k], vec);
            v.x += d.x, v.y += d.y, v.z += d.z, v.w += d.w;
          }
          lora_store4<OUT>(y_at + off, 0, left[k], vec, v);
        }
      }
    }
    if (old_at) old_at += 2 * row8;
    y_at += 2 * row8;
    if (++s > kLoraAhead) s = 0;
  }
}

}  // namespace qg
