// Projection of e4m3 rows by e4m3 weights, each with a scale for blocks of 128:
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] W[n, k].
//
// A block's inner sums come from the fifth-generation tensor cores (kind::f8f6f4, 32 along K an instruction,
// four to a block) and stay in tensor memory until a warpgroup has added them, times the block's two scales, to
// fp32 accumulators in its registers: the scales change with every block, so the sum over blocks cannot stay in
// tensor memory.
//
// What bounds few rows of x, up to 64, is the bytes of W, N K of them.  A CTA has a tile of 128 weight rows and all BT rows of
// x, or with few tiles a cluster of CTAs has it and each takes a share of its blocks; then every CTA leaves its sums in shared
// memory and adds a part of the tile over the cluster, in rank order.  Two CTAs are on an SM: where their number is no
// multiple of the SMs', memory serves all of them alike and they still end together, and one's start and end are the other's
// loads.  1 x 4096 x 4096 takes 6.8 us from memory (its bytes 2.5, the launch, the first loads' way and the join the rest) and 5.8
// where L2 has W, 37 x 4096 x 14336 16.2 (8.8) and 64 x 28672 x 4096 23.9 (17.9).  (Equal shares of all tiles' blocks, one persistent CTA an SM, joined through the workspace: 64 x 28672 x
// 4096 32.5 us, 64 x 4096 x 4096 19.8, most of it joins.)
//  * The weight rows are the MMA's M (TMEM lanes), the rows of x its N: a lane's accumulators then belong to
//    one weight row and BT rows of x, and 32 lanes write 32 neighbours of a row of y.
//  * Warp 0: one lane brings each unit's W and X tiles by TMA into a ring of stages (rows and columns past the
//    ends read as zeros).  Warp 1: one lane issues the unit's four MMAs into its part of a set of accumulators in
//    tensor memory.  Warps 2..5: scales and sums.
//  * Every wait is bounded; one that gives up sets the error word, and the CTA waits for its own copies and MMAs and
//    frees its TMEM before it returns.
#pragma once
#include <cuda.h>

#include <cstdint>
#include <type_traits>

#include "../../include/qgemv.h"
#include "qgemv_elems.cuh"
#include "qgemv_mma.cuh"
#include "qgemv_ptx.cuh"
#include "qgemv_tcgen05.cuh"

namespace qg {

constexpr int kScaledRows = 128;   // weight rows of a tile: one row of w_scale
constexpr int kScaledBlock = 128;  // bytes of K in a block: one 128-byte swizzle row
constexpr uint64_t kDrainNs = 1000000000ull;  // for a CTA's own copies and MMAs, whatever the handle's limit

struct ScaledArgs {
  const float* xs;
  const float* ws;
  void* y;
  int64_t xs_stride, y_stride;
  int M, N, blocks;
  int x_tiles;    // many rows
  int ks;         // CTAs (many rows: pairs) of a cluster, which share a tile's blocks
  int out;
  int* err;
  uint64_t spin_ns;
  int wide;       // the scales of four blocks are 16 aligned bytes
  int early;      // W may be read before the kernel before this one ends
  int stall;      // test hook: the first CTA withholds its first set of sums
};

__host__ __device__ constexpr int few_halves(int BT) { return BT > 32 ? 2 : 1; }  // column halves, four warps each
__host__ __device__ constexpr int few_threads(int BT) { return 32 * (2 + 4 * few_halves(BT)); }
__host__ __device__ constexpr int few_stage_bytes(int BT) { return kScaledBlock * (kScaledRows + BT); }
__host__ __device__ constexpr int few_stages(int BT) { return 108 * 1024 / few_stage_bytes(BT); }
// Blocks whose sums are handed over together (their barriers and scales are met once): two such sets fill half of tensor
// memory, or a quarter at BT = 16.
__host__ __device__ constexpr int few_set(int BT) { return BT > 32 ? 2 : 4; }
__host__ __device__ constexpr int few_tmem_cols(int BT) { return 2 * few_set(BT) * BT; }
__host__ __device__ constexpr int few_scale_bytes(int BT) { return 2 * 3 * few_set(BT) * BT * 4; }  // two sets: products, x's and W's
__host__ __device__ constexpr size_t few_smem_bytes(int BT) {
  return 1024 + static_cast<size_t>(few_stages(BT)) * few_stage_bytes(BT) + 256 + few_scale_bytes(BT);
}

__device__ __forceinline__ void copy4(uint32_t dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy4_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bar_part(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

__device__ __forceinline__ void scaled_store(void* y, int64_t at, int type, float v) {
  if (type == QGEMV_OUT_F32)
    static_cast<float*>(y)[at] = v;
  else if (type == QGEMV_OUT_F16)
    static_cast<__half*>(y)[at] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void store_remote_u32(uint32_t cluster_at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_at), "r"(v) : "memory");
}
__device__ __forceinline__ void store_remote_u64(uint32_t cluster_at, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cluster_at), "l"(v) : "memory");
}
__device__ __forceinline__ int64_t lds_u64(uint32_t at) {
  int64_t v;
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void scaled_cluster_meet() {
  __syncwarp();  // .aligned: whole warps, whatever their lanes did before
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float remote_f32(uint32_t at, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

template <int BT>
__global__ void __launch_bounds__(few_threads(BT), 2) scaled_few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                                                                        const __grid_constant__ ScaledArgs a) {
  constexpr int S = few_stages(BT), Q = few_set(BT), STAGE = few_stage_bytes(BT), WBYTES = kScaledRows * kScaledBlock;
  constexpr int H = few_halves(BT), HB = BT / H, EPI = 128 * H;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + S * STAGE;
  auto full = [&](int s) { return bars + 8u * s; };             // the stage's copies have landed
  auto empty = [&](int s) { return bars + 8u * (S + s); };      // the MMAs that read it are complete
  auto tfull = [&](int b) { return bars + 8u * (2 * S + b); };  // a set's sums are in TMEM
  auto tempty = [&](int b) { return bars + 8u * (2 * S + 2 + b); };  // and have been read
  const uint32_t done = bars + 8u * (2 * S + 4), tslot = done + 8;
  static_assert(8 * (2 * S + 4) + 8 + 8 <= 256, "barriers");
  static_assert(BT * kScaledRows * 4 <= S * STAGE, "a tile's sums take the place of the stages");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned ks = static_cast<unsigned>(a.ks), rank = blockIdx.x % ks, tile = blockIdx.x / ks;
  const int wt = static_cast<int>(tile), rows = a.M;
  const int kb0 = static_cast<int>(static_cast<int64_t>(a.blocks) * rank / ks), n = static_cast<int>(static_cast<int64_t>(a.blocks) * (rank + 1) / ks) - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int b = 0; b < 2; ++b) mbar_init(tfull(b), 1), mbar_init(tempty(b), 4 * H);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tslot, few_tmem_cols(BT));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds_u32(tslot);
  bool ok = true;
  pdl_launch_dependents();

  // The copying and the issuing warp go through their loops as a whole and let one lane do the work: what is the same for all
  // lanes then stays in uniform registers.  Each lane gives up by its own clock; all of them meet at elect.sync, and what the elected
  // one (always the same) has seen decides.  A warp that gave up signals nobody from then on: a stage is freed, and its barrier armed
  // again, only when its copies have landed and the MMAs that read them are complete.  Those that wait for it give up in turn.
  // (With a vote after every wait the many rows' kernel below takes 4 to 11 % longer.)
  if (warp == 0) {  // ---- copies
    const int ahead = a.early ? min(S, n) : 0;
    for (int j = 0; j < ahead; ++j) {
      if (elect_one()) {
        mbar_arrive_expect_tx(full(j), STAGE);
        tma_load_2d(base + j * STAGE, &wmap, (kb0 + j) * kScaledBlock, wt * kScaledRows, full(j));
      }
    }
    pdl_wait();
    int s = 0, issued = 0;
    uint32_t ph = 1;
    for (int i = 0; i < n; ++i) {
      if (ok && i >= S) ok = mbar_wait_bounded(empty(s), ph, a.spin_ns);
      if (elect_one() && ok) {
        issued = i + 1;
        if (i >= ahead) {
          mbar_arrive_expect_tx(full(s), STAGE);
          tma_load_2d(base + s * STAGE, &wmap, (kb0 + i) * kScaledBlock, wt * kScaledRows, full(s));
        }
        tma_load_2d(base + s * STAGE + WBYTES, &xmap, (kb0 + i) * kScaledBlock, 0, full(s));
      }
      if (++s == S) s = 0, ph ^= 1;
    }
    // what was issued last has landed before the CTA may leave
    for (int j = max(issued - S, 0); j < issued; ++j)
      if (!mbar_wait_bounded(full(j % S), static_cast<uint32_t>(j / S) & 1, kDrainNs)) ok = false;
  } else if (warp == 1) {  // ---- MMAs
    constexpr uint32_t idesc = tc_idesc_e4m3(kScaledRows, BT);
    const uint64_t d0 = tc_desc_sw128(base);
    pdl_wait();  // the copies do, and the time until then is not theirs
    int s = 0, b = 0;
    uint32_t ph = 0, tph = 1;
    for (int i = 0; i < n; i += Q) {
      if (ok && i >= 2 * Q) ok = mbar_wait_bounded(tempty(b), tph, a.spin_ns);
      for (int q = 0; q < Q && i + q < n; ++q) {
        if (ok) ok = mbar_wait_bounded(full(s), ph, a.spin_ns);
        tc_fence_after();
        const uint64_t wd = d0 + static_cast<uint64_t>(s * (STAGE / 16)), xd = wd + WBYTES / 16;
        if (elect_one() && ok) {
#pragma unroll
          for (int k = 0; k < kScaledBlock / 32; ++k) tc_mma_f8(tmem + (b * Q + q) * BT, wd + 2 * k, xd + 2 * k, idesc, k > 0);
          tc_commit(empty(s));
        }
        if (++s == S) s = 0, ph ^= 1;
      }
      if (elect_one() && ok && !(a.stall && blockIdx.x == 0 && i == 0)) tc_commit(tfull(b));
      if ((b ^= 1) == 0) tph ^= 1;
    }
    if (elect_one()) tc_commit(done);  // nobody leaves, or writes over the stages, while MMAs run
  } else {
    // ---- scales and sums: this thread's weight row is its TMEM lane, its columns are half hh of x's rows
    const int q4 = warp & 3, hh = (warp - 2) >> 2, r = 32 * q4 + lane, tid = threadIdx.x - 64;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q4) << 16) + hh * HB;
    constexpr int P = Q * BT;  // scales of a set: of block q and row c of x at q BT + c
    const uint32_t prod = bars + 256, raw = prod + 2 * P * 4;
    pdl_wait();
    // x's and W's scales of the set from block i on, copied a set ahead; each thread has its own of the P
    auto fetch = [&](int i, int p) {
#pragma unroll
      for (int e = tid; e < P; e += EPI) {
        const int q = e / BT, m = e % BT;
        if (i + q < n && m < rows) {
          copy4(raw + (2 * p * P + e) * 4, a.xs + m * a.xs_stride + kb0 + i + q);
          copy4(raw + ((2 * p + 1) * P + e) * 4, a.ws + static_cast<int64_t>(wt) * a.blocks + kb0 + i + q);
        }
      }
      copy4_commit();
    };
    // their products (of rows past the end, too: those have zeros in x, and whatever their scales are, nobody stores their sums)
    auto keep = [&](int p) {
      copy4_wait<0>();
#pragma unroll
      for (int e = tid; e < P; e += EPI)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(prod + (p * P + e) * 4),
                     "f"(__uint_as_float(lds_u32(raw + (2 * p * P + e) * 4)) * __uint_as_float(lds_u32(raw + ((2 * p + 1) * P + e) * 4))) : "memory");
    };
    fetch(0, 0);
    float acc[HB];
#pragma unroll
    for (int c = 0; c < HB; ++c) acc[c] = 0.f;
    int b = 0;
    uint32_t tph = 0;
    for (int i = 0; i < n;) {
      const int nq = min(Q, n - i);
      keep(b);
      fetch(i + nq, b ^ 1);
      bar_part(1, EPI);  // the products
      // a warp that gave up goes on, so that the others do not miss it at their barriers
      if (ok && !mbar_wait_bounded(tfull(b), tph, a.spin_ns)) ok = false;
      __syncwarp();
      tc_fence_after();
      constexpr int CH = 16, NC = HB / CH;
      uint32_t d[2][CH];
      auto load = [&](int q, int c, uint32_t (&v)[CH]) { tmem_ld16(lanes + (b * Q + q) * BT + c, v); };
      load(0, 0, d[0]);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        if (q < nq) {
#pragma unroll
          for (int k = 0; k < NC; ++k) {
            uint32_t(&v)[CH] = d[(q * NC + k) & 1];
            tmem_ld_arrived(v);
            // the next columns are on their way while these are added
            if (k + 1 < NC)
              load(q, (k + 1) * CH, d[(q * NC + k + 1) & 1]);
            else if (q + 1 < Q && q + 1 < nq)
              load(q + 1, 0, d[(q * NC + k + 1) & 1]);
#pragma unroll
            for (int j = 0; j < CH; j += 4) {
              const uint4 f = lds_v4(prod + (b * P + q * BT + hh * HB + k * CH + j) * 4);
              float* to = acc + k * CH + j;
              to[0] = fmaf(__uint_as_float(v[j]), __uint_as_float(f.x), to[0]);
              to[1] = fmaf(__uint_as_float(v[j + 1]), __uint_as_float(f.y), to[1]);
              to[2] = fmaf(__uint_as_float(v[j + 2]), __uint_as_float(f.z), to[2]);
              to[3] = fmaf(__uint_as_float(v[j + 3]), __uint_as_float(f.w), to[3]);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(tempty(b));
      if ((b ^= 1) == 0) tph ^= 1;
      i += nq;
    }
    if (ks == 1) {
      const int64_t col = static_cast<int64_t>(wt) * kScaledRows + r;
      if (col < a.N) {
#pragma unroll
        for (int c = 0; c < HB; ++c)
          if (hh * HB + c < rows) scaled_store(a.y, static_cast<int64_t>(hh * HB + c) * a.y_stride + col, a.out, acc[c]);
      }
    } else {
      // the MMAs have read the stages: this CTA's sums take their place, [row of x][weight row]
      if (!mbar_wait_bounded(done, 0, kDrainNs)) ok = false;
#pragma unroll
      for (int c = 0; c < HB; ++c)
        if (hh * HB + c < rows)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((hh * HB + c) * kScaledRows + r) * 4), "f"(acc[c]) : "memory");
    }
  }
  __syncwarp();
  if (warp < 2 && !mbar_wait_bounded(done, 0, kDrainNs)) ok = false;
  if (ks > 1) {
    scaled_cluster_meet();
    // this CTA's share of the tile's rows x 128 sums, over the ranks in their order
    const int all = rows * kScaledRows;
    const int e1 = static_cast<int>(static_cast<unsigned>(all) * (rank + 1) / ks);
    for (int e = static_cast<int>(static_cast<unsigned>(all) * rank / ks) + static_cast<int>(threadIdx.x); e < e1; e += few_threads(BT)) {
      float v[8];
#pragma unroll
      for (unsigned q = 0; q < 8; ++q) v[q] = q < ks ? remote_f32(base + e * 4, q) : 0.f;
      float sum = v[0];
#pragma unroll
      for (int q = 1; q < 8; ++q) sum += v[q];
      const int64_t col = static_cast<int64_t>(wt) * kScaledRows + e % kScaledRows;
      if (col < a.N) scaled_store(a.y, static_cast<int64_t>(e / kScaledRows) * a.y_stride + col, a.out, sum);
    }
    scaled_cluster_meet();  // nobody leaves while its sums are read
  }
  if (!ok) atomicOr(a.err, kDevErrTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, few_tmem_cols(BT));
  }
}

// ---------------------------------------------------------------------------- many rows
// From 65 rows of x on, what bounds the projection is the matrix instructions, or until some hundred rows still W's bytes.  A
// pair of CTAs (cta_group::2) has a tile of 256 rows of x x BN weight rows: here x is the MMA's M, so that a
// lane's accumulators belong to one row of x and a single factor xs * ws scales all of a thread's columns of a
// block.  Each CTA loads its 128 rows of x and half of the weight rows, which halves what its shared memory takes in for
// W (a CTA alone would need 96 bytes a cycle for the operands and 96 for the copies, of 128).  One persistent pair on
// every two SMs, tiles of x first, so that the weights that are being read are shared by all of x.  Eight warps
// scale and add, a half of the columns each, and write through shared memory, whole rows' pieces at a time.
// 4096 x 28672 x 4096 takes 382 us in calls one after another (360 while the card is cool; 249 at the rate for 8 bits), 4096 x 4096 x
// 14336 200.  A block of a 256 x 256 tile takes 737
// cycles, its instructions 512: the sums come out of tensor memory in 16 turns of 16 columns, each met by its additions; the other
// pairs' loads add 15 %, and the end of a tile 3500 cycles that no instruction of the next covers, for want of registers.  What all
// SMs take in, 48 bytes a cycle each, is near what the L2 gives.
// Where tiles are few, up to four pairs, a cluster, share a tile's blocks and join their sums (128 x 4096 x 14336: 21.0 us, 33.2
// with a pair to a tile).  Sums of 128 columns are read ahead and added two to an instruction (32.8 us of 36.6 in that case with a
// pair to a tile); of 256 that is slower (350 us to 357 of the large one), as registers are then short.
constexpr int kManyParts = 2;  // warpgroups of sums, each with a part of the columns
constexpr int kManyThreads = 128 * (1 + kManyParts);
constexpr int kManyRegs[2] = {88, 208};  // of the first warpgroup and the others: together what the block is launched with, 3 x 168
constexpr int kManyChunk = 16;  // columns that are read at a time
constexpr int kManyRows = 256;  // rows of x of a tile

constexpr int kManyMaxPairs = 4;  // of a cluster

__host__ __device__ constexpr int many_stage_bytes(int BN) { return kScaledBlock * (kManyRows / 2 + BN / 2); }
__host__ __device__ constexpr int many_stages(int BN) { return 176 * 1024 / many_stage_bytes(BN); }
constexpr int kManyPad = 64 / kManyParts + 4;  // so that 16-byte accesses meet no bank twice
constexpr int kManyWords = 64 / kManyParts;  // of a row that a warp stages at a time
constexpr int kManyOutBytes = 4 * kManyParts * 32 * kManyPad * 4;
constexpr int kManyScaleBytes = 8 * 128 * 4;  // products of the scales of 128 rows of x and one of W, or two, of eight blocks or four
__host__ __device__ constexpr size_t many_smem_bytes(int BN) {
  return 1024 + static_cast<size_t>(many_stages(BN)) * many_stage_bytes(BN) + 256 + kManyOutBytes + kManyScaleBytes;
}

// a0 += d0 f, a1 += d1 f in one instruction.
__device__ __forceinline__ void fma_pair(float& a0, float& a1, uint32_t d0, uint32_t d1, float f) {
  asm("{\n\t.reg .b64 a, d, q;\n\t"
      "mov.b64 a, {%0, %1};\n\tmov.b64 d, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\t"
      "fma.rn.f32x2 a, d, q, a;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(a0), "+f"(a1)
      : "r"(d0), "r"(d1), "f"(f));
}
__device__ __forceinline__ float4 remote_v4(uint32_t at, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_address(at, rank)) : "memory");
  return v;
}

template <int BN, bool JOIN>  // JOIN: ks > 1
__global__ void __launch_bounds__(kManyThreads, 1) scaled_many_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                                                                      const __grid_constant__ ScaledArgs a) {
  constexpr bool kAhead = BN == 128;
  constexpr int NB = 512 / BN, SLOTS = 2 * NB, SLOT = BN / kScaledRows * 128 * 4;  // sets of sums that fill tensor memory; slots of products
  constexpr int S = many_stages(BN), kJoinPad = BN + 4, STAGE = many_stage_bytes(BN), XBYTES = kScaledBlock * kManyRows / 2, HB = BN / kManyParts;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + S * STAGE;
  auto full = [&](int s) { return bars + 8u * s; };             // of the pair's first CTA: both CTAs' copies have landed
  auto empty = [&](int s) { return bars + 8u * (S + s); };      // the MMAs that read the stage are complete
  auto tfull = [&](int b) { return bars + 8u * (2 * S + b); };  // a block's sums are in TMEM and its scales' products in shared memory
  auto tempty = [&](int b) { return bars + 8u * (2 * S + NB + b); };  // of the first CTA: both CTAs have read them
  const uint32_t done = bars + 8u * (2 * S + 2 * NB), tslot = done + 8, failed = tslot + 4;  // failed: a CTA of the cluster gave up
  auto copied = [&](unsigned r) { return done + 16 + 8u * r; };  // of the pair's first CTA: the stages that CTA r has asked for
  static_assert(SLOTS * SLOT <= kManyScaleBytes && 8 * (2 * S + 2 * NB) + 32 <= 256, "barriers");
  static_assert(kManyRows / 2 * kJoinPad * 4 <= S * STAGE, "a tile's sums take the place of the stages");
  const uint32_t prod = bars + 256 + kManyOutBytes;  // [block % SLOTS][128 rows of W][row of x]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // JOIN: a cluster has one tile, and pair kp of it the blocks kb0 .. kb1 (whole fours, as their scales are read)
  const unsigned ks = JOIN ? static_cast<unsigned>(a.ks) : 1u, rank = blockIdx.x & 1, kp = JOIN ? (blockIdx.x >> 1) % ks : 0, lead = 2 * kp;
  const unsigned pair = (blockIdx.x >> 1) / ks, pairs = (gridDim.x >> 1) / ks;
  const int fours = (a.blocks + 3) / 4;
  const int kb0 = JOIN ? static_cast<int>(static_cast<unsigned>(fours) * kp / ks) * 4 : 0;
  const int kb1 = JOIN ? min(a.blocks, static_cast<int>(static_cast<unsigned>(fours) * (kp + 1) / ks) * 4) : a.blocks;
  const unsigned x_tiles = static_cast<unsigned>(a.x_tiles), tiles = x_tiles * ((static_cast<unsigned>(a.N) + BN - 1) / BN);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int b = 0; b < NB; ++b) mbar_init(tfull(b), 3), mbar_init(tempty(b), 2 * 4 * kManyParts);
    mbar_init(done, 1);
    fence_mbar_init();
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(failed), "r"(0) : "memory");
  }
  if (warp == 1) {
    tmem_alloc_pair(tslot, NB * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  scaled_cluster_meet();  // both CTAs' barriers are ready
  tc_fence_after();
  const uint32_t tmem = lds_u32(tslot);
  bool ok = true;
  pdl_launch_dependents();
  pdl_wait();

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kManyRegs[0]));
  if (warp == 0) {  // ---- copies (whole warps go through the loops and signal nobody once they gave up, as above)
    int s = 0;
    uint32_t ph = 1;
    bool filled = false;  // every stage has been used
    int64_t asked = 0;  // in the elected lane
    for (unsigned t = pair; t < tiles; t += pairs) {
      const int m = static_cast<int>(t % x_tiles * kManyRows + rank * (kManyRows / 2)), n = static_cast<int>(t / x_tiles * BN + rank * (BN / 2));
      for (int kb = kb0; kb < kb1; ++kb) {
        if (ok && filled) ok = mbar_wait_bounded(empty(s), ph, a.spin_ns);
        const uint32_t bar = cluster_address(full(s), lead);
        if (elect_one() && ok) {
          ++asked;
          if (rank == 0) mbar_arrive_expect_tx(full(s), 2 * STAGE);
          tma_load_2d_pair(base + s * STAGE, &xmap, kb * kScaledBlock, m, bar);
          tma_load_2d_pair(base + s * STAGE + XBYTES, &wmap, kb * kScaledBlock, n, bar);
        }
        if (++s == S) s = 0, ph ^= 1, filled = true;
      }
    }
    if (elect_one()) store_remote_u64(cluster_address(copied(rank), lead), static_cast<uint64_t>(asked));
  } else if (warp == 1) {
    if (rank == 0) {  // ---- MMAs
      constexpr uint32_t idesc = tc_idesc_e4m3(kManyRows, BN);
      const uint64_t d0 = tc_desc_sw128(base);
      int s = 0, b = 0;
      uint32_t ph = 0, tph = 1;
      bool used = false;     // all sets have been
      bool is_full = false;  // asked while the block before is being issued
      for (unsigned t = pair; t < tiles; t += pairs) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (ok && used) ok = mbar_wait_bounded(tempty(b), tph, a.spin_ns);
          if (ok && !is_full) ok = mbar_wait_bounded(full(s), ph, a.spin_ns);
          tc_fence_after();
          const uint64_t xd = d0 + static_cast<uint64_t>(s * (STAGE / 16)), wd = xd + XBYTES / 16;
          if (elect_one() && ok) {
#pragma unroll
            for (int k = 0; k < kScaledBlock / 32; ++k) tc_mma_f8_pair(tmem + b * BN, xd + 2 * k, wd + 2 * k, idesc, k > 0);
            if (!(a.stall && blockIdx.x == 0 && t == pair && kb == kb0)) tc_commit_pair(tfull(b), lead);
          }
          if (++s == S) s = 0, ph ^= 1;
          if (++b == NB) b = 0, tph ^= 1, used = true;
          is_full = mbar_test(full(s), ph);
        }
      }
      if (elect_one()) tc_commit_pair(done, lead);  // nobody leaves while MMAs run
    }
  } else if (warp < 4) {
    // ---- products of scales: two rows of x a lane.  The scales of four blocks are read while the four before them are used (rows
    // and columns past the end have none: nobody stores their sums)
    constexpr int WB = BN / kScaledRows;
    const unsigned r = (warp - 2) * 32 + lane;  // and 64 rows further
    struct Four {
      float x[2][4], w[WB][4];
    };
    auto fetch = [&](unsigned t, int kb) {
      Four v;
      const int64_t row = static_cast<int64_t>(t % x_tiles) * kManyRows + rank * (kManyRows / 2) + r, wrow = static_cast<int64_t>(t / x_tiles) * WB;
      auto four = [&](const float* at, bool in, float (&f)[4]) {
        if (a.wide) {
          const float4 q = in ? *reinterpret_cast<const float4*>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
          f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) f[q] = in && kb + q < kb1 ? at[q] : 0.f;
        }
      };
#pragma unroll
      for (int j = 0; j < 2; ++j) four(a.xs + (row + 64 * j) * a.xs_stride + kb, t < tiles && row + 64 * j < a.M, v.x[j]);
#pragma unroll
      for (int j = 0; j < WB; ++j) four(a.ws + (wrow + j) * a.blocks + kb, t < tiles && (wrow + j) * kScaledRows < a.N, v.w[j]);
      return v;
    };
    // The products of a block go out when the sums of the one before it in the same place are known to be there: its MMAs began
    // when the sums of the block before that, and with them the products, had been read.
    int b = 0, slot = 0;
    uint32_t ph = 1;
    bool used = false;
    Four next = fetch(pair, kb0);
    for (unsigned t = pair; t < tiles; t += pairs) {
      for (int kb = kb0; kb < kb1; kb += 4) {
        const Four now = next;
        const bool last = kb + 4 >= kb1;
        next = fetch(last ? t + pairs : t, last ? kb0 : kb + 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (kb + q >= kb1) break;
          if (ok && used) ok = mbar_wait_bounded(tfull(b), ph, a.spin_ns);
          const uint32_t to = prod + slot * SLOT + r * 4;
          slot = (slot + 1) % SLOTS;
#pragma unroll
          for (int w = 0; w < WB; ++w)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + (w * 128 + j * 64) * 4), "f"(now.x[j][q] * now.w[w][q]) : "memory");
          __syncwarp();
          if (elect_one() && ok) mbar_arrive(tfull(b));
          if (++b == NB) b = 0, ph ^= 1, used = true;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs[1]));
    // ---- scales and sums: this thread's row of x is its TMEM lane, its columns are part hh of the weight rows
    const int q4 = warp & 3, hh = (warp - 4) >> 2, r = 32 * q4 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q4) << 16) + hh * HB;
    const uint32_t out = bars + 256 + (warp - 4) * (32 * kManyPad * 4);
    const uint32_t mine_f = prod + ((hh * HB) / kScaledRows * 128 + r) * 4;
    const uint32_t tempty_at = cluster_address(tempty(0), lead);  // of the next set 8 bytes behind
    float acc[HB];
    int b = 0, s = 0, slot = 0;
    uint32_t tph = 0;
    for (unsigned t = pair; t < tiles; t += pairs) {
#pragma unroll
      for (int c = 0; c < HB; ++c) acc[c] = 0.f;
#pragma unroll 1
      for (int kb = kb0; kb < kb1; ++kb) {
        if (ok) ok = mbar_wait_bounded(tfull(b), tph, a.spin_ns);
        __syncwarp();
        tc_fence_after();
        const uint32_t from = lanes + b * BN;
        const float f = __uint_as_float(lds_u32(mine_f + slot * SLOT));
        slot = (slot + 1) % SLOTS;
        constexpr int CH = kManyChunk, NC = HB / CH;
        uint32_t d[kAhead ? 2 : 1][CH];
        if (kAhead) tmem_ld16(from, d[0]);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
          uint32_t(&v)[CH] = d[kAhead ? k & 1 : 0];
          if constexpr (kAhead) {
            tmem_ld_arrived(v);
            if (k + 1 < NC) tmem_ld16(from + (k + 1) * CH, d[(k + 1) & 1]);
          } else {
            tmem_ld_now(from + k * CH, v);
          }
          if (k + 1 == NC) {
            tc_fence_before();
            __syncwarp();
            if (elect_one() && ok) {
              mbar_arrive_remote(tempty_at + 8u * b);
              if (warp == 4) mbar_arrive(empty(s));  // the block's MMAs are complete, and so are their reads of its stage
            }
            if (++s == S) s = 0;
          }
#pragma unroll
          for (int j = 0; j < CH; j += 2) {
            if constexpr (kAhead) {
              fma_pair(acc[k * CH + j], acc[k * CH + j + 1], v[j], v[j + 1], f);
            } else {
              acc[k * CH + j] = fmaf(__uint_as_float(v[j]), f, acc[k * CH + j]);
              acc[k * CH + j + 1] = fmaf(__uint_as_float(v[j + 1]), f, acc[k * CH + j + 1]);
            }
          }
        }
        if (++b == NB) b = 0, tph ^= 1;
      }
      // ---- the tile: 32 rows x kManyWords words at a time through shared memory, then a row's words by neighbouring lanes, four
      // each where rows of y are whole 16 bytes apart
      const int64_t row0 = static_cast<int64_t>(t % x_tiles) * kManyRows + rank * (kManyRows / 2) + 32 * q4, col0 = static_cast<int64_t>(t / x_tiles) * BN + hh * HB;
      const int cols = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(HB), a.N - col0)));
      const int rows = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(32), a.M - row0)));
      if constexpr (JOIN) {
        // the blocks' stages have been read: these sums take their place, and each pair adds its share of the tile's rows, over the
        // pairs in their order, four columns a thread
#pragma unroll
        for (int c = 0; c < HB; c += 4)
          if (lane < rows)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(base + (r * kJoinPad + hh * HB + c) * 4), "f"(acc[c]), "f"(acc[c + 1]), "f"(acc[c + 2]),
                         "f"(acc[c + 3])
                         : "memory");
        scaled_cluster_meet();
        const int64_t m0 = static_cast<int64_t>(t % x_tiles) * kManyRows + rank * (kManyRows / 2), n0 = static_cast<int64_t>(t / x_tiles) * BN;
        const int all = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kManyRows / 2), a.M - m0))) * (BN / 4);
        const int e1 = static_cast<int>(static_cast<unsigned>(all) * (kp + 1) / ks);
        constexpr int kStep = 128 * kManyParts, U = 2;  // U pieces' reads are in flight together
        for (int e0 = static_cast<int>(static_cast<unsigned>(all) * kp / ks) + static_cast<int>(threadIdx.x) - 128; e0 < e1; e0 += U * kStep) {
          float4 v[U][kManyMaxPairs];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int e = min(e0 + u * kStep, e1 - 1);
#pragma unroll
            for (unsigned q = 0; q < kManyMaxPairs; ++q)
              v[u][q] = q < ks ? remote_v4(base + (e / (BN / 4) * kJoinPad + e % (BN / 4) * 4) * 4, 2 * q + rank) : make_float4(0.f, 0.f, 0.f, 0.f);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int e = e0 + u * kStep, row = e / (BN / 4), c = e % (BN / 4) * 4;
            if (e >= e1) break;
            float4 sum = v[u][0];
#pragma unroll
            for (int q = 1; q < kManyMaxPairs; ++q) sum.x += v[u][q].x, sum.y += v[u][q].y, sum.z += v[u][q].z, sum.w += v[u][q].w;
            const int64_t to = (m0 + row) * a.y_stride + n0 + c;
            const float f4[4] = {sum.x, sum.y, sum.z, sum.w};
            if (a.y_stride % 4 == 0 && n0 + c + 4 <= a.N) {
              if (a.out == QGEMV_OUT_F32) {
                *reinterpret_cast<float4*>(static_cast<float*>(a.y) + to) = sum;
              } else {
                const bool bf = a.out == QGEMV_OUT_BF16;
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + to) =
                    make_uint2(bf ? pair16<true>(f4[0], f4[1]) : pair16<false>(f4[0], f4[1]), bf ? pair16<true>(f4[2], f4[3]) : pair16<false>(f4[2], f4[3]));
              }
            } else {
              for (int j = 0; j < 4; ++j)
                if (n0 + c + j < a.N) scaled_store(a.y, to + j, a.out, f4[j]);
            }
          }
        }
        break;
      }
      auto flush = [&](int c, int n) {  // columns c .. of this part, n of them in a word
        constexpr int L = kManyWords / 4;  // lanes of a row
        __syncwarp();
        if (a.y_stride % (4 * n) == 0 && c + kManyWords * n <= cols) {
          const int64_t to = (row0 + lane / L) * a.y_stride + col0 + c + 4 * n * (lane % L);
          uint8_t* y = static_cast<uint8_t*>(a.y) + to * (4 / n);
#pragma unroll
          for (int i = 0; i < L; ++i) {
            const int row = 32 / L * i + lane / L;
            const uint4 w = lds_v4(out + (row * kManyPad + 4 * (lane % L)) * 4);
            if (row < rows) *reinterpret_cast<uint4*>(y) = w;
            y += 32 / L * a.y_stride * (4 / n);
          }
        } else {
          const int at = c + n * (lane % kManyWords);
          for (int i = lane / kManyWords; i < rows; i += 32 / kManyWords) {
            const uint32_t w = lds_u32(out + (i * kManyPad + lane % kManyWords) * 4);
            const int64_t to = (row0 + i) * a.y_stride + col0 + at;
            if (n == 1) {
              if (at < cols) static_cast<uint32_t*>(a.y)[to] = w;
            } else {
              if (at < cols) static_cast<uint16_t*>(a.y)[to] = static_cast<uint16_t>(w);
              if (at + 1 < cols) static_cast<uint16_t*>(a.y)[to + 1] = static_cast<uint16_t>(w >> 16);
            }
          }
        }
        __syncwarp();
      };
      const uint32_t mine = out + lane * (kManyPad * 4);
      auto put = [&](int j, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(mine + j * 4), "r"(w0), "r"(w1), "r"(w2), "r"(w3) : "memory");
      };
      auto put_pairs = [&](auto bf) {
#pragma unroll
        for (int c = 0; c < HB; c += 2 * kManyWords) {
#pragma unroll
          for (int j = 0; j < kManyWords; j += 4) {
            const float* v = acc + c + 2 * j;
            put(j, pair16<bf.value>(v[0], v[1]), pair16<bf.value>(v[2], v[3]), pair16<bf.value>(v[4], v[5]), pair16<bf.value>(v[6], v[7]));
          }
          flush(c, 2);
        }
      };
      if (a.out == QGEMV_OUT_BF16) {
        put_pairs(std::true_type{});
      } else if (a.out == QGEMV_OUT_F16) {
        put_pairs(std::false_type{});
      } else {
#pragma unroll
        for (int c = 0; c < HB; c += kManyWords) {
#pragma unroll
          for (int j = 0; j < kManyWords; j += 4) {
            const float* v = acc + c + j;
            put(j, __float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
          }
          flush(c, 1);
        }
      }
    }
  }
  if (JOIN && warp < 4) scaled_cluster_meet();  // with the sums' threads
  if (!mbar_wait_bounded(done, 0, kDrainNs)) ok = false;
  if (!ok) {
    atomicOr(a.err, kDevErrTimeout);
    for (unsigned q = 0; q < 2 * ks; ++q) store_remote_u32(cluster_address(failed, q), 1);
  }
  tc_fence_before();
  __syncthreads();
  scaled_cluster_meet();  // nobody leaves while the other CTA's arrivals are on their way
  if (lds_u32(failed)) {
    // What was copied for no MMA has landed before a CTA may leave.  Both CTAs' copies are counted at the first one's barriers, where
    // a stage is asked for again only after it was read: of each CTA the last S may be on their way, and the CTAs are no more than S
    // apart.
    if (warp == 0 && rank == 0) {
      const int64_t c0 = lds_u64(copied(0)), c1 = lds_u64(copied(1)), most = max(c0, c1);
      for (int64_t j = max(most - S, int64_t{0}); j < most; ++j) {
        const uint32_t bar = full(static_cast<int>(j % S));
        if (lane == 0 && j >= c0) mbar_arrive_expect_tx(bar, STAGE);  // the other's copy alone, of a stage that was not armed
        if (lane == 0 && j >= c1) mbar_complete_tx(bar, STAGE);       // this CTA's alone, of a stage that was armed for both
        if (!mbar_wait_bounded(bar, static_cast<uint32_t>(j / S) & 1, kDrainNs)) break;
      }
    }
    scaled_cluster_meet();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, NB * BN);
  }
}

}  // namespace qg
