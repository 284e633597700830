// Projection of e4m3 rows by e4m3 weights, each with a scale for blocks of 128:
//   y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in b} x[m, k] W[n, k].
//
// A block's inner sums come from the fifth-generation tensor cores (kind::f8f6f4, 32 along K an instruction,
// four to a block) and stay in tensor memory until a warpgroup has added them, times the block's two scales, to
// fp32 accumulators in its registers: the scales change with every block, so the sum over blocks cannot stay in
// tensor memory.
//
// Few rows of x (this kernel): what bounds it is the bytes of W, N K of them, so every SM gets the same share:
// the work is the sequence of (tile of 128 weight rows x BT rows of x, block) units, tile by tile, cut into equal
// ranges, one to a CTA.  A tile that is cut is joined by the last of its CTAs to finish (counted in the
// handle's counters), which adds the parts from the handle's workspace in their order: the result does not
// depend on who is last.
//  * The weight rows are the MMA's M (TMEM lanes), the rows of x its N: a lane's accumulators then belong to
//    one weight row and BT rows of x, and 32 lanes write 32 neighbours of a row of y.
//  * Warp 0: one lane brings each unit's W and X tiles by TMA into a ring of stages (rows and columns past the
//    ends read as zeros).  Warp 1: one lane issues the unit's four MMAs into one of NB accumulators of
//    tensor memory.  Warps 2..5: scales and sums.
//  * Every wait is bounded; one that gives up sets the error word, and the CTA waits for its own copies and MMAs and
//    frees its TMEM before it returns.
#pragma once
#include <cuda.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_elems.cuh"
#include "qgemv_ptx.cuh"
#include "qgemv_tcgen05.cuh"

namespace qg {

constexpr int kScaledRows = 128;   // weight rows of a tile: one row of w_scale
constexpr int kScaledBlock = 128;  // bytes of K in a block: one 128-byte swizzle row
constexpr int kFewThreads = 32 * 6;
constexpr uint64_t kDrainNs = 1000000000ull;  // for a CTA's own copies and MMAs, whatever the handle's limit

struct ScaledArgs {
  const float* xs;
  const float* ws;
  void* y;
  int64_t xs_stride, y_stride;
  int64_t units;  // tiles * blocks
  int M, N, blocks;
  int x_tiles;
  int out;
  float* parts;   // of cut tiles: two slots a CTA
  int* cnt;
  int* err;
  uint64_t spin_ns;
  int early;      // W may be read before the kernel before this one ends
  int stall;      // test hook: the first CTA withholds its first unit's sums
};

__host__ __device__ constexpr int few_stage_bytes(int BT) { return kScaledBlock * (kScaledRows + BT); }
__host__ __device__ constexpr int few_stages(int BT) { return 196 * 1024 / few_stage_bytes(BT); }
__host__ __device__ constexpr int few_buffers(int BT) { return BT > 64 ? 2 : 4; }
__host__ __device__ constexpr int few_tmem_cols(int BT) { return few_buffers(BT) * BT; }  // 64 .. 256
__host__ __device__ constexpr size_t few_smem_bytes(int BT) {
  return 1024 + static_cast<size_t>(few_stages(BT)) * few_stage_bytes(BT) + 256 + 4 * 2 * BT * 4;
}

__device__ __forceinline__ int count_acq_rel(int* p) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
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

// A unit of a CTA's range: tile of weights, tile of x and block; the tiles of x that share a tile of weights follow one another.
struct ScaledUnit {
  int wt, xt, kb;
  __device__ __forceinline__ ScaledUnit(int64_t u, const ScaledArgs& a) {
    const int64_t tile = u / a.blocks;
    kb = static_cast<int>(u - tile * a.blocks);
    wt = static_cast<int>(tile / a.x_tiles);
    xt = static_cast<int>(tile - static_cast<int64_t>(wt) * a.x_tiles);
  }
  __device__ __forceinline__ void next(const ScaledArgs& a) {
    if (++kb == a.blocks) {
      kb = 0;
      if (++xt == a.x_tiles) xt = 0, ++wt;
    }
  }
};

template <int BT>
__global__ void __launch_bounds__(kFewThreads, 1) scaled_few_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                                                                    const __grid_constant__ ScaledArgs a) {
  constexpr int S = few_stages(BT), NB = few_buffers(BT), STAGE = few_stage_bytes(BT), WBYTES = kScaledRows * kScaledBlock;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + S * STAGE;
  auto full = [&](int s) { return bars + 8u * s; };               // the stage's copies have landed
  auto empty = [&](int s) { return bars + 8u * (S + s); };        // the MMAs that read it are complete
  auto tfull = [&](int b) { return bars + 8u * (2 * S + b); };    // a unit's sums are in TMEM
  auto tempty = [&](int b) { return bars + 8u * (2 * S + NB + b); };  // and have been read
  const uint32_t done = bars + 8u * (2 * S + 2 * NB), tslot = done + 8, flag = tslot + 4;
  static_assert(8 * (2 * S + 2 * NB) + 8 + 8 <= 256, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t G = gridDim.x, i0 = blockIdx.x;
  const int64_t u0 = a.units * i0 / G, u1 = a.units * (i0 + 1) / G;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(full(s), 1), mbar_init(empty(s), 1);
    for (int b = 0; b < NB; ++b) mbar_init(tfull(b), 1), mbar_init(tempty(b), 4);
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

  if (warp == 0) {
    if (lane == 0) {  // ---- copies
      ScaledUnit w(u0, a), x(u0, a);
      const int ahead = a.early ? static_cast<int>(min(static_cast<int64_t>(S), u1 - u0)) : 0;
      for (int j = 0; j < ahead; ++j, w.next(a)) {
        mbar_arrive_expect_tx(full(j), STAGE);
        tma_load_2d(base + j * STAGE, &wmap, w.kb * kScaledBlock, w.wt * kScaledRows, full(j));
      }
      pdl_wait();
      int64_t i = 0;
      const int64_t n = u1 - u0;
      int s = 0;
      uint32_t ph = 1;
      for (; i < n; ++i, x.next(a)) {
        if (i >= S && !mbar_wait_bounded(empty(s), ph, a.spin_ns)) {
          ok = false;
          break;
        }
        if (i >= ahead) {
          mbar_arrive_expect_tx(full(s), STAGE);
          tma_load_2d(base + s * STAGE, &wmap, x.kb * kScaledBlock, x.wt * kScaledRows, full(s));
        }
        tma_load_2d(base + s * STAGE + WBYTES, &xmap, x.kb * kScaledBlock, x.xt * BT, full(s));
        if (++s == S) s = 0, ph ^= 1;
      }
      // what was issued last has landed before the CTA may leave
      for (int64_t j = i > S ? i - S : 0; j < i; ++j)
        if (!mbar_wait_bounded(full(static_cast<int>(j % S)), static_cast<uint32_t>(j / S) & 1, kDrainNs)) ok = false;
    }
  } else if (warp == 1) {
    if (lane == 0) {  // ---- MMAs
      constexpr uint32_t idesc = tc_idesc_e4m3(kScaledRows, BT);
      const uint64_t d0 = tc_desc_sw128(base);
      int s = 0, b = 0;
      uint32_t ph = 0, tph = 1;
      const int64_t n = u1 - u0;
      for (int64_t i = 0; i < n; ++i) {
        if ((i >= NB && !mbar_wait_bounded(tempty(b), tph, a.spin_ns)) || !mbar_wait_bounded(full(s), ph, a.spin_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t wd = d0 + static_cast<uint64_t>(s * (STAGE / 16)), xd = wd + WBYTES / 16;
#pragma unroll
        for (int k = 0; k < kScaledBlock / 32; ++k) tc_mma_f8(tmem + b * BT, wd + 2 * k, xd + 2 * k, idesc, k > 0);
        tc_commit(empty(s));
        if (!(a.stall && i0 == 0 && i == 0)) tc_commit(tfull(b));
        if (++s == S) s = 0, ph ^= 1;
        if (++b == NB) b = 0, tph ^= 1;
      }
      tc_commit(done);  // also after a failure: nobody leaves while MMAs run
      if (!mbar_wait_bounded(done, 0, kDrainNs)) ok = false;
    }
  } else {
    // ---- scales and sums: this thread's weight row is its TMEM lane
    const int q4 = warp & 3, r = 32 * q4 + lane;
    const uint32_t my_scales = bars + 256 + q4 * (2 * BT * 4);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * q4) << 16);
    constexpr int V = (BT + 31) / 32;
    pdl_wait();
    float next[V];
    auto fetch = [&](const ScaledUnit& u, bool in) {
      const float w = in ? __ldg(a.ws + static_cast<int64_t>(u.wt) * a.blocks + u.kb) : 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int64_t m = static_cast<int64_t>(u.xt) * BT + lane + 32 * j;
        next[j] = in && lane + 32 * j < BT && m < a.M ? __ldg(a.xs + m * a.xs_stride + u.kb) * w : 0.f;
      }
    };
    auto keep = [&](int p) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (lane + 32 * j < BT) asm volatile("st.shared.f32 [%0], %1;" ::"r"(my_scales + (p * BT + lane + 32 * j) * 4), "f"(next[j]) : "memory");
    };
    ScaledUnit now(u0, a), later(u0, a);
    fetch(later, u0 < u1);
    keep(0);
    later.next(a);
    fetch(later, u0 + 1 < u1);
    float acc[BT];
#pragma unroll
    for (int c = 0; c < BT; ++c) acc[c] = 0.f;
    int64_t first = u0;  // of this tile
    int b = 0, p = 0;
    uint32_t tph = 0;
    for (int64_t u = u0; u < u1; ++u) {
      __syncwarp();
      // a warp that gave up goes on without waiting, so that the others do not miss it at their barriers
      if (ok && !mbar_wait_bounded(tfull(b), tph, a.spin_ns)) ok = false;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < BT; c += 16) {
        uint32_t d[16];
        tmem_ld16(lanes + b * BT + c, d);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const uint4 f = lds_v4(my_scales + (p * BT + c + j) * 4);
          acc[c + j] = fmaf(__uint_as_float(d[j]), __uint_as_float(f.x), acc[c + j]);
          acc[c + j + 1] = fmaf(__uint_as_float(d[j + 1]), __uint_as_float(f.y), acc[c + j + 1]);
          acc[c + j + 2] = fmaf(__uint_as_float(d[j + 2]), __uint_as_float(f.z), acc[c + j + 2]);
          acc[c + j + 3] = fmaf(__uint_as_float(d[j + 3]), __uint_as_float(f.w), acc[c + j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty(b));
      if (++b == NB) b = 0, tph ^= 1;
      p ^= 1;
      keep(p);
      later.next(a);
      fetch(later, u + 2 < u1);
      if (now.kb == a.blocks - 1 || u == u1 - 1) {
        // ---- the tile, or this CTA's part of it
        bool write = true;
        const int64_t t0 = u - now.kb;  // the tile's first unit
        if (first != t0 || now.kb != a.blocks - 1) {
          const int64_t head = ((t0 + 1) * G - 1) / a.units, tail = ((t0 + a.blocks) * G - 1) / a.units;  // CTAs of its first and last unit
          float* mine = a.parts + (2 * i0 + (first == t0)) * (BT * kScaledRows) + r;
#pragma unroll
          for (int c = 0; c < BT; ++c) __stcg(mine + c * kScaledRows, acc[c]);
          bar_part(1, 128);
          if (threadIdx.x == 64) {
            const bool last = count_acq_rel(a.cnt + head) == static_cast<int>(tail - head);
            if (last) a.cnt[head] = 0;
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(flag), "r"(static_cast<uint32_t>(last)) : "memory");
          }
          bar_part(1, 128);
          write = lds_u32(flag) != 0;
          if (write) {
#pragma unroll
            for (int c0 = 0; c0 < BT; c0 += 16) {
#pragma unroll
              for (int c = 0; c < 16; ++c) acc[c0 + c] = 0.f;
              for (int64_t j = head; j <= tail; j += 2) {  // two parts in flight
                const float* one = a.parts + (2 * j + (j == head)) * (BT * kScaledRows) + r;
                const float* two = a.parts + 2 * (j + 1) * (BT * kScaledRows) + r;
                const bool both = j < tail;
                float v[16], w[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                  v[c] = __ldcg(one + (c0 + c) * kScaledRows);
                  w[c] = both ? __ldcg(two + (c0 + c) * kScaledRows) : 0.f;
                }
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[c0 + c] = acc[c0 + c] + v[c] + w[c];
              }
            }
          }
          bar_part(1, 128);  // the flag has been read
        }
        const int64_t n = static_cast<int64_t>(now.wt) * kScaledRows + r;
        if (write && n < a.N) {
          const int64_t m0 = static_cast<int64_t>(now.xt) * BT;
          const int rows = static_cast<int>(min(static_cast<int64_t>(BT), a.M - m0));
#pragma unroll
          for (int c = 0; c < BT; ++c)
            if (c < rows) scaled_store(a.y, (m0 + c) * a.y_stride + n, a.out, acc[c]);
        }
#pragma unroll
        for (int c = 0; c < BT; ++c) acc[c] = 0.f;
        first = u + 1;
      }
      now.next(a);
    }
  }
  if (!ok) atomicOr(a.err, kDevErrTimeout);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, few_tmem_cols(BT));
  }
}

}  // namespace qg
