// Attention of one new token per request over a paged key-value cache.
//
//   s_t = scale q . k_t,   p_t = 2^(s_t log2e - m),   out = sum_t p_t v_t / sum_t p_t
//
// in one pass over the cache with a running maximum m: when it moves, the sum and the output
// are scaled by 2^(m_old - m_new).  Per key-value head the query heads that share it (its group)
// are the rows of one small matrix product, so the cache is read once for all of them.
//
// The kernel is bound by the bytes of the cache, so everything else is arranged around a steady
// stream of copies:
//  * Work.  The cache of a request and key-value head is cut into tiles of TT tokens (4 KB or
//    8 KB of keys).  All tiles of the batch, in the order (request, head, token), are cut into
//    equal contiguous shares, one per CTA and inside it one per warp, whatever the requests'
//    lengths: every CTA sums the lengths itself and finds its share, so nothing is planned on
//    the host and ragged batches keep all SMs busy to the end.
//  * Copies.  Every warp has its own ring of stages, filled by TMA (a tile's pages are rows of a
//    five-dimensional tensor: 128-byte row parts, in-page token, part, head, page) and waited
//    for on an mbarrier.  Page numbers are read by lanes, a batch of tiles ahead of the copies that use them.  No
//    warp waits for another until the end.
//  * Products.  mma.sync m16n8k16: q (rows: query heads) times keys (columns: tokens), then the
//    weights times values.  Memory sets the pace: an SM gets 22 bytes per clock, an 8 KB tile
//    (keys and values of 16 tokens of 128-wide bf16 heads) every 370 clocks.  A warp takes about
//    1300 clocks for one (copying the next 500, scores 260, softmax 290, values 200), so that the
//    eight warps of an SM are through one every 160; of e4m3 codes, whose 8 KB are 32 tokens, in
//    about 2500.  tcgen05 would add a round trip through tensor memory for products of 8 rows.
//    Measured: 32 requests of 24 to 44 thousand tokens, 64 query and 8 key-value heads, bf16:
//    623 us, 6.95 TB/s; 16 requests of 9 to 70 thousand in e4m3: 165 us, 6.2 TB/s; 64 requests of
//    1 to 6000 in bf16: 39.8 us, 4.7 TB/s; one request of 1000 in fp16: 12 us (11.3 in a graph), all latency.
//    Heads of 256 spill registers (54 to 342 bytes a thread): 128 accumulators stand beside the queries.
//  * Precision.  A weight enters the second product as the sum of two 16-bit values: 16 bits of it in
//    bf16, 2^-17 against the output's 2^-9, and 22 in fp16.  fp16's steps end at 2^-24, so there weights, at
//    most 1, are taken times 2^14 and the output divided by it: below 2^-38 of the largest they are rounded
//    away, where they are counted in l (times 1, that was 2^-24: 4000 tokens 17.5 nats below one of value 0 gave 0).
//    With at most 8 heads in a group the low parts are rows 8..15 of the same instruction, which would
//    be empty otherwise; with 9..16 they are a second instruction.
//  * 8-bit caches: codes are converted to fp16 in registers (exactly); key scales multiply the
//    scores, value scales the weights.  There m follows the largest s_t log2e + log2 vscale_t, so that the
//    weights p_t vscale_t end at 1 (before the 2^14) and fp16 holds them whatever the scales; l is counted from the same m.
//  * Join.  A (request, head) that lies inside one warp's share is written by that warp.
//    Others leave (m, l, O) pieces: in shared memory, which the CTA joins in token order, and
//    where CTAs share one in the workspace, which the CTA that arrives last joins in CTA order.
//    The results do not depend on which one that is.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_mma.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = 32 * kAttnWarps;
constexpr int kAttnCounters = 340;  // at most so many CTAs, with three counters each

struct AttnArgs {
  const void* q;
  void* out;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  int64_t q_stride, out_stride, table_stride, scale_stride;
  float scale_log2;  // scale * log2(e)
  int window, requests, table_width, q_heads, kv_heads, group, splits;  // splits: groups of up to MR heads per kv head
  int page_size, pages;
  uint32_t page_mul;  // t / page_size = (t * page_mul) >> 32 >> page_shift for 0 <= t < 2^31
  int page_shift;
  int chunk_log2;    // tokens copied at once: the largest power of two that divides the page, at most TT
  int type;          // element type of q and out
  int min_units;     // a CTA's smallest share
  int seg_cost;      // units that a (request, head) costs beyond its tiles
  float* ws;
  int* cnt;
  int* err;
  uint64_t spin_ns;
  int stall;
};

// Shapes that follow from the head size and the cache type (KT: qgemv_kv_t).
template <int D, int KT, int MR>
struct AttnShape {
  static constexpr int kEl = KT == QGEMV_KV_E4M3 ? 1 : 2;
  static constexpr int kRow = D * kEl;                        // bytes of a token's head
  static constexpr int kRB = kRow < 128 ? kRow : 128;         // bytes of a row part in shared memory
  static constexpr int kParts = kRow / kRB;
  static constexpr int kTT = kRow >= 256 ? 16 : 4096 / kRow;  // tokens per tile
  static constexpr int kTTLog2 = kTT == 16 ? 4 : kTT == 32 ? 5 : 6;
  static constexpr int kTile = kTT * kRow;                    // bytes of keys (and of values)
  static constexpr int kScaleBytes = KT == QGEMV_KV_E4M3 ? 2 * kTT * 4 : 0;
  static constexpr int kPiece = MR * (D + 2);                 // floats of a piece: m, l, O
  // two where rings of two stages fit (64 requests of 2000 tokens, 8 heads of 256 in e4m3: 161 us with one, 107 to 112 with two)
  static constexpr int kCtasPerSm = D == 256 && (kEl == 2 || MR == 16) ? 1 : 2;
  static constexpr int kBudget = kCtasPerSm == 1 ? 232448 : 115712;
  static constexpr int kStatic = 1664;  // at least the kernel's static shared memory
  static constexpr int kFixed = 1024 + kAttnWarps * kPiece * 4;
  static constexpr int kFit = (kBudget - kFixed - kStatic) / (kAttnWarps * (2 * kTile + kScaleBytes));
  static constexpr int kStages = kFit < 3 ? kFit : 3;
  static constexpr int kSmem = kFixed + kAttnWarps * kStages * (2 * kTile + kScaleBytes);
  static_assert(kStages >= 2 && kPiece * 4 <= kStages * 2 * kTile, "shared memory");
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(a)
               : "memory");
}

// Four e4m3 codes as two fp16 pairs (exact).
__device__ __forceinline__ void e4m3x4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(four));
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int x, int row, int part, int head, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(part), "r"(head), "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// One arrival on `bar` when this thread's cp.async so far are there.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// What a warp has to know of a tile when it computes it (shared memory, one per tile in flight).
struct __align__(16) AttnTile {
  int r, hx;     // request; kv head * splits + split
  int lo, hi;    // tokens that the request sees
  int tok;       // first token
  int ends;      // bit 0: first tile of its (request, head); bit 1: last; bit 2: last of the share
  int bad;       // chunks whose page is outside the cache
  int pad;
  int64_t at;    // first unit of the (request, head)
};

// Where a warp's share begins: first unit of its (request, head), units left after its cost, tiles to skip.
struct AttnStart {
  int64_t at, left;
  int r, hx, skip;
};

// A piece of a (request, head) that more than one warp has a share of; its tiles are the units lo .. hi.
struct AttnPiece {
  int64_t lo, hi;
  int r, hx;
};

// The n pieces of one (request, head) that are to be joined (r = -1: none), into workspace piece `to` or (-1) the
// output.  The CTA's own: a mask of slots 2 warp + which.  In the workspace: piece `from`, then every
// `step` from `next` on.
struct AttnSet {
  int r, hx, n, to;
  uint32_t slots;
  int from, next, step;
};

// A (request, head) of up to so many units is one CTA's: where every CTA has a share, and where some have none.
constexpr int kAttnWhole = 32, kAttnWholeIdle = 16;

// More pieces than this are joined in groups first, each by the CTA that completes it.
constexpr int kAttnJoinMax = 24, kAttnJoinGroup = 16;

__device__ __forceinline__ int attn_page(const AttnArgs& p, int t) {
  return static_cast<int>(__umulhi(static_cast<uint32_t>(t), p.page_mul) >> p.page_shift);
}

// Length of request r in tokens, clamped to its row of the table.
__device__ __forceinline__ int attn_clamp(const AttnArgs& p, int len) {
  const int64_t end = min(static_cast<int64_t>(p.table_width) * p.page_size, int64_t{0x7fffff00});
  if (len < 0 || len > end) {
    atomicOr(p.err, kDevErrIndex);
    return len < 0 ? 0 : static_cast<int>(end);
  }
  return len;
}
__device__ __forceinline__ int attn_first(const AttnArgs& p, int len) { return p.window && len > p.window ? len - p.window : 0; }

// The kv head and the first query head in its group of head group hx.
template <int MR>
__device__ __forceinline__ void attn_group(const AttnArgs& p, int hx, int& kv, int& g0) {
  kv = p.splits == 1 ? hx : hx / p.splits;
  g0 = (hx - kv * p.splits) * MR;
}

// a / b for b < 2^31: 32-bit arithmetic where a allows it.
__device__ __forceinline__ int64_t attn_div(int64_t a, int b) {
  return a >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Two neighbouring outputs.
__device__ __forceinline__ void attn_store2(const AttnArgs& p, int64_t at, float a, float b) {
  uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at);
  *o = p.type == QGEMV_OUT_F16 ? pair16<false>(a, b) : pair16<true>(a, b);
}

__device__ __forceinline__ float attn_lse(float m, float l) {
  return l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : __int_as_float(0xff800000);
}

__device__ __forceinline__ int atom_add_acq_rel(int* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Joins four elements (from d) of head g of n pieces (at piece(i): m[MR], l[MR], O[MR][D]; SMEM: in shared
// memory, else in the workspace, read past L1) in their order, U at a time, whose loads are all in flight
// together.
template <int MR, int D, bool SMEM, class Piece>
__device__ __forceinline__ float4 attn_join(int n, int g, int d, Piece piece, float& m, float& l) {
  constexpr int U = SMEM ? 4 : 8;
  const float neg = __int_as_float(0xff800000);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  m = neg, l = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += U) {
    float mi[U], li[U];
    float4 o[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u < n) {
        const float* q = piece(i0 + u);
        const float4* v = reinterpret_cast<const float4*>(q + 2 * MR + g * D + d);
        mi[u] = SMEM ? q[g] : __ldcg(q + g);
        li[u] = SMEM ? q[MR + g] : __ldcg(q + MR + g);
        o[u] = SMEM ? *v : __ldcg(v);
      } else {
        mi[u] = neg;
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u) mn = fmaxf(mn, mi[u]);
    const float base = mn == neg ? 0.f : mn, f = ex2(m - base);
    m = mn;
    l *= f;
    s.x *= f, s.y *= f, s.z *= f, s.w *= f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u < n) {
        const float w = ex2(mi[u] - base);
        l += w * li[u];
        s.x += w * o[u].x, s.y += w * o[u].y, s.z += w * o[u].z, s.w += w * o[u].w;
      }
    }
  }
  return s;
}

template <int D, int KT, int MR>
__global__ void __launch_bounds__(kAttnThreads, AttnShape<D, KT, MR>::kCtasPerSm)
    attn_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttnArgs p) {
  using Sh = AttnShape<D, KT, MR>;
  constexpr bool kBF = KT == QGEMV_KV_BF16, kF8 = KT == QGEMV_KV_E4M3;
  constexpr float kLift = kBF ? 1.f : 16384.f;  // what the weights are multiplied by for the second product
  constexpr int TT = Sh::kTT, S = Sh::kStages, NT = TT / 8;  // NT: 8-token column tiles of the scores
  constexpr int OT = D / 8;                                  // 8-wide column tiles of the output
  extern __shared__ uint8_t dyn[];
  __shared__ int64_t scan[kAttnWarps];
  __shared__ int64_t bound[2];
  __shared__ AttnStart start_of[kAttnWarps];
  __shared__ AttnTile info_of[kAttnWarps][4];
  __shared__ uint64_t bars_of[kAttnWarps][4];     // of each stage: its copies are there
  __shared__ AttnPiece piece_of[2 * kAttnWarps];  // of each warp the one that began before its share, and the last
  __shared__ AttnPiece shared_of[2];
  __shared__ AttnSet set_of[2 * kAttnWarps];
  __shared__ int set_count[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float neg = __int_as_float(0xff800000);
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~uintptr_t{1023});
  float* heads_mem = reinterpret_cast<float*>(ring + kAttnWarps * S * 2 * Sh::kTile);
  uint8_t* scales_mem = reinterpret_cast<uint8_t*>(heads_mem + kAttnWarps * Sh::kPiece);
  if (lane < S) {
    mbar_init(smem_u32(&bars_of[warp][lane]), kF8 ? 33 : 1);  // the elected lane, and each for its scales
    fence_mbar_init();  // by every lane that made one: a fence orders its own thread's before the copies' signals
  }
  if (lane == 0) piece_of[2 * warp].r = piece_of[2 * warp + 1].r = -1;
  if (threadIdx.x < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(threadIdx.x ? &map_v : &map_k)) : "memory");

  pdl_wait();

  // ---- the share of this CTA and of its warps
  const int hxs = p.kv_heads * p.splits;
  // Shares are counted in units: a tile is one, and a (request, head) begins with p.seg_cost more, for
  // what it takes to begin and end one.
  auto tiles_of = [&](int len) { return (len + TT - 1) / TT - attn_first(p, len) / TT; };
  auto units_of = [&](int len) {
    const int n = tiles_of(len);
    return n ? n + p.seg_cost : 0;
  };
  const int per = (p.requests + kAttnThreads - 1) / kAttnThreads, r_lo = min(static_cast<int>(threadIdx.x) * per, p.requests),
            r_hi = min(r_lo + per, p.requests);
  int64_t mine = 0;
  int first_units = 0;  // of this thread's first request
  bool none = false;    // a request without tokens
  for (int r = r_lo; r < r_hi; ++r) {
    const int n = units_of(attn_clamp(p, p.lens[r]));
    if (r == r_lo) first_units = n;
    mine += n;
    none |= n == 0;
  }
  mine *= hxs;
  int64_t upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += u;
  }
  if (lane == 31) scan[warp] = upto;
  const bool any_none = __syncthreads_or(none);
  int64_t total = 0, before = upto - mine;
#pragma unroll
  for (int w = 0; w < kAttnWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const int cta = blockIdx.x;
  const int ctas = total >= static_cast<int64_t>(p.min_units) * gridDim.x ? gridDim.x  // with a share
                                                                          : static_cast<int>(attn_div(total + p.min_units - 1, p.min_units));
  const bool busy = cta < ctas;
  const int64_t each = busy ? attn_div(total, ctas) : 0;  // the first `more` CTAs have one unit more
  const int more = static_cast<int>(total - each * ctas);
  const int64_t even_lo = each * cta + min(cta, more), even_hi = even_lo + each + (cta < more ? 1 : 0);
  auto cta_of = [&](int64_t unit) {
    const int64_t big = (each + 1) * more;
    return static_cast<int>(unit < big ? attn_div(unit, static_cast<int>(each + 1)) : more + attn_div(unit - big, static_cast<int>(each)));
  };
  // The request of unit `at`, which is one of this thread's: where it begins, units of each (request, head).
  auto locate = [&](int64_t at, int64_t& pre, int& n) {
    int r = r_lo;
    pre = before;
    n = first_units;
    while (r < r_hi - 1 && at >= pre + static_cast<int64_t>(n) * hxs) {
      pre += static_cast<int64_t>(n) * hxs;
      n = units_of(attn_clamp(p, p.lens[++r]));
    }
    return r;
  };
  // A boundary inside a short (request, head) moves to its beginning: what the shares get less even costs less
  // than joining its pieces through the workspace, 3 us at the end of the launch (256 requests of up to 300
  // seen tokens and 16 heads: 38.6 -> 35.6 us; 64 of 400 tokens and 8 heads, of 27 units: 27.5 -> 24.3).  Where
  // CTAs are idle a head of 30 units is through sooner in pieces (one request of 450 tokens: 10.9 us, whole 12.1).
  const int64_t brief = max(int64_t{ctas == static_cast<int>(gridDim.x) ? kAttnWhole : kAttnWholeIdle}, each >> 3);
  if (busy) {
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const int64_t at = k ? even_hi : even_lo;
      if (at == total && threadIdx.x == 0) bound[k] = total;
      if (at < before || at >= before + mine) continue;
      int64_t pre;
      int n;
      locate(at, pre, n);
      bound[k] = n <= brief ? at - (at - pre - attn_div(at - pre, n) * n) : at;
    }
  }
  auto write_none = [&]() {  // the rows of requests that see no token
    for (int r = cta; r < p.requests; r += gridDim.x) {
      if (tiles_of(attn_clamp(p, p.lens[r]))) continue;
      for (int e = threadIdx.x; e < p.q_heads * (D / 2); e += kAttnThreads) attn_store2(p, r * p.out_stride + 2 * e, 0.f, 0.f);
      if (p.lse)
        for (int g = threadIdx.x; g < p.q_heads; g += kAttnThreads) p.lse[static_cast<int64_t>(r) * p.q_heads + g] = neg;
    }
  };
  __syncthreads();
  const int64_t c_lo = busy ? bound[0] : 0, c_hi = busy ? bound[1] : 0;
  if (c_lo == c_hi) {
    if (any_none) write_none();
    return;
  }
  auto warp_lo = [&](int w) { return c_lo + ((c_hi - c_lo) * w >> 2); };
  static_assert(kAttnWarps == 4, "warp shares are quarters");
#pragma unroll 1
  for (int w = 0; w < kAttnWarps; ++w) {
    const int64_t at = warp_lo(w);
    if (at < before || at >= before + mine) continue;
    int64_t pre;
    int n;
    const int r = locate(at, pre, n);
    const int hx = static_cast<int>(attn_div(at - pre, n)), in = static_cast<int>(at - pre - static_cast<int64_t>(hx) * n);
    start_of[w] = AttnStart{at - in, warp_lo(w + 1) - at - max(p.seg_cost - in, 0), r, hx, max(in - p.seg_cost, 0)};
  }
  __syncthreads();

  const int quad = lane & 3, row = lane >> 2;
  const uint32_t ring_w = smem_u32(ring) + warp * S * 2 * Sh::kTile, scale_w = smem_u32(scales_mem) + warp * S * Sh::kScaleBytes;
  const uint32_t full = smem_u32(&bars_of[warp][0]);
  const int ch = 1 << p.chunk_log2, chunks = TT >> p.chunk_log2;

  // ---- the walk over the tiles of this warp's share, in batches of tiles of one (request, head) whose chunks
  // have a lane each: the lane asks for its chunk's page while the batch before is copied
  const AttnStart st = start_of[warp];
  int64_t left = st.left, it_at = st.at;
  int it_r = st.r, it_hx = st.hx, it_t = 0, it_first = 0, it_end = 0, it_lo = 0, it_len = 0, it_next = 0, it_n = 0, it_page = -1;
  bool it_want = false;
  auto enter = [&](int r, int len) {
    it_r = r;
    it_len = len;
    it_lo = attn_first(p, len);
    it_first = it_lo / TT;
    it_end = (len + TT - 1) / TT;
    it_next = r + 1 < p.requests ? p.lens[r + 1] : 0;  // used when this request is through
  };
  auto ask = [&]() {  // the batch that begins at tile it_t
    const int at = it_t * TT + (lane << p.chunk_log2);
    it_n = static_cast<int>(min(left, static_cast<int64_t>(min(it_end - it_t, 32 >> (Sh::kTTLog2 - p.chunk_log2)))));
    it_want = left > 0 && lane < it_n * chunks && at < it_len && at + ch > it_lo;
    it_page = it_want ? p.table[it_r * p.table_stride + attn_page(p, at)] : -1;
  };
  if (left > 0) {
    enter(st.r, attn_clamp(p, p.lens[st.r]));
    it_t = it_first + st.skip;
    ask();
  }
  int b_r = 0, b_hx = 0, b_t = 0, b_n = 0, b_first = 0, b_end = 0, b_lo = 0, b_len = 0, b_page = -1, b_in = 0, b_k = 0, b_kv = 0;  // the batch in hand
  int64_t b_at = 0;
  uint32_t b_good = 0, b_bad = 0;
  bool to_copy = left > 0;
  // Copies the next tile into stage s.
  auto issue = [&](int s) {
    if (b_k == b_n) {
      b_k = 0;
      b_r = it_r, b_hx = it_hx, b_t = it_t, b_n = it_n, b_first = it_first, b_end = it_end, b_lo = it_lo, b_len = it_len, b_at = it_at;
      b_page = it_page;
      b_in = b_t * TT + (lane << p.chunk_log2);
      b_in -= attn_page(p, b_in) * p.page_size;
      const bool in = it_page >= 0 && it_page < p.pages;
      b_good = __ballot_sync(0xffffffffu, it_want && in);
      b_bad = __ballot_sync(0xffffffffu, it_want && !in);
      if (b_bad && lane == 0) atomicOr(p.err, kDevErrIndex);
      int g0;
      attn_group<MR>(p, b_hx, b_kv, g0);
      it_t += it_n;
      left -= it_n;
      if (it_t == it_end) {
        it_at += it_end - it_first + p.seg_cost;
        left -= p.seg_cost;
        if (++it_hx == hxs && left > 0) {
          it_hx = 0;
          for (int r = it_r + 1; r < p.requests; ++r) {
            enter(r, attn_clamp(p, it_next));
            if (it_end > it_first) break;
          }
        }
        it_t = it_first;
      }
      ask();
    }
    const int t = b_t + b_k, tok = t * TT, shift = b_k * chunks;
    const uint32_t mask = (2u << (chunks - 1)) - 1, good = b_good >> shift & mask;
    ++b_k;
    to_copy = b_k < b_n || left > 0;
    const uint32_t bar = full + 8 * s, dst = ring_w + s * 2 * Sh::kTile;
    auto copy = [&](int j) {  // chunk j of the tile
      const int page = __shfl_sync(0xffffffffu, b_page, shift + j), in_page = __shfl_sync(0xffffffffu, b_in, shift + j);
      if (!(good >> j & 1)) return;
      const uint32_t to = dst + (j << p.chunk_log2) * Sh::kRow;
      if (elect_one()) {
        tma_load_5d(to, &map_k, 0, in_page, 0, b_kv, page, bar);
        tma_load_5d(to + Sh::kTile, &map_v, 0, in_page, 0, b_kv, page, bar);
      }
      if constexpr (kF8) {  // two scales per token, 16 bytes a lane
        const int each16 = ch >> 2, u = lane & (each16 - 1);
        if (lane < 2 * each16) {
          const int64_t from = page * p.scale_stride + b_kv * p.page_size + in_page + 4 * u;
          cp_async16(scale_w + s * Sh::kScaleBytes + (lane < each16 ? 0 : TT * 4) + (j << p.chunk_log2) * 4 + 16 * u,
                     (lane < each16 ? p.k_scale : p.v_scale) + from);
        }
      }
    };
    if (elect_one()) {
      int4* d = reinterpret_cast<int4*>(&info_of[warp][s]);
      d[0] = make_int4(b_r, b_hx, b_lo, b_len);
      d[1] = make_int4(tok, (t == b_first ? 1 : 0) | (t == b_end - 1 ? 2 : 0) | (to_copy ? 0 : 4), b_bad >> shift & mask, 0);
      *reinterpret_cast<int64_t*>(d + 2) = b_at;
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(good)) * 2 * Sh::kRow << p.chunk_log2);
    }
    copy(0);
#pragma unroll 1
    for (int j = 1; j < chunks; ++j) copy(j);
    if constexpr (kF8) cp_async_arrive(bar);
    __syncwarp();
  };

  // Byte offset of token t of a tile, row part `part`, in shared memory (before the swizzle).
  auto line_of = [&](int t, int part) {
    return (t >> p.chunk_log2) * (Sh::kRow << p.chunk_log2) + part * (Sh::kRB << p.chunk_log2) + (t & (ch - 1)) * Sh::kRB;
  };
  // The copy's swizzle exchanges the 16-byte units of a row: address bits 4.. xor bits 7... Rows start at
  // multiples of their length, so unit u of this lane's row is at (stage + row) ^ turn ^ 16 u, where the row
  // and the turn do not depend on the tile.
  uint32_t k_row[TT / 16], v_row[TT / 16], k_turn[TT / 16], v_turn[TT / 16];
#pragma unroll
  for (int b = 0; b < TT / 16; ++b) {
    // rows of the 8x8 matrices that a lane addresses: keys (tokens 0..7, units u, u + 1; tokens 8..15, the same),
    // values (tokens 0..7, 8..15 of unit u; the same of unit u + 1)
    k_row[b] = line_of(16 * b + (lane >> 4) * 8 + (lane & 7), 0);
    v_row[b] = line_of(16 * b + (lane & 15), 0);
    k_turn[b] = ((k_row[b] >> 7 & (Sh::kRB / 16 - 1)) ^ (lane >> 3 & 1)) << 4;
    v_turn[b] = ((v_row[b] >> 7 & (Sh::kRB / 16 - 1)) ^ (lane >> 4)) << 4;
  }
  const uint32_t part_step = Sh::kRB << p.chunk_log2;

  constexpr int KS = D / 16;  // k steps of the scores
  uint32_t qa[KS][MR == 8 ? 2 : 4];
  float q_scale[2];  // scale_log2 times what the fp16 queries of rows `row`, `row` + 8 were divided by
  float o[OT][4];
  float m[2] = {neg, neg}, l[2] = {0.f, 0.f};

  // Query rows `row` (and `row` + 8) of a group in the order of the matrix product's A operand, requested
  // before the tile that needs them.
  uint32_t qn[MR / 8][KS][2];
  auto fetch_q = [&](int r, int hx) {
    int kv, g0;
    attn_group<MR>(p, hx, kv, g0);
#pragma unroll
    for (int j = 0; j < MR / 8; ++j) {
      const int g = g0 + row + 8 * j;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + r * p.q_stride + static_cast<int64_t>(kv * p.group + g) * D;
      const bool there = g < p.group;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if constexpr (kF8) {  // four consecutive elements: the order of four codes in a register
          const uint2 v = there ? *reinterpret_cast<const uint2*>(src + 16 * k + 4 * quad) : make_uint2(0, 0);
          qn[j][k][0] = v.x, qn[j][k][1] = v.y;
        } else {
          qn[j][k][0] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * quad) : 0u;
          qn[j][k][1] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * quad + 8) : 0u;
        }
      }
    }
  };
  auto take_q = [&]() {
#pragma unroll
    for (int j = 0; j < MR / 8; ++j) {
      uint32_t(&u)[KS][2] = qn[j];
      q_scale[j] = p.scale_log2;
      if (kF8 && p.type == QGEMV_OUT_BF16) {
        // bf16 queries as fp16 times a power of two per head: the largest in [2^14, 2^15), so every
        // one within 2^28 of it is exact
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = unpair16<true>(u[k][e]);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = (__float_as_int(top) >> 23) & 0xff;
        // 2^(141 - ex) takes 1.x 2^(ex - 127) to 1.x 2^14; both factors stay normal for 15 <= ex <= 254
        const bool fine = ex >= 15 && ex < 255;
        const float by = fine ? __int_as_float((127 + 141 - ex) << 23) : 1.f;
        if (fine) q_scale[j] *= __int_as_float((127 - 141 + ex) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = unpair16<true>(u[k][e]);
            u[k][e] = pair16<false>(f.x * by, f.y * by);
          }
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) qa[k][j] = u[k][0], qa[k][MR / 8 + j] = u[k][1];
    }
  };

  // The sums of the finished (part of a) request and head: out, or a piece.
  auto finish = [&](const AttnTile& d, bool whole, int slot) {
    int kv, g0;
    attn_group<MR>(p, d.hx, kv, g0);
#pragma unroll
    for (int j = 0; j < MR / 8; ++j) {
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
      l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
    }
    float* piece = slot == 0 ? heads_mem + warp * Sh::kPiece : reinterpret_cast<float*>(ring + warp * S * 2 * Sh::kTile);
    if (!whole && lane == 0) {
      const int64_t lo = d.at + p.seg_cost;
      piece_of[2 * warp + slot] = AttnPiece{lo, lo + (d.hi + TT - 1) / TT - d.lo / TT, d.r, d.hx};
    }
#pragma unroll
    for (int j = 0; j < MR / 8; ++j) {
      const int g = row + 8 * j;
      const bool there = g0 + g < p.group;
      const float f = whole ? (l[j] != 0.f ? 1.f / kLift / l[j] : 0.f) : 1.f;
      if (quad == 0) {
        if (!whole)
          piece[g] = m[j], piece[MR + g] = l[j];
        else if (there && p.lse)
          p.lse[static_cast<int64_t>(d.r) * p.q_heads + kv * p.group + g0 + g] = attn_lse(m[j], l[j]);
      }
      const int64_t at = d.r * p.out_stride + static_cast<int64_t>(kv * p.group + g0 + g) * D;
      auto put = [&](int e, float a, float b) {
        if (!whole)
          *reinterpret_cast<float2*>(piece + 2 * MR + g * D + e) = make_float2(a, b);
        else if (there)
          attn_store2(p, at + e, a, b);
      };
#pragma unroll
      for (int t = 0; t < OT; ++t) {
        if constexpr (kF8) {  // column tiles 2 i and 2 i + 1 hold the even and the odd elements
          if (t & 1) continue;
          float a[2], b[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            a[e] = (MR == 8 ? o[t][e] + o[t][2 + e] : o[t][2 * j + e]) * f;
            b[e] = (MR == 8 ? o[t + 1][e] + o[t + 1][2 + e] : o[t + 1][2 * j + e]) * f;
          }
          put(8 * t + 4 * quad, a[0], b[0]);
          put(8 * t + 4 * quad + 2, a[1], b[1]);
        } else {
          const float a = MR == 8 ? o[t][0] + o[t][2] : o[t][2 * j], b = MR == 8 ? o[t][1] + o[t][3] : o[t][2 * j + 1];
          put(8 * t + 2 * quad, a * f, b * f);
        }
      }
    }
  };

  bool alive = true, begun = false;  // begun: the current (request, head) began in this warp's share
  bool asked = false;                // its queries have been requested
  const bool any = st.left > 0;
  if (any) {
    fetch_q(st.r, st.hx);
    asked = true;
  }
  if (p.stall && cta == 0) to_copy = false;  // nothing is copied: the waits of this CTA run out
#pragma unroll 1
  for (int i = 1 - S, s = 1, lap = 0; any; ++i) {
    // stage s - 1 is free: before the first tile all are, then tile i - 1 was its last
    if (to_copy) issue(s == 0 ? S - 1 : s - 1);
    if (i < 0) {
      s = s + 1 == S ? 0 : s + 1;
      continue;
    }
    alive = mbar_wait_bounded(full + 8 * s, lap & 1, p.spin_ns);
    alive = __all_sync(0xffffffffu, alive);
    if (!alive) {
      if (lane == 0) atomicOr(p.err, kDevErrTimeout);
      break;
    }
    const AttnTile d = info_of[warp][s];
    if (i == 0 || (d.ends & 1)) {
      begun = d.ends & 1;
      if (!asked) fetch_q(d.r, d.hx);
      asked = false;
      take_q();
#pragma unroll
      for (int t = 0; t < OT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
      m[0] = m[1] = neg;
      l[0] = l[1] = 0.f;
    }
    const bool last = d.ends & 4;
    const int s_next = s + 1 == S ? 0 : s + 1;
    if (D < 256 && (d.ends & 2) && !last) {  // the next tile, already on its way, begins another
      fetch_q(info_of[warp][s_next].r, info_of[warp][s_next].hx);
      asked = true;
    }
    const uint32_t kb = ring_w + s * 2 * Sh::kTile, vb = kb + Sh::kTile;
    const bool edge = d.tok < d.lo || d.tok + TT > d.hi || d.bad;

    // scores: rows are heads, columns tokens
    float sc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
    uint32_t ka[TT / 16];
#pragma unroll
    for (int b = 0; b < TT / 16; ++b) ka[b] = (kb + k_row[b]) ^ k_turn[b];
#pragma unroll
    for (int k = 0; k < KS; k += kF8 ? 2 : 1) {  // a 16-byte unit holds half a k step, or one of codes
#pragma unroll
      for (int b = 0; b < TT / 16; ++b) {
        uint32_t w[4];
        ldsm4((ka[b] + k * 16 * Sh::kEl / Sh::kRB * part_step) ^ (k * 16 * Sh::kEl % Sh::kRB), w);
#pragma unroll
        for (int e = 0; e < (kF8 ? 2 : 1); ++e) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            uint32_t b0 = w[2 * n], b1 = w[2 * n + 1];
            if constexpr (kF8) e4m3x4(w[2 * n + e], b0, b1);
            if constexpr (MR == 8)
              mma16816<kBF>(sc[2 * b + n], qa[k + e][0], 0u, qa[k + e][1], 0u, b0, b1);
            else
              mma16816<kBF>(sc[2 * b + n], qa[k + e][0], qa[k + e][1], qa[k + e][2], qa[k + e][3], b0, b1);
          }
        }
      }
    }
    // softmax over the tile: this lane has tokens 8 t + 2 quad + {0, 1}
    float2 vsc[NT];
    float top[2] = {neg, neg};
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float2 ks = make_float2(p.scale_log2, p.scale_log2);
      if constexpr (kF8) {
        const uint32_t sa = scale_w + s * Sh::kScaleBytes + (8 * t + 2 * quad) * 4;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks.x), "=f"(ks.y) : "r"(sa));
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(vsc[t].x), "=f"(vsc[t].y) : "r"(sa + TT * 4));
      }
#pragma unroll
      for (int j = 0; j < MR / 8; ++j) {
        sc[t][2 * j] *= kF8 ? ks.x * q_scale[j] : ks.x;
        sc[t][2 * j + 1] *= kF8 ? ks.y * q_scale[j] : ks.y;
      }
      if (edge) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tk = 8 * t + 2 * quad + e;
          if (d.tok + tk < d.lo || d.tok + tk >= d.hi || (d.bad >> (tk >> p.chunk_log2) & 1)) {
            sc[t][e] = sc[t][2 + e] = neg;
            (e ? vsc[t].y : vsc[t].x) = 0.f;
          }
        }
      }
      // where a scale is below 2^-100 its weights are smaller than they might be, and l still far from its end
      const float2 up = kF8 ? make_float2(fmaxf(lg2(fabsf(vsc[t].x)), -100.f), fmaxf(lg2(fabsf(vsc[t].y)), -100.f)) : make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < MR / 8; ++j) top[j] = fmaxf(top[j], kF8 ? fmaxf(sc[t][2 * j] + up.x, sc[t][2 * j + 1] + up.y) : fmaxf(sc[t][2 * j], sc[t][2 * j + 1]));
    }
    bool moved = false;
    float keep[2] = {1.f, 1.f};
#pragma unroll
    for (int j = 0; j < MR / 8; ++j) {
      top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 1));
      top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], 2));
      const float mn = fmaxf(m[j], top[j]), base = mn == neg ? 0.f : mn;
      keep[j] = ex2(m[j] - base);
      moved |= mn > m[j];
      m[j] = mn;
      l[j] *= keep[j];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float a = ex2(sc[t][2 * j] - base), b = ex2(sc[t][2 * j + 1] - base);
        l[j] += a + b;
        sc[t][2 * j] = (kF8 ? a * vsc[t].x : a) * kLift;
        sc[t][2 * j + 1] = (kF8 ? b * vsc[t].y : b) * kLift;
      }
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int t = 0; t < OT; ++t) {
        o[t][0] *= keep[0], o[t][1] *= keep[0];
        o[t][2] *= keep[MR / 8 - 1], o[t][3] *= keep[MR / 8 - 1];
      }
    }
    if (edge) {  // what the values of unseen tokens hold must not meet their zero weights
      for (int e = lane; e < Sh::kTile / 16; e += 32) {
        const int tk = e / (Sh::kRow / 16), u = e - tk * (Sh::kRow / 16);
        if (d.tok + tk < d.lo || d.tok + tk >= d.hi || (d.bad >> (tk >> p.chunk_log2) & 1)) {
          const uint32_t a = vb + line_of(tk, u / (Sh::kRB / 16)) + (u % (Sh::kRB / 16)) * 16;
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0u) : "memory");
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before a later copy into this stage
      __syncwarp();
    }
    // weights times values
#pragma unroll
    for (int b = 0; b < TT / 16; ++b) {
      uint32_t hi[2][2], lo[2][2];  // [row half][token half]
#pragma unroll
      for (int j = 0; j < MR / 8; ++j)
#pragma unroll
        for (int n = 0; n < 2; ++n) split16<kBF>(sc[2 * b + n][2 * j], sc[2 * b + n][2 * j + 1], hi[j][n], lo[j][n]);
      const uint32_t va = (vb + v_row[b]) ^ v_turn[b];
      auto add = [&](float (&acc)[4], uint32_t b0, uint32_t b1) {
        if constexpr (MR == 8) {
          mma16816<kBF>(acc, hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
        } else {
          mma16816<kBF>(acc, hi[0][0], hi[1][0], hi[0][1], hi[1][1], b0, b1);
          mma16816<kBF>(acc, lo[0][0], lo[1][0], lo[0][1], lo[1][1], b0, b1);
        }
      };
#pragma unroll
      for (int u = 0; u < Sh::kRow / 16; u += 2) {
        uint32_t w[4];
        ldsm4t((va + u * 16 / Sh::kRB * part_step) ^ (u * 16 % Sh::kRB), w);
        if constexpr (!kF8) {
          add(o[u], w[0], w[1]);
          add(o[u + 1], w[2], w[3]);
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            // bytes: token a (even, odd element), token a + 1 (even, odd element)
            uint32_t x0, x1, y0, y1;
            e4m3x4(__byte_perm(w[2 * n], 0, 0x3120), x0, x1);
            e4m3x4(__byte_perm(w[2 * n + 1], 0, 0x3120), y0, y1);
            add(o[2 * (u + n)], x0, y0);
            add(o[2 * (u + n) + 1], x1, y1);
          }
        }
      }
    }
    __syncwarp();  // every lane is done with the stage
    const bool whole = (d.ends & 2) && begun;
    // one that began before this share, or goes on behind it, leaves a piece: where the copies were when it
    // is the last that the warp has to do, else in a place of its own
    if ((d.ends & 2) || last) finish(d, whole, !last ? 0 : 1);
    if (last) break;
    s = s_next;
    if (s == 0) ++lap;
  }
  if (!alive) {  // copies still in flight after a wait that gave up
    for (int s = 0; s < S; ++s) {
      mbar_wait_bounded(full + 8 * s, 0, p.spin_ns);
      mbar_wait_bounded(full + 8 * s, 1, p.spin_ns);
    }
  }
  pdl_launch_dependents();
  if (any_none) write_none();  // while the last warps finish
  __syncthreads();

  // ---- join: the warps' pieces in order; those of one (request, head) follow one another and are one
  // set.  First the sets of this CTA, then those that it is the last to bring a piece of.
  int sets = 0, shared_n = 0;
  if (warp == 0) {
    const AttnPiece a = piece_of[lane & 7];
    const bool there = lane < 2 * kAttnWarps && a.r >= 0;
    const uint32_t mask = __ballot_sync(0xffffffffu, there), below = mask & ((1u << lane) - 1);
    const int prev = below ? 31 - __clz(below) : lane;
    const int pr = __shfl_sync(0xffffffffu, a.r, prev), ph = __shfl_sync(0xffffffffu, a.hx, prev);
    const bool starts = there && (!below || pr != a.r || ph != a.hx);
    const uint32_t begin = __ballot_sync(0xffffffffu, starts);
    const bool shared = a.lo < c_lo || a.hi > c_hi;
    const uint32_t out = __ballot_sync(0xffffffffu, starts && shared);
    if (starts) {
      const uint32_t next = begin & ~((2u << lane) - 1);  // its pieces end before the next set's first
      const uint32_t own = mask & ~((1u << lane) - 1) & (next ? (next & -next) - 1 : 0xffu);
      set_of[__popc(begin & ((1u << lane) - 1))] = AttnSet{a.r, a.hx, __popc(own), shared ? 2 * cta + (a.lo >= c_lo ? 1 : 0) : -1, own, 0, 0, 0};
      if (shared) shared_of[__popc(out & ((1u << lane) - 1))] = a;
    }
    if (lane == 0) set_count[0] = __popc(begin), set_count[1] = __popc(out);
  }
  __syncthreads();
  sets = set_count[0], shared_n = set_count[1];
  // rounds: the CTA's own sets; those that it completed among the CTAs (of one group, where there are many); the groups
#pragma unroll 1
  for (int round = 0;; ++round) {
    // four elements of a head per thread: D / 4 threads a head, MR heads a set
    constexpr int kPer = MR * (D / 4);
#pragma unroll 1
    for (int e = threadIdx.x; e < sets * kPer; e += kAttnThreads) {
      const AttnSet t = set_of[e / kPer];
      const int g = e % kPer / (D / 4), d = e % (D / 4) * 4;
      int kv, g0;
      attn_group<MR>(p, t.hx, kv, g0);
      if (g0 + g >= p.group || t.r < 0) continue;
      float m, l;
      uint32_t slots = t.slots;
      auto mine = [&](int) -> const float* {  // they are asked for in order
        const int q = __ffs(slots) - 1;
        slots &= slots - 1;
        return reinterpret_cast<const float*>(q & 1 ? ring + (q >> 1) * S * 2 * Sh::kTile : reinterpret_cast<const uint8_t*>(heads_mem + (q >> 1) * Sh::kPiece));
      };
      auto theirs = [&](int i) -> const float* { return p.ws + static_cast<int64_t>(i ? t.next + t.step * (i - 1) : t.from) * Sh::kPiece; };
      const float4 o = round ? attn_join<MR, D, false>(t.n, g, d, theirs, m, l) : attn_join<MR, D, true>(t.n, g, d, mine, m, l);
      if (t.to >= 0) {
        float* to = p.ws + static_cast<int64_t>(t.to) * Sh::kPiece;
        if (d == 0) to[g] = m, to[MR + g] = l;
        *reinterpret_cast<float4*>(to + 2 * MR + g * D + d) = o;
      } else {
        const float f = l != 0.f ? 1.f / kLift / l : 0.f;
        const int64_t at = t.r * p.out_stride + static_cast<int64_t>(kv * p.group + g0 + g) * D + d;
        attn_store2(p, at, o.x * f, o.y * f);
        attn_store2(p, at + 2, o.z * f, o.w * f);
        if (d == 0 && p.lse) p.lse[static_cast<int64_t>(t.r) * p.q_heads + kv * p.group + g0 + g] = attn_lse(m, l);
      }
    }
    if (round == 2 || shared_n == 0) return;
    __syncthreads();
    sets = shared_n;
    bool again = false;
    if (static_cast<int>(threadIdx.x) < shared_n) {
      const AttnPiece a = shared_of[threadIdx.x];
      const int first = cta_of(a.lo), n = cta_of(a.hi - 1) - first + 1;
      const bool many = n > kAttnJoinMax;
      AttnSet t = set_of[threadIdx.x];
      if (round == 0 || (t.r >= 0 && t.to >= 0)) {  // in the second round: a group that it joined
        // Counters: of a (request, head) at the CTA where it begins; of its groups at the CTA where they begin, the
        // first group's apart from the others', since another's first group may begin there too.
        const int groups = (n + kAttnJoinGroup - 1) / kAttnJoinGroup, grp = (cta - first) / kAttnJoinGroup, at = first + grp * kAttnJoinGroup;
        const bool group = round == 0 && many;
        int* counter = p.cnt + (group ? (grp ? 2 : 1) * kAttnCounters + at : first);
        const int all = group ? min(kAttnJoinGroup, n - grp * kAttnJoinGroup) : many ? groups : n;
        // releases the CTA's pieces, which the barrier ordered before, and acquires the others'
        const bool last = atom_add_acq_rel(counter, 1) == all - 1;
        if (last) *counter = 0;  // for the next launch
        const int slots = 2 * gridDim.x;  // pieces of groups come behind those of CTAs
        t = AttnSet{last ? a.r : -1, a.hx, all, -1, 0, 0, 0, 0};
        if (group)
          t.to = slots + 2 * at + (grp ? 1 : 0), t.from = 2 * at + (grp ? 0 : 1), t.next = 2 * (at + 1), t.step = 2;
        else if (many)
          t.from = slots + 2 * first, t.next = slots + 2 * (first + kAttnJoinGroup) + 1, t.step = 2 * kAttnJoinGroup;
        else
          t.from = 2 * first + 1, t.next = 2 * (first + 1), t.step = 2;
        again = last;
      } else {
        t.r = -1;
      }
      set_of[threadIdx.x] = t;
    }
    if (!__syncthreads_or(again)) return;
  }
}

}  // namespace qg
