// The paged key-value cache of a decode step: block tables and slot maps from request lengths,
// and the store that rotates q and k and writes k and v through the slot map.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_ptx.cuh"

namespace qg {

// ------------------------------------------------------------------------------ page plan
// Per request r, with c cached and f new tokens (negative counts as 0) and page size P:
//   off  = sum of f before r                    (number of its first token)
//   room = min(f, W P - c)                      (tokens that its table row can hold)
//   have = ceil(c / P), need = ceil((c + room) / P) - have,  base = sum of need before r
// Requests after the one that crosses `capacity` get nothing and no one after them reads their
// base, so `need` may ignore the capacity and both sums come from one scan.
struct PlanItem {
  int64_t off;    // number of the request's first token
  int64_t base;   // pages opened before it
  int32_t c;      // cached tokens
  int32_t kept;   // new tokens with a slot
  int32_t have;   // pages before
};

constexpr int kPlanThreads = 512;   // also the requests per scan step
constexpr int kPlanVec = 4;         // consecutive tokens per thread

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) { return __shfl_up_sync(0xffffffffu, v, d); }

// Exclusive sums over the block of (a, b); totals in (ta, tb).  ws: 2 x 32 values in shared memory.
__device__ __forceinline__ void block_scan2(int64_t a, int64_t b, int64_t& ea, int64_t& eb, int64_t& ta, int64_t& tb,
                                            int64_t (*ws)[32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t ia = a, ib = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t ua = shfl_up64(ia, d), ub = shfl_up64(ib, d);
    if (lane >= d) ia += ua, ib += ub;
  }
  if (lane == 31) ws[0][w] = ia, ws[1][w] = ib;
  __syncthreads();
  int64_t pa = 0, pb = 0;
  ta = tb = 0;
  for (int i = 0; i < nw; ++i) {
    if (i == w) pa = ta, pb = tb;
    ta += ws[0][i];
    tb += ws[1][i];
  }
  ea = pa + ia - a;
  eb = pb + ib - b;
}

__device__ __forceinline__ int32_t sat32(int64_t v) { return v > 0x7fffffff ? 0x7fffffff : static_cast<int32_t>(v); }

// Every CTA scans all requests (8 bytes each, from L2 after the first reader) and fills its own
// range of the tokens, so nothing has to be passed between CTAs; CTA 0 also writes what there is
// one of per request.
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const qgemv_page_plan_t p, int64_t per_cta, int* err) {
  __shared__ PlanItem item[kPlanThreads];
  __shared__ int64_t ws[2][32];
  __shared__ unsigned long long tot[3];
  const int tid = threadIdx.x;
  if (tid < 3) tot[tid] = 0;
  const int64_t t0 = blockIdx.x * per_cta, t1 = min(t0 + per_cta, p.capacity);
  const int64_t P = p.page_size, room_all = min(static_cast<int64_t>(p.table_width) * P, int64_t{0x7fffffff});
  const int64_t F = max(*p.free_count, 0);
  int64_t tok = 0, pages = 0;  // carried over the scan steps
  for (int r0 = 0; r0 < p.requests; r0 += blockDim.x) {
    const int r = r0 + tid;
    int64_t c = 0, f = 0;
    if (r < p.requests) c = max(p.cached[r], 0), f = max(p.fresh[r], 0);
    const int64_t room = min(f, max(room_all - c, int64_t{0}));
    const int64_t have = (c + P - 1) / P;
    const int64_t need = room > 0 ? (c + room + P - 1) / P - have : 0;
    int64_t off, base, dt, dp;
    block_scan2(f, need, off, base, dt, dp, ws);
    off += tok;
    base += pages;
    // what the capacity and the stack leave of it
    const int64_t f1 = min(room, max(p.capacity - off, int64_t{0}));
    const int64_t need1 = f1 > 0 ? (c + f1 + P - 1) / P - have : 0;
    const int64_t got = min(need1, max(F - base, int64_t{0}));
    const int64_t kept = got < need1 ? (have + got) * P - c : f1;
    item[tid] = PlanItem{off, base, static_cast<int32_t>(c), static_cast<int32_t>(kept), static_cast<int32_t>(have)};
    if (blockIdx.x == 0 && r < p.requests) {
      p.lens[r] = static_cast<int32_t>(c + kept);
      if (p.offsets) p.offsets[r] = sat32(off);
      if (kept) atomicAdd(&tot[0], static_cast<unsigned long long>(kept));
      if (got) atomicAdd(&tot[1], static_cast<unsigned long long>(got));
      if (need1 > got) atomicAdd(&tot[2], static_cast<unsigned long long>(need1 - got));
    }
    __syncthreads();
    const int64_t a = max(t0, tok), b = min(t1, tok + dt);  // this step's tokens in this CTA's range
    const int n = min(static_cast<int>(blockDim.x), p.requests - r0);
    for (int64_t v = a / kPlanVec + tid; v * kPlanVec < b; v += blockDim.x) {
      const int64_t lo = max(v * kPlanVec, a), hi = min((v + 1) * kPlanVec, b);
      int i = 0;  // the last request of this step that starts at or before token lo
      for (int span = n; span > 1;) {
        const int half = span >> 1;
        if (item[i + half].off <= lo) i += half;
        span -= half;
      }
      int64_t slot[kPlanVec];
      int32_t pos[kPlanVec], own[kPlanVec];
      const int skip = static_cast<int>(lo - v * kPlanVec);
#pragma unroll
      for (int j = 0; j < kPlanVec; ++j) {
        const int64_t t = v * kPlanVec + j;
        slot[j] = -1;
        pos[j] = -1;
        if (t < lo || t >= hi) continue;
        while (i + 1 < n && item[i + 1].off <= t) ++i;
        own[j] = r0 + i;
        const PlanItem& q = item[i];
        const int64_t k = t - q.off;
        if (k >= q.kept) continue;
        pos[j] = static_cast<int32_t>(q.c + k);
        const int32_t at = pos[j] / p.page_size, in = pos[j] - at * p.page_size;
        int32_t* cell = p.table + (r0 + i) * p.table_stride + at;
        int32_t page;
        if (at >= q.have) {
          page = p.free_pages[F - 1 - (q.base + (at - q.have))];
          if (in == 0) *cell = page;
        } else {
          page = *cell;
        }
        if (page >= 0)
          slot[j] = static_cast<int64_t>(page) * p.page_size + in;
        else
          atomicOr(err, kDevErrIndex);
      }
      const int64_t t = v * kPlanVec;
      if (skip == 0 && hi == t + kPlanVec) {  // a whole vector: 16-byte stores
        reinterpret_cast<longlong2*>(p.slots + t)[0] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2*>(p.slots + t)[1] = make_longlong2(slot[2], slot[3]);
        if (p.positions) *reinterpret_cast<int4*>(p.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (p.owners) *reinterpret_cast<int4*>(p.owners + t) = make_int4(own[0], own[1], own[2], own[3]);
      } else {
#pragma unroll
        for (int j = 0; j < kPlanVec; ++j) {
          if (t + j < lo || t + j >= hi) continue;
          p.slots[t + j] = slot[j];
          if (p.positions) p.positions[t + j] = pos[j];
          if (p.owners) p.owners[t + j] = own[j];
        }
      }
    }
    tok += dt;
    pages += dp;
    __syncthreads();  // item and ws are rewritten
  }
  for (int64_t t = max(t0, tok) + tid; t < t1; t += blockDim.x) {  // past the last token
    p.slots[t] = -1;
    if (p.positions) p.positions[t] = -1;
    if (p.owners) p.owners[t] = -1;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (p.offsets) p.offsets[p.requests] = sat32(tok);
    p.counts[0] = sat32(tok);
    for (int i = 0; i < 3; ++i) p.counts[1 + i] = sat32(static_cast<int64_t>(tot[i]));
  }
}

// ------------------------------------------------------------------------------ cache store
// Eight consecutive elements of a head per thread, all in fp32.
template <int T>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
  if constexpr (T == QGEMV_OUT_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
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

// Thread i of the launch takes eight elements of one head of one token; the D / 8 threads of a
// head are neighbours in a warp.  The heads of a token are its q heads, then k, then v.
template <int T, int D>
__global__ void __launch_bounds__(256) kv_store_kernel(const qgemv_kv_store_t p, int* err) {
  constexpr int L = D / 8;  // threads per head
  const int hq = p.q_out ? p.q_heads : 0, hk = p.cache.kv_heads;
  const int heads = hq + 2 * hk;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / L;
  const int64_t t = unit / heads;
  if (t >= p.tokens) return;  // whole heads leave together
  const int head = static_cast<int>(unit - t * heads), d = (threadIdx.x % L) * 8;
  const bool is_q = head < hq, is_k = !is_q && head < hq + hk;
  const int h = is_q ? head : is_k ? head - hq : head - hq - hk;
  int64_t slot = -1, page = 0;
  int in = 0;
  if (!is_q) {
    slot = p.slots[t];
    page = slot / p.cache.page_size;
    in = static_cast<int>(slot - page * p.cache.page_size);
    if (slot < 0 || page >= p.cache.pages) {
      if (slot != -1 && d == 0) atomicOr(err, kDevErrIndex);
      return;
    }
  }
  int32_t pos = is_q || is_k ? p.positions[t] : 0;
  if (pos != -1 && p.rope && (pos < 0 || pos >= p.rope_positions)) {
    if (d == 0) atomicOr(err, kDevErrIndex);
    pos = -1;
  }
  const void* src = is_q ? p.q : is_k ? p.k : p.v;
  const int64_t row = t * (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) + static_cast<int64_t>(h) * D;
  float v[8];
  load8<T>(src, row + d, v);
  if ((is_q || is_k) && p.rope && d < p.rot_dim && pos >= 0) {
    const float* tab = p.rope + static_cast<int64_t>(pos) * p.rot_dim;
    const int half = p.rot_dim / 2;
    if (p.interleaved) {
      const float4 c = *reinterpret_cast<const float4*>(tab + d / 2), s = *reinterpret_cast<const float4*>(tab + half + d / 2);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j], b = v[2 * j + 1];
        v[2 * j] = a * cc[j] - b * ss[j];
        v[2 * j + 1] = b * cc[j] + a * ss[j];
      }
    } else {
      const bool first = d < half;
      const int i = first ? d : d - half;
      float o[8], c[8], s[8];
      load8<T>(src, row + (first ? d + half : d - half), o);
      load8<QGEMV_OUT_F32>(tab, i, c);
      load8<QGEMV_OUT_F32>(tab, half + i, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = first ? v[j] * c[j] - o[j] * s[j] : v[j] * c[j] + o[j] * s[j];
    }
  }
  if (is_q) {
    if (pos < 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + t * p.q_out_stride + static_cast<int64_t>(h) * D + d) =
        pack8(p.q_type, v);
    return;
  }
  const int64_t line = static_cast<int64_t>(h) * p.cache.page_size + in;
  const int64_t at = page * p.cache.page_stride + line * D + d;
  void* dst = is_k ? p.cache.k : p.cache.v;
  if (p.cache.type != QGEMV_KV_E4M3) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + at) = pack8(p.cache.type, v);
    return;
  }
  float top = 0.f;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[j])), nan |= v[j] != v[j];
  if (nan) top = __int_as_float(0x7f800000);
  const uint32_t mates = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1) << ((threadIdx.x & 31) / L * L);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mates, top, o));
  float scale = __fdiv_rn(top, 448.f);
  if (!(scale > 0.f && scale < __int_as_float(0x7f800000))) scale = 1.f;
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float* x = v + 4 * j;
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)), __NV_SATFINITE, __NV_E4M3);
    w[j] = lo | hi << 16;
  }
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(dst) + at) = make_uint2(w[0], w[1]);
  if (d == 0) (is_k ? p.cache.k_scale : p.cache.v_scale)[page * p.cache.scale_stride + line] = scale;
}

}  // namespace qg
