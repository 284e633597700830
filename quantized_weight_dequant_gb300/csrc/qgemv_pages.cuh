// The paged key-value cache of a decode step: block tables and slot maps from request lengths,
// and the store that rotates q and k and writes k and v through the slot map.
#pragma once
#include <cstdint>

#include "../../include/qgemv.h"
#include "qgemv_elems.cuh"
#include "qgemv_ptx.cuh"

namespace qg {

// ------------------------------------------------------------------------------ page plan
// Per request r, with c cached and f new tokens (negative counts as 0) and page size P:
//   off  = sum of f before r                    (number of its first token)
//   room = min(f, W P - c)                      (tokens that its table row can hold)
//   have = ceil(c / P), need = ceil((c + room) / P) - have,  base = sum of need before r
// Requests after the one that crosses `capacity` get nothing and no one after them reads their
// base, so `need` may ignore the capacity and both sums come from one scan.  What bounds it is a
// chain of latencies (lengths, scan, table and free list, writes): 4.7 us for 64 requests, 8.9 us
// for 1024 requests that bring 128 thousand tokens, with what it writes at 0.3 TB/s.
struct PlanItem {
  int64_t off;    // number of the request's first token
  int64_t base;   // pages opened before it
  int32_t c;      // cached tokens
  int32_t kept;   // new tokens with a slot
  int32_t have;   // pages before
};

constexpr int kPlanThreads = 512;   // at most; also the requests per scan step
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
  pdl_wait();
  const int tid = threadIdx.x;
  int64_t n_kept = 0, n_got = 0, n_missing = 0;  // of this thread's requests
  __shared__ unsigned long long sums[3];
  if (tid < 3) sums[tid] = 0;
  const int64_t t0 = blockIdx.x * per_cta, t1 = min(t0 + per_cta, p.capacity);
  const int64_t P = p.page_size, room_all = min(static_cast<int64_t>(p.table_width) * P, int64_t{0x7fffffff});
  const int64_t F = max(*p.free_count, 0);
  int64_t tok = 0, pages = 0;  // carried over the scan steps
  // pages of n tokens: n, like every position, is below 2^31
  auto pages_of = [&](int64_t n) { return static_cast<int64_t>((static_cast<uint32_t>(n) + static_cast<uint32_t>(p.page_size) - 1) / static_cast<uint32_t>(p.page_size)); };
  int next_c = tid < p.requests ? p.cached[tid] : 0, next_f = tid < p.requests ? p.fresh[tid] : 0;
  for (int r0 = 0; r0 < p.requests; r0 += blockDim.x) {
    const int r = r0 + tid;
    const int64_t c = max(next_c, 0), f = max(next_f, 0);
    const int r_next = r + static_cast<int>(blockDim.x);  // read while this step is worked on
    next_c = r_next < p.requests ? p.cached[r_next] : 0;
    next_f = r_next < p.requests ? p.fresh[r_next] : 0;
    const int64_t room = min(f, max(room_all - c, int64_t{0}));
    const int64_t have = pages_of(c);
    const int64_t need = room > 0 ? pages_of(c + room) - have : 0;
    int64_t off, base, dt, dp;
    block_scan2(f, need, off, base, dt, dp, ws);
    off += tok;
    base += pages;
    // what the capacity and the stack leave of it
    const int64_t f1 = min(room, max(p.capacity - off, int64_t{0}));
    const int64_t need1 = f1 == room ? need : f1 > 0 ? pages_of(c + f1) - have : 0;
    const int64_t got = min(need1, max(F - base, int64_t{0}));
    const int64_t kept = got < need1 ? (have + got) * P - c : f1;
    item[tid] = PlanItem{off, base, static_cast<int32_t>(c), static_cast<int32_t>(kept), static_cast<int32_t>(have)};
    if (blockIdx.x == 0 && r < p.requests) {
      p.lens[r] = static_cast<int32_t>(c + kept);
      if (p.offsets) p.offsets[r] = sat32(off);
      n_kept += kept;
      n_got += got;
      n_missing += need1 - got;
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
      // neighbouring tokens, and most of those of a thread, are of one page: the table is read when it changes
      int32_t page = -1, page_at = -1, page_of = -1;
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
        if (at != page_at || i != page_of) {
          int32_t* cell = p.table + (r0 + i) * p.table_stride + at;
          page_at = at, page_of = i;
          page = at >= q.have ? p.free_pages[F - 1 - (q.base + (at - q.have))] : *cell;
          if (at >= q.have && in == 0) *cell = page;
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
  pdl_launch_dependents();
  for (int64_t t = max(t0, tok) + tid; t < t1; t += blockDim.x) {  // past the last token
    p.slots[t] = -1;
    if (p.positions) p.positions[t] = -1;
    if (p.owners) p.owners[t] = -1;
  }
  if (blockIdx.x == 0) {  // the totals
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      n_kept += __shfl_xor_sync(0xffffffffu, n_kept, d);
      n_got += __shfl_xor_sync(0xffffffffu, n_got, d);
      n_missing += __shfl_xor_sync(0xffffffffu, n_missing, d);
    }
    __syncthreads();  // the sums' zeros
    if (tid % 32 == 0) atomicAdd(&sums[0], static_cast<unsigned long long>(n_kept)), atomicAdd(&sums[1], static_cast<unsigned long long>(n_got)), atomicAdd(&sums[2], static_cast<unsigned long long>(n_missing));
    __syncthreads();
    if (tid == 0) {
      if (p.offsets) p.offsets[p.requests] = sat32(tok);
      p.counts[0] = sat32(tok);
    }
    if (tid < 3) p.counts[1 + tid] = sat32(static_cast<int64_t>(sums[tid]));
  }
}

// ------------------------------------------------------------------------------ cache store
// A CTA (or gridDim.y, where tokens are few) per token: the D / 8 threads of a head are neighbours in a warp and take the token's heads (q, then
// k, then v) in turn, so that slot, position and angles are read once.  Bound by the bytes of q, k and v: the
// reads of kU heads are in flight together, and the first of them before slot and position are known.
// Eight CTAs of four warps on an SM: 8191 tokens of 48 bf16 heads of 128 into e4m3 36.4 us (5.2 TB/s;
// 43.5 in pairs of halves, which spill 20 bytes a thread; as it was first: 40.4 us as five CTAs of eight warps, 38.3 as CTAs that walk over the tokens; six heads in flight spill), into
// bf16 40.4 us (41.5 with the pairs' other halves read instead of exchanged among the lanes); 4096 tokens of fp32
// rows into fp16 27.9 us; 64 tokens of them 2.5 us in a graph.
constexpr int kStoreThreads = 128;

template <int T, int D, bool INTER>  // INTER: pairs of neighbours
__global__ void __launch_bounds__(kStoreThreads, T == QGEMV_OUT_F32 ? 6 : 8) kv_store_kernel(const __grid_constant__ qgemv_kv_store_t p, int* err) {
  constexpr int L = D / 8;  // threads per head
  constexpr int kU = 3;
  const int hq = p.q_out ? p.q_heads : 0, hk = p.cache.kv_heads;
  const int heads = hq + 2 * hk, step = static_cast<int>(blockDim.x * gridDim.y) / L;
  const int64_t t = blockIdx.x;
  const int d = (threadIdx.x % L) * 8;
  const int half = p.rot_dim / 2;
  const bool first = d < half;
  const bool turns = p.rope && d < p.rot_dim;
  // the lanes of this head, and that of them whose elements this thread's are paired with
  const int lane = threadIdx.x & 31;
  const uint32_t mates = L == 32 ? 0xffffffffu : ((1u << (L & 31)) - 1) << (lane / L * L);
  const int mate = !turns ? lane : first ? lane + half / 8 : lane - half / 8;
  constexpr int kEl = T == QGEMV_OUT_F32 ? 4 : 2;
  // this thread's elements of the token's first q, k and v head; the heads are numbered through
  const uint8_t* q_at = static_cast<const uint8_t*>(p.q) + (t * p.q_stride + d) * kEl;
  const uint8_t* k_at = static_cast<const uint8_t*>(p.k) + (t * p.k_stride + d) * kEl - hq * (D * kEl);
  const uint8_t* v_at = static_cast<const uint8_t*>(p.v) + (t * p.v_stride + d) * kEl - (hq + hk) * (D * kEl);
  Raw8<T> v[kU];
  auto read = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int head = h0 + u * step;
      if (head >= heads) break;
      v[u] = load_raw<T>((head < hq ? q_at : head < hq + hk ? k_at : v_at) + head * (D * kEl));
    }
  };
  pdl_launch_dependents();
  pdl_wait();
  const int h_first = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x) / L;
  read(h_first);
  const int64_t slot = p.slots[t];
  int32_t pos = p.positions[t];
  int64_t page = -1, cell = 0;  // cell: elements from a head's page row to this thread's
  int in = 0;
  if (slot >= 0) {
    page = slot >> 32 ? slot / p.cache.page_size : static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.cache.page_size);
    in = static_cast<int>(slot - page * p.cache.page_size);
    cell = page * p.cache.page_stride + static_cast<int64_t>(in) * D + d;
  }
  const bool stored = slot >= 0 && page < p.cache.pages;
  bool lost = pos != -1 && p.rope && (pos < 0 || pos >= p.rope_positions);
  if (threadIdx.x == 0 && blockIdx.y == 0 && (lost || (!stored && slot != -1))) atomicOr(err, kDevErrIndex);
  if (lost) pos = -1;
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
  if (turns && pos >= 0) {
    const float* tab = p.rope + static_cast<int64_t>(pos) * p.rot_dim;
    if constexpr (INTER) {
      const float4 a = *reinterpret_cast<const float4*>(tab + d / 2), b = *reinterpret_cast<const float4*>(tab + half + d / 2);
      c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w, s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
    } else {
      to_float<QGEMV_OUT_F32>(load_raw<QGEMV_OUT_F32>(reinterpret_cast<const uint8_t*>(tab + (first ? d : d - half))), c);
      to_float<QGEMV_OUT_F32>(load_raw<QGEMV_OUT_F32>(reinterpret_cast<const uint8_t*>(tab + half + (first ? d : d - half))), s);
    }
  }
  const int el = p.cache.type == QGEMV_KV_E4M3 ? 1 : 2;
  uint8_t* q_to = static_cast<uint8_t*>(p.q_out) + (t * p.q_out_stride + d) * 2;
  for (int h0 = h_first; h0 < heads; h0 += kU * step) {
    if (h0 != h_first) read(h0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int head = h0 + u * step;
      if (head >= heads) break;
      float x[8];
      to_float<T>(v[u], x);
      if (p.rope && pos >= 0 && head < hq + hk) {
        if constexpr (INTER) {
          if (turns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a = x[2 * j], b = x[2 * j + 1];
              x[2 * j] = a * c[j] - b * s[j];
              x[2 * j + 1] = b * c[j] + a * s[j];
            }
          }
        } else {
          Raw8<T> o;
#pragma unroll
          for (int j = 0; j < static_cast<int>(sizeof(o.v) / 16); ++j) {
            o.v[j].x = __shfl_sync(mates, v[u].v[j].x, mate);
            o.v[j].y = __shfl_sync(mates, v[u].v[j].y, mate);
            o.v[j].z = __shfl_sync(mates, v[u].v[j].z, mate);
            o.v[j].w = __shfl_sync(mates, v[u].v[j].w, mate);
          }
          if (turns) {
            float y[8];
            to_float<T>(o, y);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = first ? x[j] * c[j] - y[j] * s[j] : x[j] * c[j] + y[j] * s[j];
          }
        }
      }
      if (head < hq) {
        if (pos < 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = 0.f;
        }
        *reinterpret_cast<uint4*>(q_to + head * (2 * D)) = pack8(p.q_type, x);
        continue;
      }
      if (!stored) continue;
      const bool is_k = head < hq + hk;
      const int h = head - (is_k ? hq : hq + hk), lines = p.cache.page_size;
      uint8_t* to = static_cast<uint8_t*>(is_k ? p.cache.k : p.cache.v) + (cell + static_cast<int64_t>(h * lines) * D) * el;
      if (el == 2) {
        *reinterpret_cast<uint4*>(to) = pack8(p.cache.type, x);
        continue;
      }
      float top = 0.f;  // NaN where one of them is
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(x[j]));
#pragma unroll
      for (int k = L / 2; k > 0; k >>= 1) top = max_nan(top, __shfl_xor_sync(mates, top, k));
      const float scale = e4m3_scale(top);
      const uint2 code = e4m3_codes(x, top, scale);
      *reinterpret_cast<uint2*>(to) = code;
      if (d == 0)
        (is_k ? p.cache.k_scale : p.cache.v_scale)[page * p.cache.scale_stride + h * lines + in] = scale;
    }
  }
}

}  // namespace qg
