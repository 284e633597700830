// Entry points of the paged cache's bookkeeping and store.  See include/qgemv.h.
#include "qgemv_pages.cuh"

#include <cuda_runtime.h>

#include <algorithm>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

namespace {

qgemv_status_t launched() { return cudaGetLastError() == cudaSuccess ? QGEMV_OK : QGEMV_ERR_CUDA; }

template <int T, bool INTER>
void launch_store(const qgemv_kv_store_t& p, dim3 g, int threads, int* err, cudaStream_t s) {
  switch (p.cache.head_dim) {
    case 64: kv_store_kernel<T, 64, INTER><<<g, threads, 0, s>>>(p, err); break;
    case 128: kv_store_kernel<T, 128, INTER><<<g, threads, 0, s>>>(p, err); break;
    default: kv_store_kernel<T, 256, INTER><<<g, threads, 0, s>>>(p, err); break;
  }
}

template <int T>
void launch_store(const qgemv_kv_store_t& p, dim3 g, int threads, int* err, cudaStream_t s) {
  p.interleaved ? launch_store<T, true>(p, g, threads, err, s) : launch_store<T, false>(p, g, threads, err, s);
}

}  // namespace

extern "C" {

qgemv_status_t qgemv_page_plan(qgemv_handle_t hh, const qgemv_page_plan_t* plan, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !plan) return QGEMV_ERR_INVALID_ARG;
  const qgemv_page_plan_t& p = *plan;
  if (p.requests < 0 || p.page_size < 1 || p.table_width < 1 || p.table_stride < p.table_width || p.capacity < 0 ||
      p.capacity > 0x7fffffff)
    return QGEMV_ERR_BAD_SHAPE;
  if (!p.counts || !p.free_count || (p.capacity > 0 && !p.slots)) return QGEMV_ERR_INVALID_ARG;
  if (p.requests > 0 && (!p.cached || !p.fresh || !p.table || !p.free_pages || !p.lens)) return QGEMV_ERR_INVALID_ARG;
  if (!aligned16(p.slots) || !aligned16(p.positions) || !aligned16(p.owners)) return QGEMV_ERR_MISALIGNED;
  // one scan step for up to 512 requests; a few need a few warps, whose scan is shorter
  const int threads = std::min(kPlanThreads, (std::max(p.requests, 128) + 31) / 32 * 32);
  int64_t per = kPlanThreads * kPlanVec;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((p.capacity + per - 1) / per, h->sms));
  per = (p.capacity + grid - 1) / grid;
  per = (per + kPlanVec - 1) / kPlanVec * kPlanVec;  // ranges start at whole vectors
  page_plan_kernel<<<static_cast<unsigned>(grid), threads, 0, stream>>>(p, per, h->err);
  return launched();
}

qgemv_status_t qgemv_kv_store(qgemv_handle_t hh, const qgemv_kv_store_t* store, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !store) return QGEMV_ERR_INVALID_ARG;
  const qgemv_kv_store_t& p = *store;
  qgemv_status_t st = check_cache(p.cache);
  if (st != QGEMV_OK) return st;
  if (p.tokens < 0) return QGEMV_ERR_BAD_SHAPE;
  if (p.tokens > 0 && (!p.k || !p.v || !p.slots || !p.positions || !p.q != !p.q_out)) return QGEMV_ERR_INVALID_ARG;
  if (p.in < QGEMV_OUT_F32 || p.in > QGEMV_OUT_BF16 || p.interleaved < 0 || p.interleaved > 1) return QGEMV_ERR_INVALID_ARG;
  if (p.q && p.q_type != QGEMV_OUT_F16 && p.q_type != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  const int64_t D = p.cache.head_dim, Hk = p.cache.kv_heads, Hq = p.q ? p.q_heads : 0;
  if ((p.q && p.q_heads < 1) || (p.rope && (p.rope_positions < 1 || p.rot_dim < 16 || p.rot_dim % 16 || p.rot_dim > D)))
    return QGEMV_ERR_BAD_SHAPE;
  if (p.k_stride < Hk * D || p.v_stride < Hk * D || (p.q && (p.q_stride < Hq * D || p.q_out_stride < Hq * D)))
    return QGEMV_ERR_BAD_SHAPE;
  const int64_t unit = p.in == QGEMV_OUT_F32 ? 4 : 8;  // elements in 16 bytes
  if (!aligned16(p.q) || !aligned16(p.k) || !aligned16(p.v) || !aligned16(p.q_out) || !aligned16(p.rope) || p.k_stride % unit ||
      p.v_stride % unit || (p.q && (p.q_stride % unit || p.q_out_stride % 8)))
    return QGEMV_ERR_MISALIGNED;
  if (p.tokens == 0) return QGEMV_OK;
  if (p.tokens > 0x7fffffff || Hq + 2 * Hk > 0xfffff) return QGEMV_ERR_BAD_SHAPE;
  // a thread for each eight elements of the token's heads, in whole warps
  const int threads = static_cast<int>(std::min<int64_t>(kStoreThreads, ((Hq + 2 * Hk) * (D / 8) + 31) / 32 * 32));
  // few tokens: their heads are spread over as many CTAs as keep one head a thread group, and the SMs busy
  const int64_t groups = ((Hq + 2 * Hk) * (D / 8) + threads - 1) / threads;
  const dim3 grid(static_cast<unsigned>(p.tokens), static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(groups, 2 * h->sms / p.tokens))));
  switch (p.in) {
    case QGEMV_OUT_F32: launch_store<QGEMV_OUT_F32>(p, grid, threads, h->err, stream); break;
    case QGEMV_OUT_F16: launch_store<QGEMV_OUT_F16>(p, grid, threads, h->err, stream); break;
    default: launch_store<QGEMV_OUT_BF16>(p, grid, threads, h->err, stream); break;
  }
  return launched();
}

}  // extern "C"
