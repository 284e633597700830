// Entry points of the paged cache's bookkeeping and store.  See include/qgemv.h.
#include "qgemv_pages.cuh"

#include <cuda_runtime.h>

#include <algorithm>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

namespace {

template <int T, bool INTER>
const void* store_kernel_for(int dim) {
  switch (dim) {
    case 64: return reinterpret_cast<const void*>(kv_store_kernel<T, 64, INTER>);
    case 128: return reinterpret_cast<const void*>(kv_store_kernel<T, 128, INTER>);
    default: return reinterpret_cast<const void*>(kv_store_kernel<T, 256, INTER>);
  }
}

template <int T>
const void* store_kernel_for(int dim, bool interleaved) {
  return interleaved ? store_kernel_for<T, true>(dim) : store_kernel_for<T, false>(dim);
}

}  // namespace

extern "C" {

qgemv_status_t qgemv_page_plan(qgemv_handle_t hh, const qgemv_page_plan_t* plan, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !plan) return QGEMV_ERR_INVALID_ARG;
  const qgemv_page_plan_t& p = *plan;
  if (p.requests < 0 || p.requests > kMaxRequests || p.page_size < 1 || p.table_width < 1 || p.table_stride < p.table_width || p.capacity < 0 ||
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
  int* err = h->err;
  void* args[] = {const_cast<qgemv_page_plan_t*>(&p), &per, &err};
  const bool ok = launch_dependent(reinterpret_cast<const void*>(page_plan_kernel), dim3(static_cast<unsigned>(grid)), threads, 0, 1, args, stream);
  return ok ? QGEMV_OK : QGEMV_ERR_CUDA;
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
  const bool inter = p.interleaved == 1;
  const int dim = p.cache.head_dim;
  const void* fn = p.in == QGEMV_OUT_F32   ? store_kernel_for<QGEMV_OUT_F32>(dim, inter)
                   : p.in == QGEMV_OUT_F16 ? store_kernel_for<QGEMV_OUT_F16>(dim, inter)
                                           : store_kernel_for<QGEMV_OUT_BF16>(dim, inter);
  int* err = h->err;
  void* args[] = {const_cast<qgemv_kv_store_t*>(&p), &err};
  return launch_dependent(fn, grid, threads, 0, 1, args, stream) ? QGEMV_OK : QGEMV_ERR_CUDA;
}

}  // extern "C"
