// Entry point of the paged attention.  See include/qgemv.h.
#include "qgemv_attn.cuh"

#include <cuda_runtime.h>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

extern "C" qgemv_status_t qgemv_attn_decode(qgemv_handle_t hh, const qgemv_attn_decode_t* attn, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !attn) return QGEMV_ERR_INVALID_ARG;
  const qgemv_attn_decode_t& p = *attn;
  qgemv_status_t st = check_cache(p.cache);
  if (st != QGEMV_OK) return st;
  if (p.requests < 0 || p.q_heads < 1 || p.q_heads % p.cache.kv_heads || p.table_width < 1 || p.table_stride < p.table_width)
    return QGEMV_ERR_BAD_SHAPE;
  if (p.type != QGEMV_OUT_F16 && p.type != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  if (p.cache.type != QGEMV_KV_E4M3 && static_cast<int>(p.cache.type) != static_cast<int>(p.type)) return QGEMV_ERR_INVALID_ARG;
  if (p.window < 0 || !(p.scale == p.scale)) return QGEMV_ERR_INVALID_ARG;
  if (p.requests > 0 && (!p.q || !p.out || !p.table || !p.lens)) return QGEMV_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(p.q_heads) * p.cache.head_dim;
  if (p.q_stride < row || p.out_stride < row) return QGEMV_ERR_BAD_SHAPE;
  if (!aligned16(p.q) || !aligned16(p.out) || p.q_stride % 8 || p.out_stride % 8) return QGEMV_ERR_MISALIGNED;
  if (p.requests == 0) return QGEMV_OK;
  const int64_t units = static_cast<int64_t>(p.requests) * p.q_heads;
  if (units > 0x7fffffff) return QGEMV_ERR_BAD_SHAPE;
  const unsigned grid = static_cast<unsigned>((units + 3) / 4);
  switch (p.cache.head_dim) {
    case 64: attn_decode_kernel<64><<<grid, 128, 0, stream>>>(p, h->err); break;
    case 128: attn_decode_kernel<128><<<grid, 128, 0, stream>>>(p, h->err); break;
    default: attn_decode_kernel<256><<<grid, 128, 0, stream>>>(p, h->err); break;
  }
  return cudaGetLastError() == cudaSuccess ? QGEMV_OK : QGEMV_ERR_CUDA;
}
