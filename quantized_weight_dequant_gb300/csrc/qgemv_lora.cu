// Entry point of the low-rank adapters.  See include/qgemv.h.
#include "qgemv_lora.cuh"

#include <cuda_runtime.h>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

extern "C" qgemv_status_t qgemv_run_lora(qgemv_handle_t hh, const qgemv_lora_t* lora, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !lora) return QGEMV_ERR_INVALID_ARG;
  const qgemv_lora_t& p = *lora;
  if (p.type != QGEMV_OUT_F16 && p.type != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  if (p.out < QGEMV_OUT_F32 || p.out > QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  if (p.rows < 0 || p.rows > 0x7fffffff || p.N < 1 || p.N > 0x7fffffff || p.K < 8 || p.K % 8 || p.K > 0x7fffffff ||
      p.adapters < 1 || p.rank < 8 || p.rank > kLoraMaxRank || p.rank % 8 || p.x_stride < p.K || p.y_stride < p.N)
    return QGEMV_ERR_BAD_SHAPE;
  if (!p.A || !p.B) return QGEMV_ERR_INVALID_ARG;
  if (p.rows > 0 && (!p.x || !p.ids || !p.y)) return QGEMV_ERR_INVALID_ARG;
  if (!aligned16(p.x) || !aligned16(p.A) || !aligned16(p.B) || !aligned16(p.base) || !aligned16(p.y) || p.x_stride % 8)
    return QGEMV_ERR_MISALIGNED;
  if (p.rows == 0) return QGEMV_OK;
  lora_kernel<<<static_cast<unsigned>(p.rows), 256, 0, stream>>>(p, h->err);
  return cudaGetLastError() == cudaSuccess ? QGEMV_OK : QGEMV_ERR_CUDA;
}
