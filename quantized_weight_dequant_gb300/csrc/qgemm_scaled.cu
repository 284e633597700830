// Entry point of the 8-bit projection.  See include/qgemv.h.
#include "qgemm_scaled.cuh"

#include <cuda_runtime.h>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

extern "C" qgemv_status_t qgemv_run_scaled(qgemv_handle_t hh, const qgemv_scaled_t* scaled, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !scaled) return QGEMV_ERR_INVALID_ARG;
  const qgemv_scaled_t& p = *scaled;
  if (p.out != QGEMV_OUT_F32 && p.out != QGEMV_OUT_F16 && p.out != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  constexpr int64_t most = 0x7fffffff, far = int64_t{1} << 38;
  if (p.M < 0 || p.M > most || p.N < 1 || p.N > most || p.K < 16 || p.K > most || p.K % 16 || p.x_stride < p.K || p.x_stride > far ||
      p.x_scale_stride < (p.K + 127) / 128 || p.x_scale_stride > far || p.y_stride < p.N || p.y_stride > far)
    return QGEMV_ERR_BAD_SHAPE;
  if (!p.W || !p.w_scale || (p.M > 0 && (!p.x || !p.x_scale || !p.y))) return QGEMV_ERR_INVALID_ARG;
  if (!aligned16(p.x) || !aligned16(p.W) || !aligned16(p.y) || p.x_stride % 16 ||
      ((reinterpret_cast<uintptr_t>(p.x_scale) | reinterpret_cast<uintptr_t>(p.w_scale)) & 3))
    return QGEMV_ERR_MISALIGNED;
  if (p.M == 0) return QGEMV_OK;
  unsigned row_sets = static_cast<unsigned>((p.M + kFp8SimpleRows - 1) / kFp8SimpleRows);
  const int64_t grid = (p.N + 7) / 8 * row_sets;
  if (grid > most) return QGEMV_ERR_BAD_SHAPE;
  void* args[] = {const_cast<qgemv_scaled_t*>(&p), &row_sets};
  return launch_dependent(reinterpret_cast<const void*>(fp8_simple_kernel), dim3(static_cast<unsigned>(grid)), 256, 0, 1, args, stream) ? QGEMV_OK
                                                                                                                                : QGEMV_ERR_CUDA;
}
