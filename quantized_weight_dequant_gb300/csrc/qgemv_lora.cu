// Entry point of the low-rank adapters.  See include/qgemv.h.
#include "qgemv_lora.cuh"

#include <cuda_runtime.h>

#include <algorithm>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

namespace {

template <int TG, bool BF>
const void* kernel_for(int out) {
  switch (out) {
    case QGEMV_OUT_F32: return reinterpret_cast<const void*>(lora_kernel<BF, QGEMV_OUT_F32, TG>);
    case QGEMV_OUT_F16: return reinterpret_cast<const void*>(lora_kernel<BF, QGEMV_OUT_F16, TG>);
    default: return reinterpret_cast<const void*>(lora_kernel<BF, QGEMV_OUT_BF16, TG>);
  }
}

template <int TG>
qgemv_status_t launch(const Handle& h, const qgemv_lora_t& p, cudaStream_t stream) {
  // Clusters per kRows rows: one for each adapter that they can have, but no more in all than run at once
  // (then a cluster takes its share of the adapters one after another).
  constexpr int kRows = LoraShape<TG>::kRows;
  const int64_t chunks = (p.rows + kRows - 1) / kRows;
  const int64_t most = std::min<int64_t>(kRows, p.rows), resident = int64_t{h.sms} * LoraShape<TG>::kCtasPerSm / kLoraCluster;
  int slots = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, (resident + chunks - 1) / chunks)));
  // Clusters that share an adapter's N, where there are fewer than two rounds of them: at least three tiles for
  // a warp.
  const int64_t tiles = (p.N + 31) / 32;
  int shares = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(2 * resident / (chunks * slots), tiles / (3 * kLoraWarps * kLoraCluster))));
  const int64_t grid = chunks * slots * shares * kLoraCluster;
  if (grid > 0x7fffffff) return QGEMV_ERR_BAD_SHAPE;
  const void* fn = p.type == QGEMV_OUT_BF16 ? kernel_for<TG, true>(p.out) : kernel_for<TG, false>(p.out);
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(LoraSmem<TG>)) != cudaSuccess) {
    cudaGetLastError();
    return QGEMV_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(kLoraThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(LoraSmem<TG>);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kLoraCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int* err = h.err;
  void* args[] = {const_cast<qgemv_lora_t*>(&p), &slots, &shares, &err};
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) {
    cudaGetLastError();
    return QGEMV_ERR_CUDA;
  }
  return QGEMV_OK;
}

}  // namespace

extern "C" qgemv_status_t qgemv_run_lora(qgemv_handle_t hh, const qgemv_lora_t* lora, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !lora) return QGEMV_ERR_INVALID_ARG;
  const qgemv_lora_t& p = *lora;
  if (p.type != QGEMV_OUT_F16 && p.type != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  if (p.out < QGEMV_OUT_F32 || p.out > QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  if (p.rows < 0 || p.rows > 0x7fffffff || p.N < 1 || p.N > 0x40000000 || p.K < 8 || p.K % 8 || p.K > 0x7fffffff ||
      p.adapters < 1 || p.rank < 8 || p.rank > kLoraMaxRank || p.rank % 8 || p.x_stride < p.K || p.y_stride < p.N)
    return QGEMV_ERR_BAD_SHAPE;
  if (!p.A || !p.B) return QGEMV_ERR_INVALID_ARG;
  if (p.rows > 0 && (!p.x || !p.ids || !p.y)) return QGEMV_ERR_INVALID_ARG;
  if (!aligned16(p.x) || !aligned16(p.A) || !aligned16(p.B) || !aligned16(p.base) || !aligned16(p.y) || p.x_stride % 8)
    return QGEMV_ERR_MISALIGNED;
  if (p.rows == 0) return QGEMV_OK;
  return p.rows <= kLoraFewRows ? launch<1>(*h, p, stream) : launch<2>(*h, p, stream);
}
