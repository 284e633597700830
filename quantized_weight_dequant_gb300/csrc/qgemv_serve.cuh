// Launches of the serving operators, and the argument checks of those that read or write a paged cache.
#pragma once
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/qgemv.h"

namespace qg {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The kernels number requests in 32 bits and step past the last one by up to a block, so the end stays clear of 2^31.
constexpr int kMaxRequests = 1 << 30;

inline int64_t kv_elem_bytes(const qgemv_kv_cache_t& c) { return c.type == QGEMV_KV_E4M3 ? 1 : 2; }

// A programmatic dependent launch: the kernel may start while the one before it on the stream ends, so every
// kernel launched here waits (pdl_wait) before it touches memory, and lets the next one start in turn.  Among
// small launches this takes the launch latency out of the stream (1.5 us each).  What the kernel before writes
// changes while this one is there already, so nothing is read through the non-coherent path (__ldg, const
// __restrict__), which is for memory that nobody writes during a kernel's whole life.
// The dynamic shared memory that a kernel may have belongs to the function on its device, so that what one host thread asks for
// holds for another one's launch: every call asks for the same.  `most`: of a kernel whose `smem` varies, the largest.
inline bool launch_dependent(const void* fn, dim3 grid, int threads, size_t smem, int cluster, void** args, cudaStream_t stream, size_t most = 0) {
  if (most == 0) most = smem;
  // up to 48 KB, with what the kernel has statically (none more than 24 KB beside dynamic memory), need no request
  if (most > 24 * 1024 && cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most)) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess) return true;
  cudaGetLastError();
  return false;
}

inline qgemv_status_t check_cache(const qgemv_kv_cache_t& c) {
  if (!c.k || !c.v || c.type < QGEMV_KV_F16 || c.type > QGEMV_KV_E4M3) return QGEMV_ERR_INVALID_ARG;
  if (c.type == QGEMV_KV_E4M3 && (!c.k_scale || !c.v_scale)) return QGEMV_ERR_INVALID_ARG;
  if (c.pages < 1 || c.kv_heads < 1 || (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) ||
      (c.page_size != 8 && (c.page_size < 16 || c.page_size % 16)))
    return QGEMV_ERR_BAD_SHAPE;
  const int64_t lines = static_cast<int64_t>(c.kv_heads) * c.page_size;
  if (lines > 0x7fffffff || c.page_stride < lines * c.head_dim || c.page_stride > (int64_t{1} << 38))
    return QGEMV_ERR_BAD_SHAPE;
  if (c.type == QGEMV_KV_E4M3 && (c.scale_stride < lines || c.scale_stride > (int64_t{1} << 32))) return QGEMV_ERR_BAD_SHAPE;
  if (!aligned16(c.k) || !aligned16(c.v) || c.page_stride * kv_elem_bytes(c) % 16) return QGEMV_ERR_MISALIGNED;
  if (c.type == QGEMV_KV_E4M3 && (!aligned16(c.k_scale) || !aligned16(c.v_scale) || c.scale_stride % 4)) return QGEMV_ERR_MISALIGNED;
  return QGEMV_OK;
}

}  // namespace qg
