// Argument checks shared by the entry points that read or write a paged key-value cache.
#pragma once
#include <cstdint>

#include "../../include/qgemv.h"

namespace qg {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline int64_t kv_elem_bytes(const qgemv_kv_cache_t& c) { return c.type == QGEMV_KV_E4M3 ? 1 : 2; }

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
