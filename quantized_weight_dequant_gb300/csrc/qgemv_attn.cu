// Entry point of the paged attention.  See include/qgemv.h.
#include "qgemv_attn.cuh"

#include <cuda_runtime.h>

#include <algorithm>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The cache as a tensor of (row part, token in the page, part, head, page), copied in boxes of one
// part x 2^chunk_log2 tokens x all parts.
template <class Sh>
bool encode(const Handle& h, const qgemv_kv_cache_t& c, void* base, int chunk_log2, CUtensorMap* map) {
  const cuuint64_t el = Sh::kEl, row = Sh::kRow;
  const cuuint64_t dims[5] = {Sh::kRB / el, static_cast<cuuint64_t>(c.page_size), Sh::kParts, static_cast<cuuint64_t>(c.kv_heads),
                              static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[4] = {row, Sh::kRB, row * c.page_size, static_cast<cuuint64_t>(c.page_stride) * el};
  const cuuint32_t box[5] = {static_cast<cuuint32_t>(Sh::kRB / el), 1u << chunk_log2, Sh::kParts, 1, 1}, one[5] = {1, 1, 1, 1, 1};
  return reinterpret_cast<EncodeFn>(h.encode_tiled)(
             map, el == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, base, dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, Sh::kRB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KT, int MR>
qgemv_status_t launch(const Handle& h, const qgemv_attn_decode_t& p, AttnArgs a, cudaStream_t stream) {
  using Sh = AttnShape<D, KT, MR>;
  a.chunk_log2 = 3;
  while ((2 << a.chunk_log2) <= Sh::kTT && p.cache.page_size % (2 << a.chunk_log2) == 0) ++a.chunk_log2;
  CUtensorMap mk, mv;
  if (!encode<Sh>(h, p.cache, p.cache.k, a.chunk_log2, &mk) || !encode<Sh>(h, p.cache, p.cache.v, a.chunk_log2, &mv)) return QGEMV_ERR_CUDA;
  const void* fn = reinterpret_cast<const void*>(attn_decode_kernel<D, KT, MR>);
  a.splits = (a.group + MR - 1) / MR;
  // as many CTAs as run at once, and no more than the most tiles that the table can hold
  const int64_t tiles = (static_cast<int64_t>(p.table_width) * p.cache.page_size + Sh::kTT - 1) / Sh::kTT;
  const int64_t most = std::min<int64_t>(int64_t{1} << 30, tiles) * p.requests;
  const int64_t shares = std::min<int64_t>(int64_t{1} << 30, most) * (1 + a.seg_cost) * a.kv_heads * a.splits / a.min_units + 1;
  int64_t grid = std::min<int64_t>(static_cast<int64_t>(h.sms) * Sh::kCtasPerSm, shares);
  static_assert(3 * kAttnCounters <= kMaxRanges && int64_t{4} * kAttnCounters / (3 - Sh::kCtasPerSm) * Sh::kPiece <= int64_t{kWsFloats}, "workspace");
  grid = std::min<int64_t>(grid, kAttnCounters / (3 - Sh::kCtasPerSm));  // two pieces per CTA and group
  void* args[] = {&mk, &mv, &a};
  return launch_dependent(fn, dim3(static_cast<unsigned>(grid)), kAttnThreads, Sh::kSmem, 1, args, stream) ? QGEMV_OK : QGEMV_ERR_CUDA;
}

template <int D, int KT>
qgemv_status_t launch_rows(const Handle& h, const qgemv_attn_decode_t& p, const AttnArgs& a, cudaStream_t s) {
  return a.group <= 8 ? launch<D, KT, 8>(h, p, a, s) : launch<D, KT, 16>(h, p, a, s);
}

template <int D>
qgemv_status_t launch_type(const Handle& h, const qgemv_attn_decode_t& p, const AttnArgs& a, cudaStream_t s) {
  switch (p.cache.type) {
    case QGEMV_KV_F16: return launch_rows<D, QGEMV_KV_F16>(h, p, a, s);
    case QGEMV_KV_BF16: return launch_rows<D, QGEMV_KV_BF16>(h, p, a, s);
    default: return launch_rows<D, QGEMV_KV_E4M3>(h, p, a, s);
  }
}

}  // namespace

extern "C" qgemv_status_t qgemv_attn_decode(qgemv_handle_t hh, const qgemv_attn_decode_t* attn, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !attn) return QGEMV_ERR_INVALID_ARG;
  const qgemv_attn_decode_t& p = *attn;
  qgemv_status_t st = check_cache(p.cache);
  if (st != QGEMV_OK) return st;
  if (p.requests < 0 || p.requests > kMaxRequests || p.q_heads < 1 || p.q_heads % p.cache.kv_heads || p.table_width < 1 || p.table_stride < p.table_width)
    return QGEMV_ERR_BAD_SHAPE;
  if (p.type != QGEMV_OUT_F16 && p.type != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  if (p.cache.type != QGEMV_KV_E4M3 && static_cast<int>(p.cache.type) != static_cast<int>(p.type)) return QGEMV_ERR_INVALID_ARG;
  if (p.window < 0 || !(p.scale == p.scale)) return QGEMV_ERR_INVALID_ARG;
  if (p.requests > 0 && (!p.q || !p.out || !p.table || !p.lens)) return QGEMV_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(p.q_heads) * p.cache.head_dim;
  if (row > 0x3fffffff || p.q_stride < row || p.out_stride < row) return QGEMV_ERR_BAD_SHAPE;
  if (!aligned16(p.q) || !aligned16(p.out) || p.q_stride % 8 || p.out_stride % 8) return QGEMV_ERR_MISALIGNED;
  if (p.requests == 0) return QGEMV_OK;
  if (!h->encode_tiled) return QGEMV_ERR_CUDA;  // no TMA descriptors from this driver
  AttnArgs a{};
  a.q = p.q;
  a.out = p.out;
  a.lse = p.lse;
  a.table = p.table;
  a.lens = p.lens;
  a.k_scale = p.cache.k_scale;
  a.v_scale = p.cache.v_scale;
  a.q_stride = p.q_stride;
  a.out_stride = p.out_stride;
  a.table_stride = p.table_stride;
  a.scale_stride = p.cache.scale_stride;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.window = p.window;
  a.requests = p.requests;
  a.table_width = p.table_width;
  a.q_heads = p.q_heads;
  a.kv_heads = p.cache.kv_heads;
  a.group = p.q_heads / p.cache.kv_heads;
  a.page_size = p.cache.page_size;
  a.pages = p.cache.pages;
  a.type = p.type;
  a.min_units = 8;
  a.seg_cost = 2;
  // the reciprocal for t / page_size: with 2^(l-1) < page_size <= 2^l the product's excess over 2^(31+l)
  // is at most page_size <= 2^l per unit of t < 2^31
  int l = 3;
  while ((int64_t{1} << l) < a.page_size) ++l;
  a.page_mul = static_cast<uint32_t>((uint64_t{1} << (31 + l)) / a.page_size + 1);
  a.page_shift = l - 1;
  a.ws = h->ws;
  a.cnt = h->cnt;
  a.err = h->err;
  a.spin_ns = h->spin_ns;
  a.stall = h->test_stall;
  switch (p.cache.head_dim) {
    case 64: return launch_type<64>(*h, p, a, stream);
    case 128: return launch_type<128>(*h, p, a, stream);
    default: return launch_type<256>(*h, p, a, stream);
  }
}
