// Entry points of the row operators.  See include/qgemv.h.
#include "qgemv_rows.cuh"

#include <cuda_runtime.h>

#include <algorithm>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

namespace {

constexpr int kNormWarpThreads = 2048, kNormThreads = 1024;  // on an SM, a warp or a CTA to a row
constexpr int64_t kMaxStride = int64_t{1} << 40;  // elements: offsets of a row stay clear of 64 bits

bool out_type(qgemv_out_t t) { return t == QGEMV_OUT_F32 || t == QGEMV_OUT_F16 || t == QGEMV_OUT_BF16; }
int64_t out_bytes(qgemv_out_t t) { return t == QGEMV_OUT_F32 ? 4 : 2; }

template <bool WIDE, int RES, bool WARP>
const void* norm_kernel_v(int v) {
  if (v == 1) return reinterpret_cast<const void*>(norm_kernel<WIDE, RES, 1, WARP>);
  if constexpr (!WARP) {
    if (v == 4) return reinterpret_cast<const void*>(norm_kernel<WIDE, RES, 4, WARP>);
    if (v == 8) return reinterpret_cast<const void*>(norm_kernel<WIDE, RES, 8, WARP>);
  }
  return reinterpret_cast<const void*>(norm_kernel<WIDE, RES, 2, WARP>);
}
template <bool WIDE, bool WARP>
const void* norm_kernel_res(int res, int v) {
  return res == 0 ? norm_kernel_v<WIDE, 0, WARP>(v) : res == 1 ? norm_kernel_v<WIDE, 1, WARP>(v) : norm_kernel_v<WIDE, 2, WARP>(v);
}

}  // namespace

extern "C" {

qgemv_status_t qgemv_run_norm(qgemv_handle_t hh, const qgemv_norm_t* norm, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !norm) return QGEMV_ERR_INVALID_ARG;
  const qgemv_norm_t& p = *norm;
  if (!out_type(p.in) || !out_type(p.res_type) || !out_type(p.weight_type) || !out_type(p.out)) return QGEMV_ERR_INVALID_ARG;
  if (!(p.eps >= 0.f) || !(p.offset == p.offset)) return QGEMV_ERR_INVALID_ARG;
  if (p.rows < 0 || p.rows > 0x7fffffff || p.N < 8 || p.N > 65536 || p.N % (p.codes ? 16 : 8)) return QGEMV_ERR_BAD_SHAPE;
  if (p.rows > 0 && (!p.x || (!p.y && !p.codes) || (p.codes && !p.scale))) return QGEMV_ERR_INVALID_ARG;
  auto bad = [&](const void* at, int64_t stride) { return at && (stride < p.N || stride > kMaxStride); };
  if (bad(p.x, p.x_stride) || bad(p.res, p.res_stride) || bad(p.res_out, p.res_out_stride) || bad(p.y, p.y_stride) ||
      bad(p.codes, p.codes_stride) || (p.codes && (p.scale_stride < (p.N + 127) / 128 || p.scale_stride > kMaxStride)))
    return QGEMV_ERR_BAD_SHAPE;
  auto off = [](const void* at, int64_t stride, int64_t el) { return at && (!aligned16(at) || stride * el % 16); };
  if (off(p.x, p.x_stride, out_bytes(p.in)) || off(p.res, p.res_stride, out_bytes(p.res_type)) ||
      off(p.res_out, p.res_out_stride, out_bytes(p.res_type)) || off(p.y, p.y_stride, out_bytes(p.out)) || off(p.codes, p.codes_stride, 1) ||
      !aligned16(p.weight) || (p.codes && reinterpret_cast<uintptr_t>(p.scale) % 4))
    return QGEMV_ERR_MISALIGNED;
  if (p.rows == 0) return QGEMV_OK;
  // Up to 512 elements a warp has a row, and 64 warps an SM; more: a CTA (65528 rows of 256: 25.5 us, with a CTA for each 40.4; of
  // 512 the two are close, 44.1 and 39.6).  Many rows: a thread has two pieces of its row or more and a CTA goes on to the row 1024
  // threads an SM on, whose elements it reads before it finishes the first (8191 rows of 4096 in bf16: 40.0 us, 52.7 with one piece,
  // 55.8 with four, 46.7 with a CTA for each row; of 14336 144, with a CTA for each 211; fp32 rows of 4096 with a bf16 residual 48.1,
  // 53.7 with one piece, 82.5 with four; with an fp32 residual one piece would do: 83.6 and 66.4).  Few rows: as many threads as
  // there are pieces.
  const int vecs = static_cast<int>(p.N / 8);
  const bool warp = vecs <= 64;
  int v = 1;
  if (warp) {
    v = vecs <= 32 ? 1 : 2;
  } else {
    while (1024 * v < vecs) v *= 2;
    if (v == 1 && p.rows > 2 * h->sms) v = 2;
  }
  const int threads = warp ? 32 * kNormWarps : ((vecs + v - 1) / v + 31) / 32 * 32;
  const int64_t resident = static_cast<int64_t>(h->sms) * std::max(1, (warp ? kNormWarpThreads : kNormThreads) / threads);
  const int64_t grid = std::min<int64_t>(warp ? (p.rows + kNormWarps - 1) / kNormWarps : p.rows, resident);
  const int res = !p.res ? 0 : p.res_type == QGEMV_OUT_F32 ? 2 : 1;
  const bool wide = p.in == QGEMV_OUT_F32;
  const void* fn = wide ? (warp ? norm_kernel_res<true, true>(res, v) : norm_kernel_res<true, false>(res, v))
                        : (warp ? norm_kernel_res<false, true>(res, v) : norm_kernel_res<false, false>(res, v));
  void* args[] = {const_cast<qgemv_norm_t*>(&p)};
  return launch_dependent(fn, dim3(static_cast<unsigned>(grid)), threads, 0, 1, args, stream) ? QGEMV_OK : QGEMV_ERR_CUDA;
}

qgemv_status_t qgemv_quant_rows(qgemv_handle_t hh, const qgemv_quant_t* quant, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !quant) return QGEMV_ERR_INVALID_ARG;
  const qgemv_quant_t& p = *quant;
  if (!out_type(p.in)) return QGEMV_ERR_INVALID_ARG;
  if (p.rows < 0 || p.rows > 0x7fffffff || p.N < 16 || p.N % 16 || p.N > 0x40000000) return QGEMV_ERR_BAD_SHAPE;
  if (p.rows > 0 && (!p.x || !p.codes || !p.scale)) return QGEMV_ERR_INVALID_ARG;
  auto bad = [&](const void* at, int64_t stride) { return at && (stride < p.N || stride > kMaxStride); };
  if (bad(p.x, p.x_stride) || bad(p.up, p.up_stride) || bad(p.codes, p.codes_stride) || p.scale_stride < (p.N + 127) / 128 || p.scale_stride > kMaxStride)
    return QGEMV_ERR_BAD_SHAPE;
  const int64_t el = out_bytes(p.in);
  if (!aligned16(p.x) || !aligned16(p.up) || !aligned16(p.codes) || p.x_stride * el % 16 || (p.up && p.up_stride * el % 16) ||
      p.codes_stride % 16 || reinterpret_cast<uintptr_t>(p.scale) % 4)
    return QGEMV_ERR_MISALIGNED;
  int chunks = static_cast<int>((p.N + 16 * kQuantThreads - 1) / (16 * kQuantThreads));
  if (p.rows * chunks > 0x7fffffff) return QGEMV_ERR_BAD_SHAPE;
  if (p.rows == 0) return QGEMV_OK;
  const bool wide = p.in == QGEMV_OUT_F32;
  const void* fn = p.up ? (wide ? reinterpret_cast<const void*>(quant_kernel<true, true>) : reinterpret_cast<const void*>(quant_kernel<false, true>))
                        : (wide ? reinterpret_cast<const void*>(quant_kernel<true, false>) : reinterpret_cast<const void*>(quant_kernel<false, false>));
  void* args[] = {const_cast<qgemv_quant_t*>(&p), &chunks};
  return launch_dependent(fn, dim3(static_cast<unsigned>(p.rows), std::min(chunks, 65535)), kQuantThreads, 0, 1, args, stream) ? QGEMV_OK : QGEMV_ERR_CUDA;
}

}  // extern "C"
