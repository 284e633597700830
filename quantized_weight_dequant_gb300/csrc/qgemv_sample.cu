// Entry point of the sampler.  See include/qgemv.h.
#include "qgemv_sample.cuh"

#include <cuda_runtime.h>

#include <algorithm>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

namespace {

constexpr int64_t kSampleHeld = 52 * 1024;  // of a row in a CTA, beside its table: two CTAs are on an SM

template <int T>
const void* kernel_for(bool held) {
  return held ? reinterpret_cast<const void*>(sample_kernel<T, true>) : reinterpret_cast<const void*>(sample_kernel<T, false>);
}

}  // namespace

extern "C" qgemv_status_t qgemv_sample(qgemv_handle_t hh, const qgemv_sample_t* sample, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !sample) return QGEMV_ERR_INVALID_ARG;
  const qgemv_sample_t& p = *sample;
  if (p.type != QGEMV_OUT_F32 && p.type != QGEMV_OUT_F16 && p.type != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  if (p.rows < 0 || p.rows > 0x7fffffff / kSampleMaxCluster || p.V < 1 || p.V > (1 << 20) || p.stride < p.V || p.stride > (int64_t{1} << 40))
    return QGEMV_ERR_BAD_SHAPE;
  if (p.rows > 0 && (!p.logits || !p.u || !p.tokens)) return QGEMV_ERR_INVALID_ARG;
  if (!aligned16(p.logits) || ((reinterpret_cast<uintptr_t>(p.u) | reinterpret_cast<uintptr_t>(p.temperature) | reinterpret_cast<uintptr_t>(p.top_k) |
                                reinterpret_cast<uintptr_t>(p.top_p) | reinterpret_cast<uintptr_t>(p.min_p) |
                                reinterpret_cast<uintptr_t>(p.tokens) | reinterpret_cast<uintptr_t>(p.logprobs)) & 3))
    return QGEMV_ERR_MISALIGNED;
  if (p.rows == 0) return QGEMV_OK;
  // as many CTAs a row as keep two on every SM, of 2048 logits at least; they hold it in shared memory where that is enough for it
  // beside a second CTA on the SM.  (64 x 128000 without limits: 34 us, 55 with CTAs for one on an SM, 48 for four; mixed 68, 104 and 68;
  // 4 x 16000 with top-p: 21.1, 19.5 with 1024 logits at least, 25.3 with 4096; 1 x 32000 11.3, 11.3 and 12.1, 1 x 8000 11.0, 10.9 and
  // 9.1)
  const int64_t most = kSampleHeld - static_cast<int64_t>(sample_table_bytes(p.type));
  const int64_t row_bytes = (int64_t{p.V} + 16) * (p.type == QGEMV_OUT_F32 ? 4 : 2);
  int ctas = 1;
  while (ctas < kSampleMaxCluster && p.rows * ctas * 2 <= 2 * int64_t{h->sms} && p.V >= ctas * 2 * 2048) ctas *= 2;
  const bool held = row_bytes <= most * ctas;
  const size_t fixed = sizeof(SampleSmem) + sample_table_bytes(p.type), smem = fixed + (held ? static_cast<size_t>((row_bytes / 16 / ctas + 2) * 16) : 0);
  const size_t largest = fixed + (held ? static_cast<size_t>((most / 16 + 2) * 16) : 0);  // row_bytes <= most * ctas
  const void* fn = p.type == QGEMV_OUT_F32 ? kernel_for<QGEMV_OUT_F32>(held) : p.type == QGEMV_OUT_F16 ? kernel_for<QGEMV_OUT_F16>(held) : kernel_for<QGEMV_OUT_BF16>(held);
  void* args[] = {const_cast<qgemv_sample_t*>(&p)};
  return launch_dependent(fn, dim3(static_cast<unsigned>(p.rows * ctas)), kSampleThreads, smem, ctas, args, stream, largest) ? QGEMV_OK : QGEMV_ERR_CUDA;
}
