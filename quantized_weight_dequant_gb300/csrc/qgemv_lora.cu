// Entry point of the low-rank adapters.  See include/qgemv.h.
#include "qgemv_lora.cuh"

#include <cuda_runtime.h>

#include <algorithm>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

using namespace qg;

namespace {

// Rows whose sums fit the workspace are one pair of launches.
template <bool BF, int OUT>
bool launch(const Handle& h, qgemv_lora_t p, const LoraWork& work, cudaStream_t stream) {
  const bool few = p.rows <= kLoraFewRows;
  const int64_t chunks = (p.rows + kLoraChunk - 1) / kLoraChunk;
  // Sums: clusters per chunk of rows, one for each adapter that they can have, but no more in all than run at
  // once (then a cluster takes its share of the adapters one after another).
  const int64_t resident = int64_t{h.sms} * 4 / kLoraCluster;
  int slots = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(kLoraChunk, p.rows), resident / chunks)));
  LoraWork w = work;
  int* err = h.err;
  void* sums[] = {&p, &w, &slots, &err};
  const void* fn = few ? reinterpret_cast<const void*>(lora_sums_kernel<BF, 1>) : reinterpret_cast<const void*>(lora_sums_kernel<BF, 4>);
  if (!launch_dependent(fn, dim3(static_cast<unsigned>(chunks * slots * kLoraCluster)), kLoraThreads, 0, kLoraCluster, sums, stream)) return false;
  const int64_t tiles = (p.N + 31) / 32;
  if (few) {
    // as many CTAs as run at once, each with at least two tiles for a warp
    const unsigned grid = static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(int64_t{h.sms} * 4, p.rows * tiles / (2 * kLoraWarps))));
    void* args[] = {&p, &w};
    return launch_dependent(reinterpret_cast<const void*>(lora_few_kernel<BF, OUT>), dim3(grid), kLoraThreads, sizeof(LoraFewSmem), 1, args, stream);
  }
  // as many parts of the rows as fill the GPU once, at least two tiles of rows each
  const int64_t cols = (p.N + 32 * kLoraWarps - 1) / (32 * kLoraWarps);
  const int nb = w.blocks == 1 ? 1 : w.blocks == 2 ? 2 : 4;
  const int64_t at_once = int64_t{h.sms} * (nb == 1 ? 4 : nb == 2 ? 3 : 2);
  int splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(at_once / cols, (p.rows + 31) / 32)));
  void* args[] = {&p, &w, &splits};
  const dim3 grid(static_cast<unsigned>(cols * splits));
  auto run = [&](const void* kernel, size_t stage) { return launch_dependent(kernel, grid, kLoraThreads, (kLoraAhead + 1) * stage, 1, args, stream); };
  switch (nb) {
    case 1: return run(reinterpret_cast<const void*>(lora_many_kernel<BF, OUT, 1>), sizeof(LoraManyStage<BF, 1>));
    case 2: return run(reinterpret_cast<const void*>(lora_many_kernel<BF, OUT, 2>), sizeof(LoraManyStage<BF, 2>));
    default: return run(reinterpret_cast<const void*>(lora_many_kernel<BF, OUT, 4>), sizeof(LoraManyStage<BF, 4>));
  }
}

template <bool BF>
bool launch_out(const Handle& h, const qgemv_lora_t& p, const LoraWork& work, cudaStream_t stream) {
  switch (p.out) {
    case QGEMV_OUT_F32: return launch<BF, QGEMV_OUT_F32>(h, p, work, stream);
    case QGEMV_OUT_F16: return launch<BF, QGEMV_OUT_F16>(h, p, work, stream);
    default: return launch<BF, QGEMV_OUT_BF16>(h, p, work, stream);
  }
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
  const bool bf = p.type == QGEMV_OUT_BF16;
  LoraWork work{};
  work.blocks = (p.rank + 31) / 32;
  const int64_t row_bytes = int64_t{64} * work.blocks * lora_parts(bf);
  const int64_t rest_bytes = bf ? 0 : int64_t{128} * work.blocks;
  // rows at a time: whole tiles of 16, their sums, factors and adapters in the workspace
  const int64_t most = static_cast<int64_t>(kWsFloats) * 4 / (row_bytes + static_cast<int64_t>(sizeof(LoraRow)) + rest_bytes) / 32 * 32;
  work.parts = reinterpret_cast<uint4*>(h->ws);
  for (int64_t m = 0; m < p.rows; m += most) {
    qgemv_lora_t q = p;
    q.rows = std::min(most, p.rows - m);
    q.x = static_cast<const uint8_t*>(p.x) + m * p.x_stride * 2;
    q.ids = p.ids + m;
    const int64_t at = m * p.y_stride * (p.out == QGEMV_OUT_F32 ? 4 : 2);
    q.base = p.base ? static_cast<const uint8_t*>(p.base) + at : nullptr;
    q.y = static_cast<uint8_t*>(p.y) + at;
    const int64_t held = (q.rows + 15) / 16 * 16;
    work.row = reinterpret_cast<LoraRow*>(reinterpret_cast<uint8_t*>(h->ws) + held * row_bytes);
    work.rest = reinterpret_cast<float*>(work.row + held);
    if (!(bf ? launch_out<true>(*h, q, work, stream) : launch_out<false>(*h, q, work, stream))) return QGEMV_ERR_CUDA;
  }
  return QGEMV_OK;
}
