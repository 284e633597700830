// Entry point of the 8-bit projection.  See include/qgemv.h.
#include "qgemm_scaled.cuh"

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "qgemv_handle.cuh"
#include "qgemv_serve.cuh"

namespace qg {

namespace {

const void* few_kernel_for(int BT) {
  return BT > 32   ? reinterpret_cast<const void*>(scaled_few_kernel<64>)
         : BT > 16 ? reinterpret_cast<const void*>(scaled_few_kernel<32>)
                   : reinterpret_cast<const void*>(scaled_few_kernel<16>);
}
const void* many_kernel_for(int BN, bool join) {
  if (join) return BN == 128 ? reinterpret_cast<const void*>(scaled_many_kernel<128, true>) : reinterpret_cast<const void*>(scaled_many_kernel<256, true>);
  return BN == 128 ? reinterpret_cast<const void*>(scaled_many_kernel<128, false>) : reinterpret_cast<const void*>(scaled_many_kernel<256, false>);
}
int few_index(int BT) { return BT > 32 ? 2 : BT > 16 ? 1 : 0; }

}  // namespace

// How many clusters of each size run at once, asked once for a handle.
bool scaled_prepare(Handle& h) {
  auto clusters = [](const void* fn, int threads, size_t smem, int ctas) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) cudaGetLastError(), n = 0;
    return n;
  };
  // the many rows' kernels share out the registers they are launched with: of fewer, the share that grows would be waited for for ever
  auto registers = [](const void* fn) {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, fn) == cudaSuccess && fa.numRegs * (1 + kManyParts) >= kManyRegs[0] + kManyParts * kManyRegs[1];
  };
  auto prepare = [](const void* fn, size_t smem) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) == cudaSuccess;
  };
  for (int BT : {16, 32, 64}) {
    if (!prepare(few_kernel_for(BT), few_smem_bytes(BT))) return false;
    // the answer counts a single CTA to an SM, as of every kernel that allocates tensor memory; these take half of it at most, and
    // two are there at a time
    for (int ks = 2; ks <= 8; ++ks) h.scaled_clusters[few_index(BT)][ks] = 2 * clusters(few_kernel_for(BT), few_threads(BT), few_smem_bytes(BT), ks);
  }
  for (int BN : {128, 256}) {
    if (!registers(many_kernel_for(BN, false)) || !registers(many_kernel_for(BN, true))) return false;
    if (!prepare(many_kernel_for(BN, false), many_smem_bytes(BN)) || !prepare(many_kernel_for(BN, true), many_smem_bytes(BN))) return false;
    for (int ks = 2; ks <= kManyMaxPairs; ++ks) h.scaled_pairs[BN / 256][ks] = clusters(many_kernel_for(BN, true), kManyThreads, many_smem_bytes(BN), 2 * ks);
  }
  return true;
}

}  // namespace qg

using namespace qg;

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Rows of K bytes at `stride`, read in boxes of 128 bytes x `box_rows` with the 128-byte swizzle.
bool encode(const Handle& h, const void* at, int64_t rows, int64_t K, int64_t stride, int box_rows, CUtensorMap* map) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {kScaledBlock, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return reinterpret_cast<EncodeFn>(h.encode_tiled)(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(at), dims, strides, box, estr,
                                                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The launch for a shape: tiles of `columns` weight rows by `rows` rows of x, each shared by ks CTAs (of many rows: pairs of CTAs).
struct ScaledPlan {
  bool many;
  int rows, columns, ks;
  int64_t tiles, ctas;
};

ScaledPlan plan_few(const Handle& h, int64_t M, int64_t N, int64_t blocks) {
  ScaledPlan pl{false, M <= 16 ? 16 : M <= 32 ? 32 : 64, kScaledRows, 1, (N + kScaledRows - 1) / kScaledRows, 0};
  // the largest cluster with which all tiles run at once, of two blocks a CTA at least
  const int* most = h.scaled_clusters[few_index(pl.rows)];
  for (int ks = 2; ks <= 8; ++ks)
    if (pl.tiles <= most[ks] && blocks >= 2 * ks) pl.ks = ks;
  pl.ctas = pl.tiles * pl.ks;
  return pl;
}

ScaledPlan plan_many(const Handle& h, int64_t M, int64_t N, int64_t blocks) {
  ScaledPlan pl{true, kManyRows, 256, 1, 0, 0};
  const int64_t x_tiles = (M + kManyRows - 1) / kManyRows;
  // What takes the least time, in units of 0.065 us: rounds of tiles, a pair to each, or fewer tiles than pairs with their blocks
  // shared in clusters and joined.  A block of 128 weight rows takes 4 units and one of 256 6, the end of a tile 14 or 28, a join
  // 33 or 58.  128 x 4096 x 14336: 21.0 us with 128 rows and two pairs to a tile, 33.2 with one, 25.5 with 256 rows and three
  // pairs; 512 x 4096 x 4096: 13.1 with 128 rows alone, 16.4 with 256 and two pairs; 300 x 4096 x 14336: 31.8 with 256 and two pairs,
  // 33.1 with 128; 4096 x 28672 x 4096: 359 with 256, 430 with 128.
  const int64_t pairs = std::max(1, h.sms / 2), fours = (blocks + 3) / 4;
  double least = 0.;
  for (int bn : {256, 128}) {
    const int64_t tiles = x_tiles * ((N + bn - 1) / bn), block = bn == 256 ? 6 : 4, end = bn == 256 ? 28 : 14, join = bn == 256 ? 58 : 33;
    for (int ks = 1; ks <= kManyMaxPairs; ++ks) {
      if (ks > 1 && (tiles > h.scaled_pairs[bn / 256][ks] || fours < ks)) continue;
      const int64_t rounds = ks > 1 ? 1 : (tiles + pairs - 1) / pairs, each = ks > 1 ? (fours + ks - 1) / ks * 4 : blocks;
      const double cost = static_cast<double>(rounds) * static_cast<double>(each * block + end) + (ks > 1 ? join : 0);
      if (least == 0. || cost < least) least = cost, pl.columns = bn, pl.ks = ks;
    }
  }
  pl.tiles = x_tiles * ((N + pl.columns - 1) / pl.columns);
  pl.ctas = 2 * pl.ks * (pl.ks > 1 ? pl.tiles : std::min<int64_t>(pl.tiles, pairs));
  return pl;
}

// The plan of a valid shape with rows.
qgemv_status_t plan_scaled(const Handle& h, int64_t M, int64_t N, int64_t K, ScaledPlan& pl) {
  const int64_t blocks = (K + kScaledBlock - 1) / kScaledBlock;
  pl = M > 64 ? plan_many(h, M, N, blocks) : plan_few(h, M, N, blocks);
  return pl.tiles > 0x7fffffff ? QGEMV_ERR_BAD_SHAPE : QGEMV_OK;
}

bool shape_ok(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t most = 0x7fffffff;
  return M >= 0 && M <= most && N >= 1 && N <= most && K >= 16 && K <= most && K % 16 == 0;
}

qgemv_status_t launch(const Handle& h, const qgemv_scaled_t& p, const ScaledPlan& pl, ScaledArgs a, cudaStream_t stream) {
  CUtensorMap wmap, xmap;
  if (!encode(h, p.W, p.N, p.K, p.K, pl.many ? pl.columns / 2 : kScaledRows, &wmap) ||
      !encode(h, p.x, p.M, p.K, p.x_stride, pl.many ? kManyRows / 2 : pl.rows, &xmap))
    return QGEMV_ERR_CUDA;
  a.ks = pl.ks;
  void* args[] = {&wmap, &xmap, &a};
  const dim3 grid(static_cast<unsigned>(pl.ctas));
  const bool ok = pl.many ? launch_dependent(many_kernel_for(pl.columns, pl.ks > 1), grid, kManyThreads, many_smem_bytes(pl.columns), 2 * pl.ks, args, stream)
                          : launch_dependent(few_kernel_for(pl.rows), grid, few_threads(pl.rows), few_smem_bytes(pl.rows), pl.ks, args, stream);
  return ok ? QGEMV_OK : QGEMV_ERR_CUDA;
}

}  // namespace

extern "C" qgemv_status_t qgemv_run_scaled(qgemv_handle_t hh, const qgemv_scaled_t* scaled, cudaStream_t stream) {
  const Handle* h = handle_of(hh);
  if (!h || !scaled) return QGEMV_ERR_INVALID_ARG;
  const qgemv_scaled_t& p = *scaled;
  if (p.out != QGEMV_OUT_F32 && p.out != QGEMV_OUT_F16 && p.out != QGEMV_OUT_BF16) return QGEMV_ERR_INVALID_ARG;
  constexpr int64_t far = int64_t{1} << 38;
  if (!shape_ok(p.M, p.N, p.K) || p.x_stride < p.K || p.x_stride > far || p.x_scale_stride < (p.K + 127) / 128 || p.x_scale_stride > far ||
      p.y_stride < p.N || p.y_stride > far)
    return QGEMV_ERR_BAD_SHAPE;
  if (!p.W || !p.w_scale || (p.M > 0 && (!p.x || !p.x_scale || !p.y))) return QGEMV_ERR_INVALID_ARG;
  if (!aligned16(p.x) || !aligned16(p.W) || !aligned16(p.y) || p.x_stride % 16 ||
      ((reinterpret_cast<uintptr_t>(p.x_scale) | reinterpret_cast<uintptr_t>(p.w_scale)) & 3))
    return QGEMV_ERR_MISALIGNED;
  if (p.M == 0) return QGEMV_OK;
  if (!h->encode_tiled) return QGEMV_ERR_CUDA;  // no TMA descriptors from this driver
  ScaledPlan pl;
  const qgemv_status_t st = plan_scaled(*h, p.M, p.N, p.K, pl);
  if (st != QGEMV_OK) return st;
  ScaledArgs a{};
  a.xs = p.x_scale;
  a.ws = p.w_scale;
  a.y = p.y;
  a.xs_stride = p.x_scale_stride;
  a.y_stride = p.y_stride;
  a.M = static_cast<int>(p.M);
  a.N = static_cast<int>(p.N);
  a.blocks = static_cast<int>((p.K + kScaledBlock - 1) / kScaledBlock);
  a.out = p.out;
  a.err = h->err;
  a.spin_ns = h->spin_ns;
  a.early = h->pdl;
  a.stall = h->test_stall;
  a.x_tiles = static_cast<int>((p.M + kManyRows - 1) / kManyRows);
  a.wide = a.blocks % 4 == 0 && p.x_scale_stride % 4 == 0 && aligned16(p.x_scale) && aligned16(p.w_scale);
  return launch(*h, p, pl, a, stream);
}

extern "C" qgemv_status_t qgemv_describe_scaled(qgemv_handle_t hh, int64_t M, int64_t N, int64_t K, char* buf, size_t len) {
  const Handle* h = handle_of(hh);
  if (!h) return QGEMV_ERR_INVALID_ARG;
  if (!shape_ok(M, N, K)) return QGEMV_ERR_BAD_SHAPE;
  ScaledPlan pl{};
  const qgemv_status_t st = M > 0 ? plan_scaled(*h, M, N, K, pl) : QGEMV_OK;
  if (st != QGEMV_OK || !buf || !len) return st;
  if (M == 0)
    snprintf(buf, len, "path=none");
  else
    snprintf(buf, len, "path=%s rows=%d columns=%d share=%d tiles=%lld ctas=%lld", pl.many ? "many" : "few", pl.rows, pl.columns, pl.ks,
             static_cast<long long>(pl.tiles), static_cast<long long>(pl.ctas));
  return QGEMV_OK;
}
