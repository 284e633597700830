// The handle behind qgemv_handle_t, shared by the files that implement its entry points.
#pragma once
#include <cstddef>
#include <cstdint>

#include "../../include/qgemv.h"

namespace qg {

constexpr size_t kWsFloats = size_t{4} << 20;    // split-K column sums: N * K-columns <= 4 Mi
constexpr int kMaxRanges = 1024;                 // split-K row ranges (one counter each)

struct Handle {
  int device = 0;
  int sms = 0;
  int l2_bytes = 0;
  size_t smem_optin = 0;
  int* err = nullptr;
  float* ws = nullptr;  // split-K column sums
  int* cnt = nullptr;   // split-K per-range arrival counts, zero between launches
  int ctas_per_sm = 2;
  int ksplit = 0;       // 0: split K-columns over CTAs when the workspace holds them; 1: never
  int grid_per_sm = 0;  // CTAs launched per SM (0: as many as fit, ctas_per_sm)
  size_t dyn_smem_max[6][3][3] = {};  // [format][R 1/2/4][D 2/3/4]
  size_t group_smem_max[2][3] = {};   // mixed-format grouped kernel [R 2/4][D 2/3/4]
  size_t group1_smem_max[6][2][2][3] = {};  // one-format grouped kernels [format][pairs][R 2/4][D 2/3/4]
  size_t batch_smem_max[6][2] = {};          // small-batch kernels [format][D 2/3]
  void* encode_tiled = nullptr;              // the driver's cuTensorMapEncodeTiled (null: no TMA path)
  int tc_cluster_max[3] = {1, 1, 1};         // largest cluster (K splits) the GEMM kernels can run [BT 64/128/256]
  int force_path = 0;
  int ring_depth = 0;
  int rows_per_stage = 0;
  uint64_t spin_ns = 1000000000ull;
  int pdl = 0;
  int test_stall = 0;
};

inline Handle* handle_of(qgemv_handle_t h) { return reinterpret_cast<Handle*>(h); }

}  // namespace qg
