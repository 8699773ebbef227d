// fp4_gemm_host.h -- host side of the GEMM that its translation units share: tensor maps, the
// plan of a problem, and the launches of the longer epilogues.
#pragma once

#include "fp4_gemm_kernel.cuh"
#include "fp4_ops.h"

namespace fp4 {

// A scale-factor buffer as a tensor map of 256-byte rows (CTA pairs load the atoms with it).
bool make_sf_map(CUtensorMap* m, const void* base, uint64_t bytes, uint32_t box_rows);

struct Plan {
  bool swap;
  bool pair;  // 256 x 256 tiles on CTA pairs
  int BN, ACC, mode;
  int64_t Mk, Nk;
  int tiles_m, tiles_n, num_kb;
  int64_t units;
  size_t ws_bytes;
};
Plan make_plan(int64_t M, int64_t N, int64_t K, int groups, int mx, bool row_major_out = false);

// Launches a planned product with the kEpiFull epilogue (fp4_gemm_full.cu).
cudaError_t dispatch_full(const Plan& pl, int mx, const GemmMaps& tm, const GemmArgs& a, cudaStream_t st);

}  // namespace fp4
