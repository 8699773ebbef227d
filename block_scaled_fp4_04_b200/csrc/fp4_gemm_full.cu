// fp4_gemm_full.cu -- the GEMM kernels with the long epilogue of fp4_gemm_epilogue_ex: any
// activation, a residual, a copy of the pre-activation (kEpiFull in fp4_gemm_kernel.cuh).
#include "fp4_gemm_host.h"

namespace fp4 {

template <bool MX>
static cudaError_t dispatch_full_t(const Plan& pl, const GemmMaps& tm, const GemmArgs& a, cudaStream_t st) {
  if (pl.BN >= 128 && pl.mode != kModeStreamK && a.sectors && a.Nk % 16 == 0) {
    if (pl.BN == 128) return run<128, MX, 2, false, false, kEpiFullWhole>(tm, a, pl.units, st);
    return pl.pair ? run<256, MX, 1, true, false, kEpiFullWhole>(tm, a, pl.units, st)
                   : run<256, MX, 1, false, false, kEpiFullWhole>(tm, a, pl.units, st);
  }
  if constexpr (MX) {  // (up to 32 rows of NVFP4 take the decode kernel, or stay in place)
    if (pl.BN == 16) return run<16, MX, 2, false, false, kEpiFull>(tm, a, pl.units, st);
    if (pl.BN == 32) return run<32, MX, 2, false, false, kEpiFull>(tm, a, pl.units, st);
  }
  switch (pl.BN) {
    case 64: return run<64, MX, 2, false, false, kEpiFull>(tm, a, pl.units, st);
    case 128: return run<128, MX, 2, false, false, kEpiFull>(tm, a, pl.units, st);
    default:
      return pl.pair ? run<256, MX, 1, true, false, kEpiFull>(tm, a, pl.units, st)
                     : run<256, MX, 1, false, false, kEpiFull>(tm, a, pl.units, st);
  }
}

cudaError_t dispatch_full(const Plan& pl, int mx, const GemmMaps& tm, const GemmArgs& a, cudaStream_t st) {
  return mx ? dispatch_full_t<true>(pl, tm, a, st) : dispatch_full_t<false>(pl, tm, a, st);
}

}  // namespace fp4
