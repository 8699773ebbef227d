// fp4_i8.cuh -- inline-PTX wrappers of the signed 8-bit tensor-core MMA (tcgen05 kind::i8).
#pragma once

#include "fp4_ptx.cuh"

namespace fp4 {

// D (+)= A * B^T in signed 8-bit integers with 32-bit integer sums, K = 32 per instruction.
__device__ __forceinline__ void tc_mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t"
      "}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// M = 256 over a CTA pair: A rows 0..127 and B rows 0..N/2-1 from the leader's shared memory, the
// rest from the peer's; D rows split the same way.
__device__ __forceinline__ void tc_mma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t"
      "}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of the kind::i8 MMA: signed 8-bit A and B (1 in bits 7..9 and 10..12),
// K-major, 32-bit integer sums (2 in bits 4..5), N / 8, M / 16.
__host__ __device__ __forceinline__ uint32_t mma_idesc_i8(int n, int m = 128) {
  return 2u << 4 | 1u << 7 | 1u << 10 | (static_cast<uint32_t>(n) >> 3) << 17 | (static_cast<uint32_t>(m) >> 4) << 24;
}

}  // namespace fp4
