// fp4_rows.cuh -- helpers shared by the row kernels around the GEMM (layer norm and the
// activation's backward pass): vector loads and stores of FP32 / BF16 rows, block scales and
// codes of values held in registers, and launches with programmatic dependency.
#pragma once

#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp4_codes.cuh"
#include "fp4_internal.h"
#include "fp4_ptx.cuh"

namespace fp4 {

// Programmatic dependent launch.  A kernel lets the next one start only after its own wait: a
// product whose weights are ready reads them without waiting, as they were written before the
// kernel just before it, and so everything older than that kernel has to be finished by then.
// (With the calls the other way round, act_backward writing a weight's codes, layer norm, then
// such a product read the old codes in 159 of 200 runs.)
__device__ __forceinline__ void rows_allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void rows_wait_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// V consecutive elements of a row as they lie in memory: one 16-byte word (V = 8 BF16 or 4
// FP32), or, for rows that do not start at 16 bytes, a pair (V = 2: even lengths) or a single
// element.
template <typename T, int V>
struct RowVec {
  static constexpr int kWords = V == 1 ? 1 : V * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // data read once: kept out of L1.  (Not the read-only path: an output may stand in an
  // input's place.)
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      if constexpr (sizeof(T) == 4) w[0] = *reinterpret_cast<const unsigned*>(p);
      else w[0] = *reinterpret_cast<const unsigned short*>(p);
    } else if constexpr (V == 2 && sizeof(T) == 2) {
      w[0] = *reinterpret_cast<const unsigned*>(p);
    } else if constexpr (V == 2) {
      const uint2 t = *reinterpret_cast<const uint2*>(p);
      w[0] = t.x;
      w[1] = t.y;
    } else {
      static_assert(V * sizeof(T) == 16, "one 16-byte word");
      asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "l"(p));
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
      v[0] = __uint_as_float(w[0] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};

__device__ __forceinline__ uint32_t rows_pack_bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Stores V values at element offset `off` of a BF16 or FP32 matrix (streaming: the output is
// not read back here).  V > 1: off is a multiple of V and the matrix 16-byte aligned.
template <int V>
__device__ __forceinline__ void store_row_vec(void* out, int out_bf16, int64_t off, const float (&v)[V]) {
  if constexpr (V == 1) {
    if (out_bf16) static_cast<__nv_bfloat16*>(out)[off] = __float2bfloat16_rn(v[0]);
    else static_cast<float*>(out)[off] = v[0];
  } else if (out_bf16) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = rows_pack_bf16x2(v[2 * i], v[2 * i + 1]);
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(out) + off;
    if constexpr (V == 8) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else if constexpr (V == 4) __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    else __stcs(reinterpret_cast<unsigned*>(p), w[0]);
  } else if constexpr (V == 2) {
    __stcs(reinterpret_cast<float2*>(static_cast<float*>(out) + off), make_float2(v[0], v[1]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + off);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) __stcs(p + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
  }
}

// V FP32 parameters (weights, biases): re-read by every row, so cached.
template <int V>
__device__ __forceinline__ void load_params(const float* p, float (&v)[V]) {
  if constexpr (V == 1) {
    v[0] = __ldg(p);
  } else if constexpr (V == 2) {
    const float2 f = __ldg(reinterpret_cast<const float2*>(p));
    v[0] = f.x;
    v[1] = f.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + i));
      v[i] = f.x;
      v[i + 1] = f.y;
      v[i + 2] = f.z;
      v[i + 3] = f.w;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

__device__ __forceinline__ uint32_t abs_bits_of(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Block formats a row kernel can write its result in, besides or instead of FP32 / BF16.
enum { kCodesNone = 0, kCodesNv = 1, kCodesMx = 2 };

struct RowCodes {
  uint8_t* codes;     // [rows, cols / 2]
  uint8_t* scales;    // 128 x 4 atoms
  const float* g;     // NVFP4: the caller's global scale
  int64_t cols;       // columns of the coded matrix
  int64_t atoms;      // scale atoms per 128-row block
};

// Encodes V (4 or 8) values of columns [col, col + V) of row `row`; the lanes of a block's
// 16 (NVFP4) or 32 (MXFP4) columns are neighbours and combine its maximum by shuffles.  Every
// lane of the warp calls it; `ok` says whether the lane's columns exist.  The same FP32 steps
// as the quantize kernels, so the codes are those of quantizing the values as FP32.
// Returns whether the block holds a non-finite value.
template <int FMT, int V>
__device__ __forceinline__ bool encode_row_vec(const RowCodes& c, float g, int64_t row, int64_t col, bool ok,
                                               const float (&v)[V]) {
  static_assert(V == 4 || V == 8, "one 16-byte word of FP32 or BF16 input");
  constexpr int BLOCK = FMT == kCodesMx ? 32 : 16;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, abs_bits_of(v[i]));
#pragma unroll
  for (int d = 1; d < BLOCK / V; d <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
  uint32_t sb;
  float mul;
  if constexpr (FMT == kCodesMx) {
    sb = e8m0_code(__fdiv_rn(__uint_as_float(m), 6.0f));
    mul = e8m0_inverse(sb);
  } else {
    mul = nvfp4_block_scale(__uint_as_float(m), g, sb);
  }
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = v[i] == 0.0f ? v[i] : __fmul_rn(v[i], mul);  // 1/denom may have overflowed
  if (ok) {
    uint8_t* dst = c.codes + row * (c.cols / 2) + col / 2;
    if constexpr (V == 8) *reinterpret_cast<uint32_t*>(dst) = pack8<kE2M1Hardware>(s);
    else *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(pack4<kE2M1Hardware>(s));
    if (col % BLOCK == 0) {
      const int64_t k = col / BLOCK;
      c.scales[((row / 128) * c.atoms + k / 4) * 512 + (row % 32) * 16 + ((row % 128) / 32) * 4 + k % 4] =
          static_cast<uint8_t>(sb);
    }
  }
  return ok && m >= 0x7F800000u;
}

template <typename... KArgs, typename... Args>
static cudaError_t launch_rows(void (*kern)(KArgs...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                               Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

}  // namespace fp4
