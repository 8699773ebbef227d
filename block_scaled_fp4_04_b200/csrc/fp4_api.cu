// fp4_api.cu -- the extern "C" entry points declared in include/fp4.h: argument
// checks, workspace sizing, the per-device status word, and kernel launches.
#include <cuda_runtime.h>
#include <cstdint>
#include <cstdio>
#include <mutex>

#include "fp4.h"
#include "fp4_internal.h"
#include "fp4_moe.h"
#include "fp4_ops.h"
#include "fp4_ptx.cuh"

namespace fp4 {

// Latched device-side errors (kStatusNonFinite, kStatusTimeout); one word per device.
__device__ unsigned g_status_word;

static thread_local char g_err[256];

static fp4_status fail(fp4_status s, const char* msg) {
  snprintf(g_err, sizeof(g_err), "%s", msg);
  return s;
}

static fp4_status cuda_fail(cudaError_t e, const char* where) {
  snprintf(g_err, sizeof(g_err), "%s: %s", where, cudaGetErrorString(e));
  return FP4_ERR_CUDA;
}

constexpr int kMaxDevices = 64;

int num_sms() {
  static int cache[kMaxDevices] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= kMaxDevices) return 148;
  if (!cache[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = n > 0 ? n : 148;
  }
  return cache[dev];
}

// Address of this device's status word, and a check that the device is an sm_100.
static fp4_status device_state(unsigned** status) {
  static unsigned* addr[kMaxDevices] = {nullptr};
  static int ok[kMaxDevices] = {0};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(FP4_ERR_UNSUPPORTED, "device index out of range");
  std::lock_guard<std::mutex> lock(mu);
  if (!ok[dev]) {
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (major != 10 || minor != 0) return fail(FP4_ERR_UNSUPPORTED, "libfp4 is built for sm_100a (B200) only");
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_status_word);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(status)");
    addr[dev] = static_cast<unsigned*>(p);
    ok[dev] = 1;
  }
  *status = addr[dev];
  return FP4_OK;
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
constexpr int64_t kMaxDim = (1ll << 31) - 256;  // rows, columns and tiles are counted in 32 bits

// Test hook (fp4_debug_stall_next_decode): the CTA whose amax share the next fused decode
// launch of this thread leaves unpublished, plus one (0: none).
static thread_local int g_stall_next_decode = 0;

}  // namespace fp4

using namespace fp4;

extern "C" {

const char* fp4_version(void) { return "libfp4 0.1 (sm_100a)"; }

const char* fp4_last_error(void) { return g_err; }

size_t fp4_scales_bytes(int64_t rows, int64_t cols, fp4_fmt fmt) {
  if (rows <= 0 || cols <= 0) return 0;
  const int64_t blk = fmt == FP4_MXFP4 || fmt == FP4_MXFP8 ? 32 : 16;
  const int64_t scols = (cols + blk - 1) / blk;
  return static_cast<size_t>(((rows + 127) / 128) * 128 * ((scols + 3) / 4) * 4);
}

size_t fp4_scales_bytes_grouped(int64_t total_rows, int num_groups, int64_t cols, fp4_fmt fmt) {
  if (total_rows < 0 || num_groups <= 0 || cols <= 0) return 0;
  const int64_t blk = fmt == FP4_MXFP4 ? 32 : 16;
  const int64_t scols = (cols + blk - 1) / blk;
  return static_cast<size_t>(((total_rows + 127) / 128 + num_groups) * 128 * ((scols + 3) / 4) * 4);
}

size_t fp4_quantize_workspace_size(void) { return kQuantWorkspaceBytes; }

fp4_status fp4_amax(const void* x, int64_t n, fp4_dtype in_dtype, float* amax_out, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!x || !amax_out || !workspace) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (n <= 0) return fail(FP4_ERR_INVALID_ARG, "n must be positive");
  if (in_dtype != FP4_F32 && in_dtype != FP4_BF16) return fail(FP4_ERR_INVALID_ARG, "in_dtype");
  if (!aligned16(x) || !aligned16(workspace)) return fail(FP4_ERR_INVALID_ARG, "x and workspace must be 16-byte aligned");
  if (!aligned4(amax_out)) return fail(FP4_ERR_INVALID_ARG, "amax_out alignment");
  if (workspace_bytes < kQuantWorkspaceBytes) return fail(FP4_ERR_INVALID_ARG, "workspace too small");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaError_t e = launch_amax(x, n, in_dtype == FP4_BF16, static_cast<uint32_t*>(workspace), amax_out, nullptr,
                              status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "amax launch");
}

static fp4_status quantize_common(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, fp4_fmt fmt,
                                  int block, uint8_t* codes, uint8_t* scales, float* gout, uint8_t* codesT,
                                  uint8_t* scalesT, const float* gin, void* ws, size_t ws_bytes, int num_groups,
                                  const int32_t* offsets, void* stream, int variant = kQuantPlain,
                                  const uint32_t* rbits = nullptr, uint32_t signs = 0) {
  if (!x || !codes || !scales) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (rows <= 0 || cols <= 0) return fail(FP4_ERR_INVALID_ARG, "rows and cols must be positive");
  if (cols % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "cols must be a multiple of 32");
  if (rows > kMaxDim) return fail(FP4_ERR_UNSUPPORTED, "rows too large");  // row offsets are int32
  if (in_dtype != FP4_F32 && in_dtype != FP4_BF16) return fail(FP4_ERR_INVALID_ARG, "in_dtype");
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4 && fmt != FP4_MXFP8) return fail(FP4_ERR_INVALID_ARG, "fmt");
  if (fmt == FP4_MXFP8) {
    if (block != 32) return fail(FP4_ERR_INVALID_ARG, "MXFP8 block must be 32");
    if (num_groups) return fail(FP4_ERR_UNSUPPORTED, "grouped MXFP8 quantization");
    if (variant != kQuantPlain) return fail(FP4_ERR_UNSUPPORTED, "quantizer variants are FP4 only");
    variant = kQuantFp8;
  }
  const bool two_d = block == 256;
  if (fmt == FP4_NVFP4 && block != 16 && block != 256) return fail(FP4_ERR_INVALID_ARG, "NVFP4 block must be 16 or 256");
  if (fmt == FP4_MXFP4 && block != 32) return fail(FP4_ERR_INVALID_ARG, "MXFP4 block must be 32");
  if (two_d && (!codesT || !scalesT)) return fail(FP4_ERR_INVALID_ARG, "block 256 needs codesT and scalesT");
  if (!two_d && (codesT || scalesT)) return fail(FP4_ERR_INVALID_ARG, "codesT/scalesT only for block 256");
  if (two_d && rows % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "block 256 needs rows % 32 == 0");
  if (two_d && num_groups) return fail(FP4_ERR_UNSUPPORTED, "grouped 2-D quantization");
  if (fmt == FP4_NVFP4 && !gout) return fail(FP4_ERR_INVALID_ARG, "NVFP4 needs global_out");
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || (codesT && !aligned16(codesT)) ||
      (scalesT && !aligned16(scalesT)))
    return fail(FP4_ERR_INVALID_ARG, "x, codes and scales must be 16-byte aligned");
  if (num_groups && (num_groups > kMaxGroups || !offsets)) return fail(FP4_ERR_INVALID_ARG, "groups / offsets");
  if (!aligned4(gout) || !aligned4(gin) || !aligned4(offsets))
    return fail(FP4_ERR_INVALID_ARG, "global scale / offsets alignment");
  if (variant != kQuantPlain && two_d) return fail(FP4_ERR_UNSUPPORTED, "quantizer variants are 1-D only");
  if (variant == kQuantMxFloor && fmt != FP4_MXFP4) return fail(FP4_ERR_INVALID_ARG, "the E8M0 floor is for MXFP4");
  if (variant == kQuantSR && (fmt != FP4_NVFP4 || !rbits || !aligned16(rbits)))
    return fail(FP4_ERR_INVALID_ARG, "stochastic rounding: NVFP4, 16-byte aligned random words");
  const bool need_amax = fmt == FP4_NVFP4 && !gin;
  if (need_amax && (!ws || ws_bytes < kQuantWorkspaceBytes || !aligned16(ws)))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small or misaligned (fp4_quantize_workspace_size)");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int bf16 = in_dtype == FP4_BF16;
  const int mx = fmt == FP4_MXFP4 || fmt == FP4_MXFP8;
  cudaError_t e = cudaSuccess;
  if (variant == kQuantPlain && !two_d && !num_groups && quantize_small_fits(rows, cols, bf16, mx)) {
    // one launch: amax, global scale and encode by one thread-block cluster
    e = launch_quantize_small(x, rows, cols, bf16, mx, codes, scales, mx ? nullptr : gin, gout, status, st);
    return e == cudaSuccess ? FP4_OK : cuda_fail(e, "quantize launch");
  }
  const float* g = nullptr;
  if (fmt == FP4_NVFP4) {
    if (need_amax) {
      e = launch_amax(x, rows * cols, bf16, static_cast<uint32_t*>(ws), nullptr, gout, status, st,
                      variant == kQuantRHT, signs);
      if (e != cudaSuccess) return cuda_fail(e, "amax launch");
      g = gout;
    } else {
      if (gout && gout != gin) {
        e = cudaMemcpyAsync(gout, gin, sizeof(float), cudaMemcpyDeviceToDevice, st);
        if (e != cudaSuccess) return cuda_fail(e, "global scale copy");
      }
      g = gin;
    }
  } else if (gout) {
    e = launch_set_value(gout, 1.0f, st);
    if (e != cudaSuccess) return cuda_fail(e, "global scale write");
  }
  if (two_d)
    e = launch_quantize_2d(x, rows, cols, bf16, codes, scales, codesT, scalesT, g, status, st);
  else
    e = launch_quantize_1d(x, rows, cols, bf16, mx, codes, scales, g, offsets, num_groups, status, st, variant, rbits,
                           signs);
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "quantize launch");
}

fp4_status fp4_quantize(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, fp4_fmt fmt, int block,
                        uint8_t* codes_out, uint8_t* scales_out, float* global_out, uint8_t* codesT_out,
                        uint8_t* scalesT_out, const float* global_in, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return quantize_common(x, rows, cols, in_dtype, fmt, block, codes_out, scales_out, global_out, codesT_out,
                         scalesT_out, global_in, workspace, workspace_bytes, 0, nullptr, stream);
}

fp4_status fp4_quantize_ex(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, fp4_fmt fmt, int block,
                           unsigned flags, uint8_t* codes_out, uint8_t* scales_out, float* global_out,
                           uint8_t* codesT_out, uint8_t* scalesT_out, const float* global_in, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (flags & ~static_cast<unsigned>(FP4_QUANT_E8M0_FLOOR)) return fail(FP4_ERR_INVALID_ARG, "unknown flag");
  return quantize_common(x, rows, cols, in_dtype, fmt, block, codes_out, scales_out, global_out, codesT_out,
                         scalesT_out, global_in, workspace, workspace_bytes, 0, nullptr, stream,
                         (flags & FP4_QUANT_E8M0_FLOOR) ? kQuantMxFloor : kQuantPlain);
}

fp4_status fp4_quantize_sr(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, const uint32_t* rbits,
                           uint8_t* codes_out, uint8_t* scales_out, float* global_out, const float* global_in,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return quantize_common(x, rows, cols, in_dtype, FP4_NVFP4, 16, codes_out, scales_out, global_out, nullptr, nullptr,
                         global_in, workspace, workspace_bytes, 0, nullptr, stream, kQuantSR, rbits, 0);
}

fp4_status fp4_quantize_rht(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, fp4_fmt fmt,
                            uint32_t signs, uint8_t* codes_out, uint8_t* scales_out, float* global_out,
                            const float* global_in, void* workspace, size_t workspace_bytes, void* stream) {
  if (signs > 0xFFFFu) return fail(FP4_ERR_INVALID_ARG, "signs: 16 bits");
  return quantize_common(x, rows, cols, in_dtype, fmt, fmt == FP4_MXFP4 ? 32 : 16, codes_out, scales_out, global_out,
                         nullptr, nullptr, global_in, workspace, workspace_bytes, 0, nullptr, stream, kQuantRHT,
                         nullptr, signs);
}

fp4_status fp4_global_scale(const float* amax, float* global_out, void* stream) {
  if (!amax || !global_out) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (!aligned4(amax) || !aligned4(global_out)) return fail(FP4_ERR_INVALID_ARG, "amax / global_out alignment");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  const cudaError_t e = launch_global_scale(amax, global_out, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "global scale launch");
}

fp4_status fp4_quantize_grouped(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, fp4_fmt fmt,
                                int num_groups, const int32_t* offsets, uint8_t* codes_out, uint8_t* scales_out,
                                float* global_out, const float* global_in, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (num_groups <= 0) return fail(FP4_ERR_INVALID_ARG, "num_groups must be positive");
  return quantize_common(x, rows, cols, in_dtype, fmt, fmt == FP4_NVFP4 ? 16 : 32, codes_out, scales_out,
                         global_out, nullptr, nullptr, global_in, workspace, workspace_bytes, num_groups, offsets,
                         stream);
}

fp4_status fp4_dequantize(const uint8_t* codes, const uint8_t* scales, const float* global, int64_t rows,
                          int64_t cols, fp4_fmt fmt, float* out, void* stream) {
  if (!codes || !scales || !out) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (!aligned4(global) || !aligned4(out)) return fail(FP4_ERR_INVALID_ARG, "global / out alignment");
  if (rows <= 0 || cols <= 0 || cols % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "shape");
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return fail(FP4_ERR_INVALID_ARG, "fmt");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaError_t e = launch_dequantize(codes, scales, fmt == FP4_NVFP4 ? global : nullptr, rows, cols,
                                    fmt == FP4_MXFP4, out, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "dequantize launch");
}

size_t fp4_gemm_workspace_size(int64_t M, int64_t N, int64_t K, fp4_fmt fmt) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return gemm_workspace_bytes(M, N, K, fmt == FP4_MXFP4);
}

// What every dense or grouped product needs of its arguments.
static fp4_status gemm_check(const GemmProblem& g, fp4_fmt fmt, fp4_dtype out_dtype) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return fail(FP4_ERR_INVALID_ARG, "fmt");
  if (out_dtype != FP4_F32 && out_dtype != FP4_BF16) return fail(FP4_ERR_INVALID_ARG, "out_dtype");
  if (!g.A || !g.B || !g.sA || !g.sB || (!g.D && !g.q_codes)) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (g.M <= 0 || g.N <= 0 || g.K <= 0) return fail(FP4_ERR_INVALID_ARG, "M, N, K must be positive");
  if (g.K % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "K must be a multiple of 32");
  if (g.M > kMaxDim || g.N > kMaxDim || g.K > kMaxDim) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (g.num_groups > 0 && g.N > kMaxDim / g.num_groups) return fail(FP4_ERR_UNSUPPORTED, "too many weight rows");
  if (!aligned16(g.A) || !aligned16(g.B) || !aligned16(g.sA) || !aligned16(g.sB) || (g.D && !aligned16(g.D)))
    return fail(FP4_ERR_INVALID_ARG, "A, B, scales and D must be 16-byte aligned");
  if (!aligned4(g.gA) || !aligned4(g.gB) || !aligned4(g.q_g) || !aligned4(g.offsets))
    return fail(FP4_ERR_INVALID_ARG, "global scale / offsets alignment");
  return FP4_OK;
}

// Whether the workspace stands where the kernels' widest access to it can.
static bool workspace_aligned(const GemmProblem& g) {
  return aligned16(g.ws) ||
         reinterpret_cast<uintptr_t>(g.ws) %
                 gemm_workspace_align(g.M, g.N, g.K, g.mx, g.q_codes != nullptr || g.amax_out != nullptr) ==
             0;
}

static fp4_status gemm_common(const GemmProblem& g, fp4_fmt fmt, fp4_dtype out_dtype, void* stream,
                              const GemmFull* full = nullptr) {
  const fp4_status c = gemm_check(g, fmt, out_dtype);
  if (c != FP4_OK) return c;
  if (!g.num_groups && !workspace_aligned(g)) return fail(FP4_ERR_INVALID_ARG, "workspace alignment");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  const char* why = nullptr;
  cudaError_t err = cudaSuccess;
  const int rc = launch_gemm_full(GemmProblemFull{g, full}, status, static_cast<cudaStream_t>(stream), &why, &err);
  if (rc == 1) return fail(FP4_ERR_INVALID_ARG, why);
  if (rc == 2) return cuda_fail(err, "gemm launch");
  return FP4_OK;
}

static bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

fp4_status fp4_gemm_mixed(fp4_fmt a_fmt, const uint8_t* A, const uint8_t* sA, fp4_fmt b_fmt, const uint8_t* B,
                          const uint8_t* sB, int64_t M, int64_t N, int64_t K, void* D, fp4_dtype out_dtype,
                          void* stream) {
  if ((a_fmt != FP4_MXFP4 && a_fmt != FP4_MXFP8) || (b_fmt != FP4_MXFP4 && b_fmt != FP4_MXFP8))
    return fail(FP4_ERR_INVALID_ARG, "a_fmt and b_fmt must each be FP4_MXFP4 or FP4_MXFP8");
  if (out_dtype != FP4_F32 && out_dtype != FP4_BF16) return fail(FP4_ERR_INVALID_ARG, "out_dtype");
  if (!A || !B || !sA || !sB || !D) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (M <= 0 || N <= 0 || K <= 0) return fail(FP4_ERR_INVALID_ARG, "M, N, K must be positive");
  if (K % 128 != 0) return fail(FP4_ERR_INVALID_ARG, "K must be a multiple of 128");
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!aligned32(A) || !aligned32(B) || !aligned16(sA) || !aligned16(sB) || !aligned16(D))
    return fail(FP4_ERR_INVALID_ARG, "A and B must be 32-byte aligned, scales and D 16-byte aligned");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  GemmProblem g{};
  g.mx = 1;
  g.A = A;
  g.sA = sA;
  g.B = B;
  g.sB = sB;
  g.M = M;
  g.N = N;
  g.K = K;
  g.D = D;
  g.out_bf16 = out_dtype == FP4_BF16;
  const char* why = nullptr;
  cudaError_t err = cudaSuccess;
  const int rc = launch_gemm_mixed(g, a_fmt == FP4_MXFP8, b_fmt == FP4_MXFP8, status, static_cast<cudaStream_t>(stream),
                                   &why, &err);
  if (rc == 1) return fail(FP4_ERR_INVALID_ARG, why);
  if (rc == 2) return cuda_fail(err, "gemm launch");
  return FP4_OK;
}

fp4_status fp4_gemm_ex(fp4_fmt fmt, const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* B,
                       const uint8_t* sB, const float* gB, int64_t M, int64_t N, int64_t K, void* D,
                       fp4_dtype out_dtype, void* workspace, size_t workspace_bytes, unsigned flags,
                       void* stream) {
  if (flags & ~static_cast<unsigned>(FP4_GEMM_WEIGHTS_READY)) return fail(FP4_ERR_INVALID_ARG, "unknown flag");
  GemmProblem g{};
  g.mx = fmt == FP4_MXFP4;
  g.A = A;
  g.sA = sA;
  g.gA = gA;
  g.B = B;
  g.sB = sB;
  g.gB = gB;
  g.M = M;
  g.N = N;
  g.K = K;
  g.D = D;
  g.out_bf16 = out_dtype == FP4_BF16;
  g.ws = workspace;
  g.ws_bytes = workspace_bytes;
  g.weights_ready = (flags & FP4_GEMM_WEIGHTS_READY) ? 1 : 0;
  return gemm_common(g, fmt, out_dtype, stream);
}

fp4_status fp4_gemm(fp4_fmt fmt, const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* B,
                    const uint8_t* sB, const float* gB, int64_t M, int64_t N, int64_t K, void* D, fp4_dtype out_dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return fp4_gemm_ex(fmt, A, sA, gA, B, sB, gB, M, N, K, D, out_dtype, workspace, workspace_bytes, 0u, stream);
}

static bool act_ok(fp4_act act) { return act >= FP4_ACT_NONE && act <= FP4_ACT_GELU_TANH; }
static bool dtype_ok(fp4_dtype t) { return t == FP4_F32 || t == FP4_BF16; }

static fp4_status epilogue_common(fp4_fmt fmt, const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* B,
                                  const uint8_t* sB, const float* gB, int64_t M, int64_t N, int64_t K,
                                  const float* bias, fp4_act act, void* D, fp4_dtype out_dtype, uint8_t* Dcodes,
                                  uint8_t* Dscales, const float* gD, float* amax_out, void* workspace,
                                  size_t workspace_bytes, unsigned flags, void* stream, const GemmFull* full) {
  if (!D && !Dcodes) return fail(FP4_ERR_INVALID_ARG, "no output: D and Dcodes are both NULL");
  if (Dcodes && (!Dscales || !gD)) return fail(FP4_ERR_INVALID_ARG, "FP4 output needs Dscales and gD");
  if (Dcodes && N % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "FP4 output needs N % 32 == 0");
  if (Dcodes && (!aligned16(Dcodes) || !aligned16(Dscales))) return fail(FP4_ERR_INVALID_ARG, "Dcodes / Dscales alignment");
  if (bias && !aligned4(bias)) return fail(FP4_ERR_INVALID_ARG, "bias alignment");
  GemmProblem g{};
  g.mx = fmt == FP4_MXFP4;
  g.A = A;
  g.sA = sA;
  g.gA = gA;
  g.B = B;
  g.sB = sB;
  g.gB = gB;
  g.M = M;
  g.N = N;
  g.K = K;
  g.D = D;
  g.out_bf16 = out_dtype == FP4_BF16;
  g.ws = workspace;
  g.ws_bytes = workspace_bytes;
  g.weights_ready = (flags & FP4_GEMM_WEIGHTS_READY) ? 1 : 0;
  g.bias = bias;
  g.act = act;
  g.q_codes = Dcodes;
  g.q_scales = Dscales;
  g.q_g = gD;
  g.amax_out = amax_out;
  if (!aligned4(amax_out)) return fail(FP4_ERR_INVALID_ARG, "amax_out alignment");
  // every check before the first thing is enqueued
  const fp4_status c = gemm_check(g, fmt, out_dtype);
  if (c != FP4_OK) return c;
  const size_t need = full ? gemm_full_workspace_bytes(M, N, K, g.mx, Dcodes || amax_out)
                           : gemm_workspace_bytes(M, N, K, g.mx, Dcodes || amax_out);
  if (need && (!workspace || workspace_bytes < need))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small (see fp4_gemm_epilogue_workspace_size)");
  if (full ? need && !aligned16(workspace) : !workspace_aligned(g))
    return fail(FP4_ERR_INVALID_ARG, "workspace alignment");
  if (amax_out) {
    const cudaError_t e = cudaMemsetAsync(amax_out, 0, sizeof(float), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "zeroing amax_out");
  }
  if (Dcodes && (M % 128 != 0 || (N / 16) % 4 != 0)) {
    // the kernel writes the scale bytes of real rows and blocks; the layout's pad bytes
    // (rows up to a multiple of 128, block columns up to a multiple of 4) must read as 0
    const cudaError_t e =
        cudaMemsetAsync(Dscales, 0, fp4_scales_bytes(M, N, FP4_NVFP4), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "zero-filling the scale pads");
  }
  return gemm_common(g, fmt, out_dtype, stream, full);
}

fp4_status fp4_gemm_epilogue(fp4_fmt fmt, const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* B,
                             const uint8_t* sB, const float* gB, int64_t M, int64_t N, int64_t K, const float* bias,
                             fp4_act act, void* D, fp4_dtype out_dtype, uint8_t* Dcodes, uint8_t* Dscales,
                             const float* gD, float* amax_out, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (act != FP4_ACT_NONE && act != FP4_ACT_RELU) return fail(FP4_ERR_INVALID_ARG, "act");
  return epilogue_common(fmt, A, sA, gA, B, sB, gB, M, N, K, bias, act, D, out_dtype, Dcodes, Dscales, gD, amax_out,
                         workspace, workspace_bytes, 0u, stream, nullptr);
}

fp4_status fp4_gemm_epilogue_ex(fp4_fmt fmt, const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* B,
                                const uint8_t* sB, const float* gB, int64_t M, int64_t N, int64_t K, const float* bias,
                                fp4_act act, const void* residual, fp4_dtype residual_dtype, void* D,
                                fp4_dtype out_dtype, void* pre, uint8_t* Dcodes, uint8_t* Dscales, const float* gD,
                                float* amax_out, void* workspace, size_t workspace_bytes, unsigned flags,
                                void* stream) {
  if (!act_ok(act)) return fail(FP4_ERR_INVALID_ARG, "act");
  if (flags & ~static_cast<unsigned>(FP4_GEMM_WEIGHTS_READY)) return fail(FP4_ERR_INVALID_ARG, "unknown flag");
  if (residual && !dtype_ok(residual_dtype)) return fail(FP4_ERR_INVALID_ARG, "residual_dtype");
  if (!aligned16(residual) || !aligned16(pre)) return fail(FP4_ERR_INVALID_ARG, "residual and pre must be 16-byte aligned");
  if (residual && residual == D && residual_dtype != out_dtype)
    return fail(FP4_ERR_INVALID_ARG, "a residual in D's place needs D's type");
  if (pre && (pre == D || pre == residual)) return fail(FP4_ERR_INVALID_ARG, "pre must be a buffer of its own");
  const GemmFull full{residual, residual_dtype == FP4_BF16, pre};
  // scale, bias and ReLU alone are the plain epilogue
  const bool plain = !residual && !pre && (act == FP4_ACT_NONE || act == FP4_ACT_RELU);
  return epilogue_common(fmt, A, sA, gA, B, sB, gB, M, N, K, bias, act, D, out_dtype, Dcodes, Dscales, gD, amax_out,
                         workspace, workspace_bytes, flags, stream, plain ? nullptr : &full);
}

size_t fp4_gemm_gated_workspace_size(int64_t M, int64_t F, int64_t K, fp4_fmt fmt, int rows_in_place) {
  if (M <= 0 || F <= 0 || K <= 0) return 0;
  return gated_workspace_bytes(M, F, K, fmt == FP4_MXFP4, rows_in_place != 0);
}

// Checks what every gated product needs; launches it.
static fp4_status gated_common(GatedProblem& g, fp4_fmt fmt, fp4_act act, fp4_dtype out_dtype, void* stream) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return fail(FP4_ERR_INVALID_ARG, "fmt");
  if (!dtype_ok(out_dtype)) return fail(FP4_ERR_INVALID_ARG, "out_dtype");
  if (!act_ok(act)) return fail(FP4_ERR_INVALID_ARG, "act");
  if (!g.A || !g.sA || !g.Wg || !g.sWg || !g.Wu || !g.sWu) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (!g.H && !g.q_codes) return fail(FP4_ERR_INVALID_ARG, "no output: H and Hcodes are both NULL");
  if (!g.G != !g.U) return fail(FP4_ERR_INVALID_ARG, "G and U: both or neither");
  if (g.G && (g.G == g.U || g.G == g.H || g.U == g.H)) return fail(FP4_ERR_INVALID_ARG, "H, G and U must be different buffers");
  if (g.M <= 0 || g.F <= 0 || g.K <= 0) return fail(FP4_ERR_INVALID_ARG, "M, F, K must be positive");
  if (g.K % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "K must be a multiple of 32");
  if (g.M > kMaxDim || g.F > kMaxDim || g.K > kMaxDim) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (g.num_groups > 0 && g.F > kMaxDim / g.num_groups) return fail(FP4_ERR_UNSUPPORTED, "too many weight rows");
  if (!aligned16(g.A) || !aligned16(g.sA) || !aligned16(g.Wg) || !aligned16(g.sWg) || !aligned16(g.Wu) ||
      !aligned16(g.sWu) || !aligned16(g.H) || !aligned16(g.G) || !aligned16(g.U))
    return fail(FP4_ERR_INVALID_ARG, "A, weights, scales, H, G and U must be 16-byte aligned");
  if (!aligned4(g.bias_g) || !aligned4(g.bias_u)) return fail(FP4_ERR_INVALID_ARG, "bias alignment");
  if (!aligned4(g.gA) || !aligned4(g.gWg) || !aligned4(g.gWu) || !aligned4(g.q_g) || !aligned4(g.offsets))
    return fail(FP4_ERR_INVALID_ARG, "global scale / offsets alignment");
  if (g.q_codes && (!g.q_scales || !g.q_g)) return fail(FP4_ERR_INVALID_ARG, "FP4 output needs Hscales and gH");
  if (g.q_codes && g.F % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "FP4 output needs F % 32 == 0");
  if (g.q_codes && (!aligned16(g.q_codes) || !aligned16(g.q_scales))) return fail(FP4_ERR_INVALID_ARG, "Hcodes / Hscales alignment");
  if (!aligned4(g.amax_out)) return fail(FP4_ERR_INVALID_ARG, "amax_out alignment");
  g.mx = fmt == FP4_MXFP4;
  g.act = act;
  g.out_bf16 = out_dtype == FP4_BF16;
  if (g.num_groups == 0) {
    const size_t need = gated_workspace_bytes(g.M, g.F, g.K, g.mx, g.q_codes || g.amax_out);
    if (need && (!g.ws || g.ws_bytes < need || !aligned16(g.ws)))
      return fail(FP4_ERR_INVALID_ARG, "workspace too small or misaligned (see fp4_gemm_gated_workspace_size)");
  }
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (g.amax_out) {
    const cudaError_t e = cudaMemsetAsync(g.amax_out, 0, sizeof(float), st);
    if (e != cudaSuccess) return cuda_fail(e, "zeroing amax_out");
  }
  if (g.q_codes && (g.M % 128 != 0 || (g.F / 16) % 4 != 0)) {  // the scale layout's pads read as 0
    const cudaError_t e = cudaMemsetAsync(g.q_scales, 0, fp4_scales_bytes(g.M, g.F, FP4_NVFP4), st);
    if (e != cudaSuccess) return cuda_fail(e, "zero-filling the scale pads");
  }
  const char* why = nullptr;
  cudaError_t err = cudaSuccess;
  const int rc = launch_gated(g, status, st, &why, &err);
  if (rc == 1) return fail(FP4_ERR_INVALID_ARG, why);
  if (rc == 2) return cuda_fail(err, "gated GEMM launch");
  return FP4_OK;
}

fp4_status fp4_gemm_gated(fp4_fmt fmt, const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* Wg,
                          const uint8_t* sWg, const float* gWg, const uint8_t* Wu, const uint8_t* sWu, const float* gWu,
                          int64_t M, int64_t F, int64_t K, const float* bias_g, const float* bias_u, fp4_act act,
                          void* H, fp4_dtype out_dtype, void* G, void* U, uint8_t* Hcodes, uint8_t* Hscales,
                          const float* gH, float* amax_out, void* workspace, size_t workspace_bytes, unsigned flags,
                          void* stream) {
  if (flags & ~static_cast<unsigned>(FP4_GEMM_WEIGHTS_READY)) return fail(FP4_ERR_INVALID_ARG, "unknown flag");
  GatedProblem g{};
  g.A = A;
  g.sA = sA;
  g.gA = gA;
  g.Wg = Wg;
  g.sWg = sWg;
  g.gWg = gWg;
  g.Wu = Wu;
  g.sWu = sWu;
  g.gWu = gWu;
  g.M = M;
  g.F = F;
  g.K = K;
  g.bias_g = bias_g;
  g.bias_u = bias_u;
  g.H = H;
  g.G = G;
  g.U = U;
  g.q_codes = Hcodes;
  g.q_scales = Hscales;
  g.q_g = gH;
  g.amax_out = amax_out;
  g.ws = workspace;
  g.ws_bytes = workspace_bytes;
  g.weights_ready = (flags & FP4_GEMM_WEIGHTS_READY) ? 1 : 0;
  return gated_common(g, fmt, act, out_dtype, stream);
}

static size_t quant_ws_aligned() { return (kQuantWorkspaceBytes + 255) / 256 * 256; }

size_t fp4_gemm_gated_bf16a_workspace_size(int64_t M, int64_t F, int64_t K) {
  if (M <= 0 || F <= 0 || K <= 0) return 0;
  return quant_ws_aligned() + gated_workspace_bytes(M, F, K, 0, false);
}

fp4_status fp4_gemm_gated_bf16a(const void* X, const uint8_t* Wg, const uint8_t* sWg, const float* gWg,
                                const uint8_t* Wu, const uint8_t* sWu, const float* gWu, int64_t M, int64_t F,
                                int64_t K, const float* bias_g, const float* bias_u, fp4_act act, void* H,
                                fp4_dtype out_dtype, void* G, void* U, uint8_t* Xcodes, uint8_t* Xscales, float* gX,
                                void* workspace, size_t workspace_bytes, unsigned flags, void* stream) {
  if (!X || !Wg || !sWg || !Wu || !sWu || !H || !Xcodes || !Xscales || !gX || !workspace)
    return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (M <= 0 || F <= 0 || K <= 0 || K % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "shape (K % 32 == 0)");
  if (M > kMaxDim || F > kMaxDim || K > kMaxDim) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!dtype_ok(out_dtype)) return fail(FP4_ERR_INVALID_ARG, "out_dtype");
  if (!act_ok(act)) return fail(FP4_ERR_INVALID_ARG, "act");
  if (flags & ~static_cast<unsigned>(FP4_GEMM_WEIGHTS_READY)) return fail(FP4_ERR_INVALID_ARG, "unknown flag");
  if (!G != !U) return fail(FP4_ERR_INVALID_ARG, "G and U: both or neither");
  if (G && (G == U || G == H || U == H)) return fail(FP4_ERR_INVALID_ARG, "H, G and U must be different buffers");
  if (!aligned16(X) || !aligned16(Wg) || !aligned16(sWg) || !aligned16(Wu) || !aligned16(sWu) || !aligned16(H) ||
      !aligned16(G) || !aligned16(U) || !aligned16(Xcodes) || !aligned16(Xscales) || !aligned16(workspace))
    return fail(FP4_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  if (!aligned4(bias_g) || !aligned4(bias_u)) return fail(FP4_ERR_INVALID_ARG, "bias alignment");
  if (!aligned4(gWg) || !aligned4(gWu) || !aligned4(gX)) return fail(FP4_ERR_INVALID_ARG, "global scale alignment");
  if (workspace_bytes < fp4_gemm_gated_bf16a_workspace_size(M, F, K))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small (see fp4_gemm_gated_bf16a_workspace_size)");
  uint8_t* const ws = static_cast<uint8_t*>(workspace) + quant_ws_aligned();
  const size_t ws_bytes = workspace_bytes - quant_ws_aligned();
  if (!gated_decode_eligible(M, F, K)) {
    const fp4_status s = fp4_quantize(X, M, K, FP4_BF16, FP4_NVFP4, 16, Xcodes, Xscales, gX, nullptr, nullptr, nullptr,
                                      workspace, kQuantWorkspaceBytes, stream);
    if (s != FP4_OK) return s;
    return fp4_gemm_gated(FP4_NVFP4, Xcodes, Xscales, gX, Wg, sWg, gWg, Wu, sWu, gWu, M, F, K, bias_g, bias_u, act, H,
                          out_dtype, G, U, nullptr, nullptr, nullptr, nullptr, ws, ws_bytes, flags, stream);
  }
  unsigned* status;
  const fp4_status ds = device_state(&status);
  if (ds != FP4_OK) return ds;
  DecodeProblem q{};
  q.W = Wg;
  q.sW = sWg;
  q.gW = gWg;
  q.X = X;
  q.Xq_out = Xcodes;
  q.Xs_out = Xscales;
  q.gX_out = gX;
  q.M = M;
  q.N = F;
  q.K = K;
  q.D = H;
  q.out_bf16 = out_dtype == FP4_BF16;
  q.ws = ws;
  q.ws_bytes = ws_bytes;
  q.weights_ready = (flags & FP4_GEMM_WEIGHTS_READY) ? 1 : 0;
  q.bias = bias_g;
  q.act = act;
  DecodeExtra x{};
  x.W2 = Wu;
  x.sW2 = sWu;
  x.gW2 = gWu;
  x.bias2 = bias_u;
  x.pre = G;
  x.pre2 = U;
  const char* why = nullptr;
  cudaError_t err = cudaSuccess;
  const int rc = launch_decode_extra(q, x, status, static_cast<cudaStream_t>(stream), &why, &err);
  if (rc == 1) return fail(FP4_ERR_INVALID_ARG, why);
  if (rc == 2) return cuda_fail(err, "gated decode GEMM launch");
  return FP4_OK;
}

fp4_status fp4_gemm_gated_grouped(fp4_fmt fmt, int num_groups, const int32_t* offsets, const uint8_t* A,
                                  const uint8_t* sA, const float* gA, const uint8_t* Wg, const uint8_t* sWg,
                                  const float* gWg, const uint8_t* Wu, const uint8_t* sWu, const float* gWu,
                                  int64_t total_rows, int64_t F, int64_t K, const float* bias_g, const float* bias_u,
                                  fp4_act act, void* H, fp4_dtype out_dtype, void* G, void* U, void* stream) {
  if (num_groups <= 0 || num_groups > kMaxGroups || !offsets) return fail(FP4_ERR_INVALID_ARG, "groups / offsets");
  GatedProblem g{};
  g.A = A;
  g.sA = sA;
  g.gA = gA;
  g.Wg = Wg;
  g.sWg = sWg;
  g.gWg = gWg;
  g.Wu = Wu;
  g.sWu = sWu;
  g.gWu = gWu;
  g.M = total_rows;
  g.F = F;
  g.K = K;
  g.bias_g = bias_g;
  g.bias_u = bias_u;
  g.H = H;
  g.G = G;
  g.U = U;
  g.num_groups = num_groups;
  g.offsets = offsets;
  return gated_common(g, fmt, act, out_dtype, stream);
}

// Checks of a block-scaled copy that a row kernel writes, and its scale pads' zero-fill.
static fp4_status check_codes(fp4_fmt fmt, const uint8_t* codes, const uint8_t* scales, const float* global, int64_t cols,
                              CodesOut* q) {
  *q = CodesOut{0, nullptr, nullptr, nullptr};
  if (!codes) return FP4_OK;
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return fail(FP4_ERR_INVALID_ARG, "fmt");
  if (!scales) return fail(FP4_ERR_INVALID_ARG, "FP4 output needs scales");
  if (fmt == FP4_NVFP4 && !global) return fail(FP4_ERR_INVALID_ARG, "NVFP4 output needs the caller's global scale");
  if (cols % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "FP4 output needs cols % 32 == 0");
  if (!aligned16(codes) || !aligned16(scales)) return fail(FP4_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
  if (!aligned4(global)) return fail(FP4_ERR_INVALID_ARG, "global scale alignment");
  q->fmt = fmt == FP4_MXFP4 ? 2 : 1;
  q->codes = const_cast<uint8_t*>(codes);
  q->scales = const_cast<uint8_t*>(scales);
  q->g = global;
  return FP4_OK;
}

static cudaError_t clear_row_outputs(const CodesOut& q, fp4_fmt fmt, int64_t rows, int64_t cols, float* amax_out,
                                     cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (amax_out) e = cudaMemsetAsync(amax_out, 0, sizeof(float), st);
  if (e == cudaSuccess && q.codes && (rows % 128 != 0 || (cols / (fmt == FP4_MXFP4 ? 32 : 16)) % 4 != 0))
    e = cudaMemsetAsync(q.scales, 0, fp4_scales_bytes(rows, cols, fmt), st);  // the layout's pads read as 0
  return e;
}

size_t fp4_act_backward_workspace_size(int64_t rows, int64_t cols, int gated) {
  if (rows <= 0 || cols <= 0) return 0;
  return act_grad_workspace_bytes(rows, cols, gated != 0);
}

fp4_status fp4_act_backward(const void* dH, const void* G, const void* U, int64_t rows, int64_t cols, fp4_dtype in_dtype,
                            fp4_act act, void* dZ, fp4_dtype out_dtype, float* dbias, fp4_fmt fmt, uint8_t* codes,
                            uint8_t* scales, const float* global, float* amax_out, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!dH || !G) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (!dZ && !codes) return fail(FP4_ERR_INVALID_ARG, "no output: dZ and codes are both NULL");
  if (rows <= 0 || cols <= 0) return fail(FP4_ERR_INVALID_ARG, "rows and cols must be positive");
  if (rows > (1ll << 31) - 256 || cols > (1ll << 30) - 256) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(FP4_ERR_INVALID_ARG, "in_dtype / out_dtype");
  if (!act_ok(act)) return fail(FP4_ERR_INVALID_ARG, "act");
  if (!aligned16(dH) || !aligned16(G) || !aligned16(U) || !aligned16(dZ))
    return fail(FP4_ERR_INVALID_ARG, "dH, G, U and dZ must be 16-byte aligned");
  if (dZ && (dZ == dH || dZ == G || dZ == U)) return fail(FP4_ERR_INVALID_ARG, "dZ must be a buffer of its own");
  if (!aligned4(dbias) || !aligned4(amax_out)) return fail(FP4_ERR_INVALID_ARG, "dbias / amax_out alignment");
  CodesOut q;
  const fp4_status cs = check_codes(fmt, codes, scales, global, cols, &q);
  if (cs != FP4_OK) return cs;
  if (dbias && (!workspace || !aligned16(workspace) || workspace_bytes < act_grad_workspace_bytes(rows, cols, U != nullptr)))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small or misaligned (see fp4_act_backward_workspace_size)");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = clear_row_outputs(q, fmt, rows, U ? 2 * cols : cols, amax_out, st);
  if (e != cudaSuccess) return cuda_fail(e, "clearing outputs");
  ActGradProblem p{};
  p.dh = dH;
  p.g = G;
  p.u = U;
  p.bf16 = in_dtype == FP4_BF16;
  p.rows = rows;
  p.cols = cols;
  p.act = act;
  p.dz = dZ;
  p.dz_bf16 = out_dtype == FP4_BF16;
  p.dbias = dbias;
  p.q = q;
  p.amax_out = amax_out;
  p.ws = static_cast<float*>(workspace);
  e = launch_act_grad(p, status, st);
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "activation backward launch");
}

fp4_status fp4_layernorm(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, const float* weight,
                         const float* bias, float eps, void* y, fp4_dtype out_dtype, float* mean, float* rstd,
                         fp4_fmt fmt, uint8_t* codes, uint8_t* scales, const float* global, float* amax_out,
                         void* stream) {
  if (!x) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (!y && !codes) return fail(FP4_ERR_INVALID_ARG, "no output: y and codes are both NULL");
  if (rows <= 0 || cols <= 0) return fail(FP4_ERR_INVALID_ARG, "rows and cols must be positive");
  if (rows > (1ll << 31) - 256 || cols > (1ll << 30)) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(FP4_ERR_INVALID_ARG, "in_dtype / out_dtype");
  if (!(eps >= 0.0f) || eps > 3.4e38f) return fail(FP4_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (!aligned16(x) || !aligned16(y)) return fail(FP4_ERR_INVALID_ARG, "x and y must be 16-byte aligned");
  if (y == x && in_dtype != out_dtype) return fail(FP4_ERR_INVALID_ARG, "y in x's place needs x's type");
  if (!aligned4(weight) || !aligned4(bias) || !aligned4(mean) || !aligned4(rstd) || !aligned4(amax_out))
    return fail(FP4_ERR_INVALID_ARG, "weight / bias / mean / rstd / amax_out alignment");
  CodesOut q;
  const fp4_status cs = check_codes(fmt, codes, scales, global, cols, &q);
  if (cs != FP4_OK) return cs;
  if (q.codes && (!aligned16(weight) || !aligned16(bias)))
    return fail(FP4_ERR_INVALID_ARG, "FP4 output needs 16-byte aligned weight and bias");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = clear_row_outputs(q, fmt, rows, cols, amax_out, st);
  if (e != cudaSuccess) return cuda_fail(e, "clearing outputs");
  LayerNormProblem p{};
  p.x = x;
  p.bf16 = in_dtype == FP4_BF16;
  p.rows = rows;
  p.cols = cols;
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.y = y;
  p.y_bf16 = out_dtype == FP4_BF16;
  p.mean = mean;
  p.rstd = rstd;
  p.q = q;
  p.amax_out = amax_out;
  e = launch_layernorm(p, status, st);
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "layer norm launch");
}

size_t fp4_layernorm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return layernorm_grad_workspace_bytes(rows, cols);
}

fp4_status fp4_layernorm_backward(const void* dy, const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype,
                                  const float* weight, const float* mean, const float* rstd, const void* dres, void* dx,
                                  fp4_dtype out_dtype, float* dweight, float* dbias, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  if (!dy || !x || !mean || !rstd || !dx) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (rows <= 0 || cols <= 0) return fail(FP4_ERR_INVALID_ARG, "rows and cols must be positive");
  if (rows > (1ll << 31) - 256 || cols > (1ll << 30)) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(FP4_ERR_INVALID_ARG, "in_dtype / out_dtype");
  if (!aligned16(dy) || !aligned16(x) || !aligned16(dres) || !aligned16(dx))
    return fail(FP4_ERR_INVALID_ARG, "dy, x, dres and dx must be 16-byte aligned");
  if (!aligned4(weight) || !aligned4(mean) || !aligned4(rstd) || !aligned4(dweight) || !aligned4(dbias))
    return fail(FP4_ERR_INVALID_ARG, "weight / mean / rstd / dweight / dbias alignment");
  if (dx == x || ((dx == dy || dx == dres) && in_dtype != out_dtype))
    return fail(FP4_ERR_INVALID_ARG, "dx may be dy or dres of the same type, not x");
  if ((dweight || dbias) && (!workspace || !aligned16(workspace) || workspace_bytes < layernorm_grad_workspace_bytes(rows, cols)))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small or misaligned (see fp4_layernorm_backward_workspace_size)");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  LayerNormGradProblem p{};
  p.dy = dy;
  p.x = x;
  p.bf16 = in_dtype == FP4_BF16;
  p.rows = rows;
  p.cols = cols;
  p.weight = weight;
  p.mean = mean;
  p.rstd = rstd;
  p.dres = dres;
  p.dx = dx;
  p.dx_bf16 = out_dtype == FP4_BF16;
  p.dweight = dweight;
  p.dbias = dbias;
  p.ws = static_cast<float*>(workspace);
  const cudaError_t e = launch_layernorm_grad(p, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "layer norm backward launch");
}

// ------------------------------------------------------------------ tokens to experts and back
constexpr int64_t kMaxSlots = 1ll << 30, kMaxMoeCols = 1ll << 24;

static fp4_status check_moe(int64_t tokens, int64_t cols, int topk, fp4_dtype in_dtype, fp4_dtype out_dtype,
                            const int32_t* row_of) {
  if (!row_of) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (tokens <= 0 || cols <= 0 || topk <= 0) return fail(FP4_ERR_INVALID_ARG, "tokens, cols and topk must be positive");
  if (topk > 1024 || tokens > kMaxSlots / topk || cols > kMaxMoeCols)
    return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return fail(FP4_ERR_INVALID_ARG, "in_dtype / out_dtype");
  if (!aligned4(row_of)) return fail(FP4_ERR_INVALID_ARG, "row_of alignment");
  return FP4_OK;
}

size_t fp4_moe_sort_workspace_size(int64_t tokens, int topk, int num_experts) {
  if (tokens <= 0 || topk <= 0 || num_experts <= 0 || topk > 1024 || num_experts > kMaxGroups || tokens > kMaxSlots / topk)
    return 0;
  return moe_sort_workspace_bytes(tokens * topk, num_experts);
}

fp4_status fp4_moe_sort(const void* ids, int id_bytes, int64_t tokens, int topk, int num_experts, int32_t* offsets,
                        int32_t* row_of, int32_t* scale_row_of, void* workspace, size_t workspace_bytes, void* stream) {
  const fp4_status c = check_moe(tokens, 1, topk, FP4_F32, FP4_F32, row_of);
  if (c != FP4_OK) return c;
  if (!ids || !offsets) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (id_bytes != 4 && id_bytes != 8) return fail(FP4_ERR_INVALID_ARG, "id_bytes must be 4 or 8");
  if (num_experts <= 0 || num_experts > kMaxGroups) return fail(FP4_ERR_INVALID_ARG, "num_experts");
  if ((reinterpret_cast<uintptr_t>(ids) & (id_bytes - 1)) || !aligned4(offsets) || !aligned4(scale_row_of))
    return fail(FP4_ERR_INVALID_ARG, "ids / offsets / scale_row_of alignment");
  const size_t need = moe_sort_workspace_bytes(tokens * topk, num_experts);
  if (need && (!workspace || !aligned4(workspace) || workspace_bytes < need))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small or misaligned (see fp4_moe_sort_workspace_size)");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  const cudaError_t e = launch_moe_sort(ids, id_bytes, tokens * topk, num_experts, offsets, row_of, scale_row_of, workspace,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "sort launch");
}

fp4_status fp4_moe_dispatch(const void* x, int64_t tokens, int64_t cols, fp4_dtype in_dtype, int topk,
                            const int32_t* row_of, void* y, fp4_dtype out_dtype, void* stream) {
  const fp4_status c = check_moe(tokens, cols, topk, in_dtype, out_dtype, row_of);
  if (c != FP4_OK) return c;
  if (!x || !y) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(y)) return fail(FP4_ERR_INVALID_ARG, "x and y must be 16-byte aligned");
  if (x == y) return fail(FP4_ERR_INVALID_ARG, "y must not be x");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  DispatchProblem p{};
  p.x = x;
  p.bf16 = in_dtype == FP4_BF16;
  p.tokens = tokens;
  p.cols = cols;
  p.topk = topk;
  p.row_of = row_of;
  p.y = y;
  p.y_bf16 = out_dtype == FP4_BF16;
  const cudaError_t e = launch_moe_dispatch(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "dispatch launch");
}

fp4_status fp4_moe_dispatch_codes(const void* x, int64_t tokens, int64_t cols, fp4_dtype in_dtype, int topk,
                                  const int32_t* row_of, const int32_t* scale_row_of, int num_experts,
                                  const int32_t* offsets, fp4_fmt fmt, uint8_t* codes, uint8_t* scales,
                                  const float* global, void* stream) {
  const fp4_status c = check_moe(tokens, cols, topk, in_dtype, FP4_F32, row_of);
  if (c != FP4_OK) return c;
  if (!x || !codes || !scale_row_of || !offsets) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (num_experts <= 0 || num_experts > kMaxGroups) return fail(FP4_ERR_INVALID_ARG, "num_experts");
  if (!aligned16(x)) return fail(FP4_ERR_INVALID_ARG, "x must be 16-byte aligned");
  if (!aligned4(scale_row_of) || !aligned4(offsets)) return fail(FP4_ERR_INVALID_ARG, "scale_row_of / offsets alignment");
  DispatchCodesProblem p{};
  const fp4_status cs = check_codes(fmt, codes, scales, global, cols, &p.q);
  if (cs != FP4_OK) return cs;
  if (static_cast<const void*>(codes) == x) return fail(FP4_ERR_INVALID_ARG, "codes must not be x");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  p.x = x;
  p.bf16 = in_dtype == FP4_BF16;
  p.tokens = tokens;
  p.cols = cols;
  p.topk = topk;
  p.num_experts = num_experts;
  p.row_of = row_of;
  p.scale_row_of = scale_row_of;
  p.offsets = offsets;
  const cudaError_t e = launch_moe_dispatch_codes(p, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "dispatch launch");
}

static fp4_status i8_rows(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, int topk, const int32_t* row_of,
                          const int32_t* valid, int8_t* codes, float* row_scales, void* stream) {
  if (!x || !codes || !row_scales) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (cols % 16 != 0) return fail(FP4_ERR_INVALID_ARG, "8-bit rows need cols % 16 == 0");
  if (static_cast<const void*>(codes) == x) return fail(FP4_ERR_INVALID_ARG, "codes must not be x");
  if (!aligned16(x) || !aligned16(codes)) return fail(FP4_ERR_INVALID_ARG, "x and codes must be 16-byte aligned");
  if (!aligned4(row_scales) || !aligned4(valid)) return fail(FP4_ERR_INVALID_ARG, "row_scales / rows_valid alignment");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  I8RowsProblem p{};
  p.x = x;
  p.bf16 = in_dtype == FP4_BF16;
  p.rows = rows;
  p.cols = cols;
  p.topk = topk;
  p.row_of = row_of;
  p.valid = valid;
  p.codes = codes;
  p.scales = row_scales;
  const cudaError_t e = launch_quantize_i8(p, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "8-bit quantize launch");
}

fp4_status fp4_moe_dispatch_i8(const void* x, int64_t tokens, int64_t cols, fp4_dtype in_dtype, int topk,
                               const int32_t* row_of, int8_t* codes, float* row_scales, void* stream) {
  const fp4_status c = check_moe(tokens, cols, topk, in_dtype, FP4_F32, row_of);
  if (c != FP4_OK) return c;
  return i8_rows(x, tokens, cols, in_dtype, topk, row_of, nullptr, codes, row_scales, stream);
}

fp4_status fp4_quantize_i8(const void* x, int64_t rows, int64_t cols, fp4_dtype in_dtype, int8_t* codes,
                           float* row_scales, const int32_t* rows_valid, void* stream) {
  if (rows <= 0 || cols <= 0) return fail(FP4_ERR_INVALID_ARG, "rows and cols must be positive");
  if (rows > kMaxDim || cols > kMaxDim) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!dtype_ok(in_dtype)) return fail(FP4_ERR_INVALID_ARG, "in_dtype");
  return i8_rows(x, rows, cols, in_dtype, 1, nullptr, rows_valid, codes, row_scales, stream);
}

fp4_status fp4_moe_combine(const void* y, fp4_dtype in_dtype, const int32_t* row_of, const float* weights, int64_t tokens,
                           int topk, int64_t cols, const void* residual, fp4_dtype residual_dtype, void* out,
                           fp4_dtype out_dtype, void* stream) {
  const fp4_status c = check_moe(tokens, cols, topk, in_dtype, out_dtype, row_of);
  if (c != FP4_OK) return c;
  if (!y || !out) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (residual && !dtype_ok(residual_dtype)) return fail(FP4_ERR_INVALID_ARG, "residual_dtype");
  if (!aligned16(y) || !aligned16(out) || !aligned16(residual))
    return fail(FP4_ERR_INVALID_ARG, "y, residual and out must be 16-byte aligned");
  if (!aligned4(weights)) return fail(FP4_ERR_INVALID_ARG, "weights alignment");
  if (out == y) return fail(FP4_ERR_INVALID_ARG, "out must not be y");
  if (out == residual && out_dtype != residual_dtype)
    return fail(FP4_ERR_INVALID_ARG, "out in the residual's place needs its type");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  CombineProblem p{};
  p.y = y;
  p.bf16 = in_dtype == FP4_BF16;
  p.row_of = row_of;
  p.weights = weights;
  p.tokens = tokens;
  p.cols = cols;
  p.topk = topk;
  p.res = residual;
  p.res_bf16 = residual_dtype == FP4_BF16;
  p.out = out;
  p.out_bf16 = out_dtype == FP4_BF16;
  const cudaError_t e = launch_moe_combine(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "combine launch");
}

fp4_status fp4_moe_combine_backward(const void* dout, const void* y, fp4_dtype in_dtype, const int32_t* row_of,
                                    const float* weights, int64_t tokens, int topk, int64_t cols, void* dy,
                                    fp4_dtype out_dtype, float* dweights, void* stream) {
  const fp4_status c = check_moe(tokens, cols, topk, in_dtype, out_dtype, row_of);
  if (c != FP4_OK) return c;
  if (!dout || (dweights && !y)) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (!dy && !dweights) return fail(FP4_ERR_INVALID_ARG, "no output: dy and dweights are both NULL");
  if (!aligned16(dout) || !aligned16(y) || !aligned16(dy))
    return fail(FP4_ERR_INVALID_ARG, "dout, y and dy must be 16-byte aligned");
  if (!aligned4(weights) || !aligned4(dweights)) return fail(FP4_ERR_INVALID_ARG, "weights / dweights alignment");
  if (dy == dout) return fail(FP4_ERR_INVALID_ARG, "dy must not be dout");
  if (dy && dy == y && in_dtype != out_dtype) return fail(FP4_ERR_INVALID_ARG, "dy in y's place needs y's type");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  CombineGradProblem p{};
  p.dout = dout;
  p.y = y;
  p.bf16 = in_dtype == FP4_BF16;
  p.row_of = row_of;
  p.weights = weights;
  p.tokens = tokens;
  p.cols = cols;
  p.topk = topk;
  p.dy = dy;
  p.dy_bf16 = out_dtype == FP4_BF16;
  p.dweights = dweights;
  const cudaError_t e = launch_moe_combine_grad(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "combine backward launch");
}

// ------------------------------------------------------------------ products in 8-bit integers
constexpr int64_t kMaxI8K = 131056;  // K (-128)^2 < 2^31

static fp4_status gemm_i8_common(const I8Problem& p, fp4_act act, fp4_dtype out_dtype, void* stream) {
  if (!p.A || !p.sA || !p.B || !p.sB || !p.D) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (p.M <= 0 || p.N <= 0 || p.K <= 0) return fail(FP4_ERR_INVALID_ARG, "M, N and K must be positive");
  if (p.K % 16 != 0) return fail(FP4_ERR_INVALID_ARG, "K must be a multiple of 16");
  if (p.M > kMaxDim || p.N > kMaxDim / std::max(1, p.num_groups) || p.K > kMaxI8K)
    return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (!act_ok(act)) return fail(FP4_ERR_INVALID_ARG, "act");
  if (!dtype_ok(out_dtype)) return fail(FP4_ERR_INVALID_ARG, "out_dtype");
  if (!aligned16(p.A) || !aligned16(p.B) || !aligned16(p.D))
    return fail(FP4_ERR_INVALID_ARG, "A, B and D must be 16-byte aligned");
  if (!aligned4(p.sA) || !aligned4(p.sB) || !aligned4(p.bias) || !aligned4(p.offsets))
    return fail(FP4_ERR_INVALID_ARG, "scales / bias / offsets alignment");
  // (the workspace's size goes by the device's SM count)
  const size_t need = i8_workspace_bytes(p.M, p.N, p.K, p.num_groups);
  if (need && (!p.ws || !aligned16(p.ws) || p.ws_bytes < need))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small or misaligned (see fp4_gemm_i8_workspace_size)");
  unsigned* status;
  const fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  const char* why = "";
  cudaError_t e = cudaSuccess;
  const int r = launch_gemm_i8(p, status, static_cast<cudaStream_t>(stream), &why, &e);
  if (r == 1) return fail(FP4_ERR_INVALID_ARG, why);
  return r == 0 ? FP4_OK : cuda_fail(e, "8-bit GEMM launch");
}

size_t fp4_gemm_i8_workspace_size(int64_t M, int64_t N, int64_t K) { return i8_workspace_bytes(M, N, K, 0); }

size_t fp4_gemm_i8_grouped_workspace_size(int num_groups, int64_t total_rows, int64_t N, int64_t K) {
  return num_groups > 0 && num_groups <= kMaxGroups ? i8_workspace_bytes(total_rows, N, K, num_groups) : 0;
}

fp4_status fp4_gemm_i8(const int8_t* A, const float* sA, const int8_t* B, const float* sB, int64_t M, int64_t N, int64_t K,
                       const float* bias, fp4_act act, void* D, fp4_dtype out_dtype, void* workspace,
                       size_t workspace_bytes, unsigned flags, void* stream) {
  if (flags & ~static_cast<unsigned>(FP4_GEMM_WEIGHTS_READY)) return fail(FP4_ERR_INVALID_ARG, "unknown flag");
  I8Problem p{};
  p.A = A;
  p.B = B;
  p.sA = sA;
  p.sB = sB;
  p.M = M;
  p.N = N;
  p.K = K;
  p.bias = bias;
  p.act = act;
  p.D = D;
  p.out_bf16 = out_dtype == FP4_BF16;
  p.ws = workspace;
  p.ws_bytes = workspace_bytes;
  p.weights_ready = (flags & FP4_GEMM_WEIGHTS_READY) != 0;
  return gemm_i8_common(p, act, out_dtype, stream);
}

fp4_status fp4_gemm_i8_grouped(int num_groups, const int32_t* offsets, const int8_t* A, const float* sA, const int8_t* B,
                               const float* sB, int64_t total_rows, int64_t N, int64_t K, const float* bias, fp4_act act,
                               void* D, fp4_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (num_groups <= 0 || num_groups > kMaxGroups || !offsets) return fail(FP4_ERR_INVALID_ARG, "groups / offsets");
  I8Problem p{};
  p.A = A;
  p.B = B;
  p.sA = sA;
  p.sB = sB;
  p.M = total_rows;
  p.N = N;
  p.K = K;
  p.bias = bias;
  p.act = act;
  p.D = D;
  p.out_bf16 = out_dtype == FP4_BF16;
  p.ws = workspace;
  p.ws_bytes = workspace_bytes;
  p.num_groups = num_groups;
  p.offsets = offsets;
  return gemm_i8_common(p, act, out_dtype, stream);
}

size_t fp4_gemm_epilogue_workspace_size(int64_t M, int64_t N, int64_t K, fp4_fmt fmt, int rows_in_place) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  const int mx = fmt == FP4_MXFP4;  // (the plain epilogue's plan can be another one)
  return std::max(gemm_full_workspace_bytes(M, N, K, mx, rows_in_place != 0),
                  gemm_workspace_bytes(M, N, K, mx, rows_in_place != 0));
}

size_t fp4_gemm_bf16a_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0) return 0;
  return gemm_bf16a_workspace_bytes(M, N, K);
}

fp4_status fp4_gemm_bf16a(const void* X, const uint8_t* B, const uint8_t* sB, const float* gB, int64_t M, int64_t N,
                          int64_t K, void* D, fp4_dtype out_dtype, uint8_t* Xcodes, uint8_t* Xscales, float* gX,
                          void* workspace, size_t workspace_bytes, unsigned flags, void* stream) {
  if (!X || !B || !sB || !D || !Xcodes || !Xscales || !gX || !workspace) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (M <= 0 || N <= 0 || K <= 0 || K % 32 != 0) return fail(FP4_ERR_INVALID_ARG, "shape (K % 32 == 0)");
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return fail(FP4_ERR_UNSUPPORTED, "dimension too large");
  if (out_dtype != FP4_F32 && out_dtype != FP4_BF16) return fail(FP4_ERR_INVALID_ARG, "out_dtype");
  if (flags & ~static_cast<unsigned>(FP4_GEMM_WEIGHTS_READY)) return fail(FP4_ERR_INVALID_ARG, "unknown flag");
  if (!aligned16(X) || !aligned16(B) || !aligned16(sB) || !aligned16(D) || !aligned16(Xcodes) || !aligned16(Xscales) ||
      !aligned16(workspace))
    return fail(FP4_ERR_INVALID_ARG, "buffers must be 16-byte aligned");
  if (!aligned4(gB) || !aligned4(gX)) return fail(FP4_ERR_INVALID_ARG, "global scale alignment");
  if (workspace_bytes < gemm_bf16a_workspace_bytes(M, N, K))
    return fail(FP4_ERR_INVALID_ARG, "workspace too small (see fp4_gemm_bf16a_workspace_size)");
  const size_t qws = (kQuantWorkspaceBytes + 255) / 256 * 256;
  if (decode_eligible(M, N, K)) {
    // one launch: every CTA derives the activations' global scale and quantizes its K
    // segment of them itself while its weight stages stream in
    unsigned* status;
    const fp4_status ds = device_state(&status);
    if (ds != FP4_OK) return ds;
    DecodeProblem q{};
    q.W = B;
    q.sW = sB;
    q.gW = gB;
    q.X = X;
    q.Xq_out = Xcodes;
    q.Xs_out = Xscales;
    q.gX_out = gX;
    q.M = M;
    q.N = N;
    q.K = K;
    q.D = D;
    q.out_bf16 = out_dtype == FP4_BF16;
    q.ws = static_cast<uint8_t*>(workspace) + qws;
    q.ws_bytes = workspace_bytes - qws;
    q.weights_ready = (flags & FP4_GEMM_WEIGHTS_READY) ? 1 : 0;
    q.stall_plus1 = g_stall_next_decode;
    g_stall_next_decode = 0;
    const char* why = nullptr;
    cudaError_t err = cudaSuccess;
    const int rc = launch_decode(q, status, static_cast<cudaStream_t>(stream), &why, &err);
    if (rc == 1) return fail(FP4_ERR_INVALID_ARG, why);
    if (rc == 2) return cuda_fail(err, "decode GEMM launch");
    return FP4_OK;
  }
  // larger M: the activations' amax and codes, then the GEMM, chained by programmatic
  // dependent launch (FP4_GEMM_WEIGHTS_READY lets the GEMM stream the weights early)
  const fp4_status s = fp4_quantize(X, M, K, FP4_BF16, FP4_NVFP4, 16, Xcodes, Xscales, gX, nullptr, nullptr, nullptr, workspace,
                   kQuantWorkspaceBytes, stream);
  if (s != FP4_OK) return s;
  return fp4_gemm_ex(FP4_NVFP4, Xcodes, Xscales, gX, B, sB, gB, M, N, K, D, out_dtype,
                     static_cast<uint8_t*>(workspace) + qws, workspace_bytes - qws, flags, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------------
// Allocation-free GEMM.  Some callers cannot allocate device memory: a host (plugin
// runtime, embedded engine) that owns every device byte and hands this library no
// allocator.  They still need the split-K scratch that decode-sized GEMMs use, so this
// variant takes it from a fixed array compiled into the library instead of from the
// caller.
namespace fp4 {
constexpr size_t kNoAllocScratchBytes = size_t(4) << 20;  // 4 MiB on every device that loads the library
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

// Device address of the array on the current device.  The array's host-side name is
// only a stand-in; the device address comes from cudaGetSymbolAddress, done once per
// device with that device current (the first call on a device does it, so make that
// first call before any stream capture).
static fp4_status noalloc_scratch(void** out) {
  static void* addr[kMaxDevices] = {nullptr};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(FP4_ERR_UNSUPPORTED, "device index out of range");
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress(no-alloc scratch)");
    addr[dev] = p;
  }
  *out = addr[dev];
  return FP4_OK;
}
}  // namespace fp4

extern "C" {

fp4_status fp4_gemm_noalloc(fp4_fmt fmt, const uint8_t* A, const uint8_t* sA, const float* gA, const uint8_t* B,
                            const uint8_t* sB, const float* gB, int64_t M, int64_t N, int64_t K, void* D,
                            fp4_dtype out_dtype, void* stream) {
  if (fmt != FP4_NVFP4 && fmt != FP4_MXFP4) return fail(FP4_ERR_INVALID_ARG, "fmt");
  const size_t need = (M > 0 && N > 0 && K > 0) ? gemm_workspace_bytes(M, N, K, fmt == FP4_MXFP4) : 0;
  if (need > kNoAllocScratchBytes) {
    snprintf(g_err, sizeof(g_err),
             "fp4_gemm_noalloc: this shape needs %zu bytes of scratch but the built-in array holds %zu "
             "(4 MiB); use fp4_gemm with a caller workspace",
             need, kNoAllocScratchBytes);
    return FP4_ERR_INVALID_ARG;
  }
  void* ws = nullptr;
  if (need) {
    fp4_status s = noalloc_scratch(&ws);
    if (s != FP4_OK) return s;
    // every call shares the array: clear the part this call accumulates into
    cudaError_t e = cudaMemsetAsync(ws, 0, need, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "clearing the no-alloc scratch");
  }
  return fp4_gemm(fmt, A, sA, gA, B, sB, gB, M, N, K, D, out_dtype, ws, need, stream);
}

fp4_status fp4_gemm_grouped(fp4_fmt fmt, int num_groups, const int32_t* offsets, const uint8_t* A,
                            const uint8_t* sA, const float* gA, const uint8_t* B, const uint8_t* sB,
                            const float* gB, int64_t total_rows, int64_t N, int64_t K, void* D,
                            fp4_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (num_groups <= 0 || num_groups > kMaxGroups || !offsets) return fail(FP4_ERR_INVALID_ARG, "groups / offsets");
  if (N % 128 != 0) return fail(FP4_ERR_INVALID_ARG, "grouped GEMM needs N % 128 == 0");
  if (total_rows <= 0) return fail(FP4_ERR_INVALID_ARG, "total_rows must be positive");
  GemmProblem g{};
  g.mx = fmt == FP4_MXFP4;
  g.A = A;
  g.sA = sA;
  g.gA = gA;
  g.B = B;
  g.sB = sB;
  g.gB = gB;
  g.M = total_rows;
  g.N = N;
  g.K = K;
  g.D = D;
  g.out_bf16 = out_dtype == FP4_BF16;
  g.ws = workspace;
  g.ws_bytes = workspace_bytes;
  g.num_groups = num_groups;
  g.offsets = offsets;
  return gemm_common(g, fmt, out_dtype, stream);
}

fp4_status fp4_get_status(void* stream) {
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  unsigned v = 0;
  e = cudaMemcpyFromSymbol(&v, g_status_word, sizeof(v));
  if (e != cudaSuccess) return cuda_fail(e, "status read");
  const unsigned zero = 0;
  e = cudaMemcpyToSymbol(g_status_word, &zero, sizeof(zero));
  if (e != cudaSuccess) return cuda_fail(e, "status clear");
  if (v & kStatusTimeout) return fail(FP4_ERR_TIMEOUT, "a device-side wait timed out");
  if (v & kStatusNonFinite) return fail(FP4_ERR_NONFINITE, "non-finite input element");
  return FP4_OK;
}

fp4_status fp4_mma_peak(int iters, int grid, unsigned long long* cycles, void* stream) {
  if (!cycles || iters <= 0 || iters > (1 << 24) || grid <= 0 || grid > 4 * num_sms())
    return fail(FP4_ERR_INVALID_ARG, "iters in 1..2^24, grid in 1..4 x SMs, cycles non-null");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  const cudaError_t e = launch_mma_peak(iters, grid, cycles, status, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "MMA peak launch");
}

fp4_status fp4_debug_stall_next_decode(int cta) {
  if (cta < 0) return fail(FP4_ERR_INVALID_ARG, "cta must be >= 0");
  g_stall_next_decode = cta + 1;
  return FP4_OK;
}

fp4_status fp4_debug_encode(const float* in, int64_t n, int which, uint8_t* out, void* stream) {
  if (!in || !out) return fail(FP4_ERR_INVALID_ARG, "null pointer");
  if (n <= 0 || which < 0 || which > 4) return fail(FP4_ERR_INVALID_ARG, "n / which");
  unsigned* status;
  fp4_status s = device_state(&status);
  if (s != FP4_OK) return s;
  cudaError_t e = launch_debug_encode(in, n, which, out, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FP4_OK : cuda_fail(e, "debug encode launch");
}

}  // extern "C"
