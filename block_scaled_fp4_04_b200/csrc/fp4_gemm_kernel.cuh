// fp4_gemm_kernel.cuh -- the block-scaled GEMM kernel and its launch, shared by the plain,
// the extended-epilogue and the gated translation units (fp4_gemm.cu describes its structure).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "fp4_act.cuh"
#include "fp4_codes.cuh"
#include "fp4_internal.h"
#include "fp4_ptx.cuh"

namespace fp4 {

enum { kModeTile = 0, kModeStreamK = 1, kModeGrouped = 2 };

struct GemmArgs {
  const uint8_t* sfa;
  const uint8_t* sfb;
  int64_t sfa_rb_bytes;     // bytes per 128-row block of A's scales
  int64_t sfb_rb_bytes;
  int64_t sfb_group_bytes;  // grouped: bytes of one expert's B scales
  int sf_atoms_k;           // scale atoms along K per row-block
  int sfb_rbs;              // row-blocks of B (per expert)
  const float* ga;
  const float* gb;
  int Mk, Nk, K, num_kb;    // kernel orientation
  void* out;
  int64_t ldo;
  int out_bf16, transposed, vec_store;
  int indep;  // 1: kernel A, 2: kernel B may be read before the preceding kernel finishes
  float* ws;        // stream-K: FP32 partial sums [Mk, Nk], zero between calls
  int* tile_cnt;    // stream-K: K steps summed so far per tile, zero between calls
  int mode;
  int tiles_m, tiles_n, group_m;
  int64_t total_units;
  int num_groups;
  const int32_t* offsets;
  int b_rows_per_group;
  unsigned* status;
  // epilogue after the scale ("Rubin FP4 GEMM overview" 3.2 / 4.2): + bias[n], activation,
  // and optionally an NVFP4 copy of the result (16-blocks along n, caller's global scale)
  const float* bias;   // [N] (output columns), or null
  int act;             // 0: none, 1: ReLU
  uint8_t* q_codes;    // [M, N/2] NVFP4 codes of the result, or null
  uint8_t* q_scales;   // swizzled scale atoms of the [M, N/16] block scales
  const float* q_g;    // global scale of the NVFP4 result (device)
  int64_t q_atoms;     // scale atoms per 128-row block of the result: ceil(N/16, 4) / 4
  unsigned* amax_out;  // max |result| as float bits (zeroed before the launch), or null
  uint32_t f8_fmt;     // kind::mxf8f6f4: A's format | B's format << 3 (E4M3 0, E2M1 5)
  // kEpiFull, kEpiGated
  const void* res;       // [M, N] added after the activation, or null
  int res_bf16;
  int bias_any;          // a bias is given
  int ws_ld;             // floats per row of partial sums, a multiple of 4
  int sectors;           // rows of the output, its copies and the residual start at 32-byte sectors
  void* pre;             // kEpiFull: the pre-activation; kEpiGated: G; [M, N] in the output type, or null
  void* pre2;            // kEpiGated: U
  const uint8_t* sfb2;   // kEpiGated: the up operand's scales, global scale, bias
  const float* gb2;
  const float* bias2;
  int64_t bias_group;    // grouped: floats between two experts' biases
};

struct Work {
  int a_row, b_row;    // TMA row coordinates of the A and B boxes
  int out_row0;        // first output row (kernel orientation)
  int rows_valid;      // rows of the tile that exist
  int n0;              // first column (kernel orientation)
  int sfa_rb;          // A scale row-block
  int64_t sfb_off;     // byte offset of B's first scale row-block
  int group;
  int kb0, kb1;
  int tile;
};

// TN: output columns per tile (BN, or half of it where a tile holds gate and up columns).
template <int BN, int TN = BN>
struct Sched {
  const GemmArgs& p;
  const int* s_mt;   // grouped: 128-row block prefix per group (= A scale row-blocks)
  const int* s_off;  // grouped: row offsets
  const int* s_pt;   // grouped CTA pairs: 256-row tile prefix per group
  int64_t u, u_end;  // stream-K: current / end unit; tile modes: current unit
  int64_t total;

  int vgrid;         // pipelines in the grid; this one is number vb
  int mtile;         // output rows per M tile: 128, or 256 for a CTA pair
  int sub_row;       // CTA pair: this CTA's first row (and first B row) within the tile
  // vb / vg: this pipeline's index among all pipelines of the grid, and their count
  __device__ Sched(const GemmArgs& args, const int* mt, const int* off, int vb, int vg, int mtile_ = 128,
                   int sub_row_ = 0, const int* pt = nullptr)
      : p(args), s_mt(mt), s_off(off), s_pt(pt), vgrid(vg), mtile(mtile_), sub_row(sub_row_) {
    if (p.mode == kModeStreamK) {
      const int64_t T = p.total_units;
      u = T * vb / vg;
      u_end = T * (vb + 1) / vg;
      total = T;
    } else if (p.mode == kModeGrouped) {
      total = static_cast<int64_t>(tiles_prefix()[p.num_groups]) * p.tiles_n;
      u = vb;
    } else {
      total = p.total_units;
      u = vb;
    }
  }

  __device__ bool next(Work& w) {
    if (p.mode == kModeStreamK) {
      if (u >= u_end) return false;
      const int tile = static_cast<int>(u / p.num_kb);
      const int kb0 = static_cast<int>(u % p.num_kb);
      const int64_t kb1_ = static_cast<int64_t>(kb0) + (u_end - u);
      const int kb1 = static_cast<int>(kb1_ < p.num_kb ? kb1_ : p.num_kb);
      u += kb1 - kb0;
      const int mt = tile / p.tiles_n, nt = tile % p.tiles_n;
      plain(w, mt, nt);
      w.kb0 = kb0;
      w.kb1 = kb1;
      w.tile = tile;
      return true;
    }
    if (u >= total) return false;
    const int64_t cur = u;
    u += vgrid;
    if (p.mode == kModeGrouped) {
      const int E = p.num_groups;
      const int* tp = tiles_prefix();
      int lo = 0, hi = E - 1;  // last group e with tp[e] * tiles_n <= cur
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<int64_t>(tp[mid]) * p.tiles_n <= cur) lo = mid;
        else hi = mid - 1;
      }
      const int e = lo;
      const int mte = tp[e + 1] - tp[e];
      const int64_t local = cur - static_cast<int64_t>(tp[e]) * p.tiles_n;
      const int nt = static_cast<int>(local / mte), mt = static_cast<int>(local % mte);
      // a pair's second CTA may get rows of the next group (or none): they are loaded
      // and multiplied but never stored
      w.a_row = s_off[e] + mt * mtile + sub_row;
      w.out_row0 = w.a_row;
      w.rows_valid = max(0, min(128, s_off[e + 1] - w.a_row));
      w.n0 = nt * TN;
      w.b_row = e * p.b_rows_per_group + w.n0 + (TN == BN ? sub_row : 0);
      w.sfa_rb = s_mt[e] + mt * (mtile / 128) + sub_row / 128;
      w.sfb_off = e * p.sfb_group_bytes + static_cast<int64_t>(w.n0 / 128) * p.sfb_rb_bytes;
      w.group = e;
      w.kb0 = 0;
      w.kb1 = p.num_kb;
      w.tile = static_cast<int>(cur);
      return true;
    }
    // tile mode: rasterize in groups of group_m m-tiles so concurrently running CTAs
    // share A and B tiles in L2
    const int per_group = p.group_m * p.tiles_n;
    const int gi = static_cast<int>(cur / per_group);
    const int first_m = gi * p.group_m;
    const int gsize = min(p.tiles_m - first_m, p.group_m);
    const int r = static_cast<int>(cur % per_group);
    plain(w, first_m + r % gsize, r / gsize);
    w.kb0 = 0;
    w.kb1 = p.num_kb;
    w.tile = static_cast<int>(cur);
    return true;
  }

  // grouped: M-tile prefix per group in this schedule's tile height
  __device__ const int* tiles_prefix() const { return mtile == 256 ? s_pt : s_mt; }

  __device__ void plain(Work& w, int mt, int nt) {
    w.a_row = mt * mtile + sub_row;
    w.out_row0 = w.a_row;
    w.rows_valid = max(0, min(128, p.Mk - w.a_row));
    w.n0 = nt * TN;
    // a pair's CTAs each load half of the tile's B rows (gated: the gate's, the up's)
    w.b_row = w.n0 + (TN == BN ? sub_row : 0);
    w.sfa_rb = w.a_row / 128;
    w.sfb_off = static_cast<int64_t>(w.n0 / 128) * p.sfb_rb_bytes;
    w.group = 0;
  }
};

// Small-N tiles (decode) run two independent pipelines per CTA ("sub-CTAs" of 192
// threads, each with its own producer, MMA issuer, epilogue warps, shared-memory ring
// and TMEM columns).  One thread issues all tcgen05 operations of a pipeline, and at
// N = 16..64 the issue latency of that thread -- not the tensor pipe -- bounds how fast
// weight stages are consumed, so two issuers per SM double the rate.  (Two CTAs per SM
// would do the same, but a kernel that allocates TMEM is scheduled one CTA per SM.)
#ifndef FP4_SMALL_N_PIPES
#define FP4_SMALL_N_PIPES 2
#endif
template <int BN>
constexpr int pipes_per_cta() { return BN <= 32 ? FP4_SMALL_N_PIPES : BN <= 64 ? 2 : 1; }

// F8: the kind::mxf8f6f4 MMA (E2M1 or E4M3 operands, one byte per element in shared
// memory, an E8M0 scale per 32): a stage holds 128 K elements, one scale atom per row-block.
template <int BN, bool MX, int ACC, bool PAIR = false, bool F8 = false, int EPI = kEpiPlain>
struct Cfg {
  static constexpr bool kGated = EPI == kEpiGated || EPI == kEpiGatedWhole;
  static_assert(!kGated || BN == 256, "gated tiles: 128 gate and 128 up columns");
  static_assert(EPI == kEpiPlain || !F8, "mixed-format products have the plain epilogue");
  static_assert(!F8 || MX, "mixed-format MMAs: E8M0 scales");
  static_assert(!PAIR || (BN == 256 && ACC == 1), "CTA pairs run 256 x 256 tiles");
  static constexpr int kP = pipes_per_cta<BN>();
  // Single-pipeline kernels (128/256-wide tiles) add copier warps that move each stage's
  // scale factors into TMEM, so that these copies are not serialised behind the MMA
  // thread's own MMAs: one for A's atoms and one per 128-row block of B's.
  static constexpr bool kSepCp = kP == 1;
  static constexpr int kCopiers = kSepCp ? 1 + (BN >= 128 ? BN / 128 : 1) : 0;
  // One-pipeline kernels run two epilogue warps per TMEM lane quarter, one per column
  // half: twice the TMEM read and store rate, and half a row of packed BF16 per thread
  // is few enough registers to hold the tile while TMEM is already handed back.
  // The long epilogues have too much arithmetic for that: four warps per quarter, which take 32
  // sums at a time and hold the last 32 (half of the tile) while TMEM is handed back.  Measured
  // on tiles of one K step (8192 x 8192 outputs, BF16) with bias, GELU, residual and pre-activation:
  // 276 us with eight warps that held all their 128 sums at 128 registers, 159 us so.  SILU alone
  // gains nothing by it (88 / 98 us): the switch over the activation takes what the warps give.
  static constexpr bool kLong = kSepCp && EPI != kEpiPlain;
  static constexpr int kEpiWarps = kLong ? 16 : kSepCp ? 8 : 4;
  static constexpr int kEpiCols = BN * 4 / kEpiWarps;  // accumulator columns per epilogue thread
  static constexpr int kTileCols = kGated ? BN / 2 : BN;  // output columns of a tile
  static constexpr int kThreads = kSepCp ? 64 + 32 * kEpiWarps + 32 * kCopiers : 192 * kP;
  static constexpr int kAtomsKT = F8 ? 1 : MX ? 2 : 4;  // scale atoms per stage (256 K; 128 K for F8)
  static constexpr int kNRB = BN >= 128 ? BN / 128 : 1;  // B scale row-blocks per tile
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = (PAIR ? BN / 2 : BN) * 128;  // a pair's CTA holds half of B's rows
  static constexpr int kSFABytes = kAtomsKT * 512;
  static constexpr int kSFBBytes = kNRB * kAtomsKT * 512;
  // rounded up to 1024 bytes (the 128-byte swizzle's alignment): only the mixed-format
  // stages (one scale atom per row-block) need the padding
  static constexpr int kStageBytes = (kABytes + kBBytes + kSFABytes + kSFBBytes + 1023) / 1024 * 1024;
  // grouped schedules use 128-wide tiles only, so multi-pipeline kernels skip the group tables
  static constexpr int kGroupBytes = kP == 1 ? (PAIR ? 3 : 2) * (kMaxGroups + 1) * 4 : 0;
  // long epilogues: two tiles' biases (gated: gate's and up's)
  static constexpr int kBiasOff = (1024 /*barriers, flags*/ + kGroupBytes + 15) / 16 * 16;
  static constexpr int kMiscBytes = kLong ? kBiasOff + 2 * BN * 4 : 1024 + kGroupBytes;
  // the opt-in limit per block, less the alignment slack and the static shared memory
  static constexpr int kSmemLimit = 227 * 1024 - 1024 - 256;
  static constexpr int kStagesFit = (kSmemLimit / kP - kMiscBytes) / kStageBytes;
  static constexpr int kStages = kStagesFit > 12 ? 12 : kStagesFit;
  // one pipeline's share; the next pipeline's stages start 1024-byte aligned
  static constexpr int kSubBytes = (kStages * kStageBytes + kMiscBytes + 1023) / 1024 * 1024;
  static constexpr int kSmemBytes = kP == 1 ? kStages * kStageBytes + kMiscBytes + 1024 : kP * kSubBytes + 1024;
  static_assert(kSmemBytes + 256 <= 227 * 1024, "shared memory opt-in limit");
  static constexpr int kSFACols = kAtomsKT * 4;
  static constexpr int kSFBCols = kNRB * kAtomsKT * 4;
  static constexpr int kSFSlot = kSFACols + kSFBCols;
  // TMEM slots for the stages' scale factors: with a separate copier, as many as fit
  // (up to 4, and fewer than the ring's stages) so that it can run ahead of the MMAs
  static constexpr int kSlotsFit = (512 - ACC * BN) / kSFSlot;
  static constexpr int kSFSlots = !kSepCp ? 2 : (kSlotsFit < 4 ? kSlotsFit : 4) < kStages ? (kSlotsFit < 4 ? kSlotsFit : 4)
                                                                                           : kStages - 1;
  static constexpr int kColsUsed = ACC * BN + kSFSlots * kSFSlot;
  static constexpr int kTmemCols = kColsUsed <= 32 ? 32 : kColsUsed <= 64 ? 64 : kColsUsed <= 128 ? 128
                                   : kColsUsed <= 256 ? 256 : 512;  // per pipeline
  // one allocation for all pipelines: a power of two of at least 32 columns
  static constexpr int kTmemAlloc = kP * kTmemCols <= 32 ? 32 : kP * kTmemCols <= 64 ? 64
                                    : kP * kTmemCols <= 128 ? 128 : kP * kTmemCols <= 256 ? 256 : 512;
  static_assert(kP * kTmemCols <= 512, "TMEM budget");
  static_assert(kSFSlots >= 2 && kSFSlots < kStages, "scale-factor slots");
  static_assert(kStageBytes % 1024 == 0 && kSubBytes % 1024 == 0, "128-byte swizzled stages need 1024-byte alignment");
  static_assert(kStages >= 2, "shared memory budget");
  static_assert(BN % 16 == 0 && BN >= 16 && BN <= 256, "MMA N");
};

__device__ __forceinline__ void latch_timeout(volatile int* abort, unsigned* status) {
  *abort = 1;
  atomicOr(status, kStatusTimeout);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void red_add_v4(float* addr, float a, float b, float c, float d) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(addr), "f"(a), "f"(b), "f"(c),
               "f"(d)
               : "memory");
}

// Waits until the grids this one depends on (programmatic dependent launch) have
// finished and their writes are visible; a no-op when launched without the attribute.
__device__ __forceinline__ void wait_prior_grids() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the kernel launched after this one on the stream start its prologue now (it still
// waits for this grid's completion before it reads what this grid writes).  Called by warps
// that have waited for the grids before this one: the next kernel may read weights without a
// wait of its own, if they were written before this kernel, so what is older must be finished.
__device__ __forceinline__ void allow_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void store_out(const GemmArgs& p, int64_t off, float v) {
  if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[off] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(p.out)[off] = v;
}

// Stores 16 consecutive kernel columns [col, col+16) of one kernel row.  With swapped
// operands (transposed) kernel row = output column and kernel column = output row.
__device__ __forceinline__ void store_row16(const GemmArgs& p, int row, int col, const float (&v)[16]) {
  if (p.transposed) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (col + j < p.Nk) store_out(p, static_cast<int64_t>(col + j) * p.ldo + row, v[j]);
    return;
  }
  const int64_t base = static_cast<int64_t>(row) * p.ldo + col;
  if (p.vec_store && col + 16 <= p.Nk) {
    if (p.out_bf16) {
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + base);
      dst[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                          pack_bf16x2(v[6], v[7]));
      dst[1] = make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]),
                          pack_bf16x2(v[14], v[15]));
    } else {
      float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + base);
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (col + j < p.Nk) store_out(p, base + j, v[j]);
}

// Bias and activation of 16 consecutive kernel columns [col, col+16) of kernel row `row`
// (values already multiplied by gA * gB).  With swapped operands the kernel row is the
// output column, which indexes the bias.
__device__ __forceinline__ void epi_bias_act(const GemmArgs& p, int row, int col, float (&v)[16]) {
  if (p.bias) {
    if (p.transposed) {
      const float b = p.bias[row];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __fadd_rn(v[j], b);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (col + j < p.Nk) v[j] = __fadd_rn(v[j], __ldg(p.bias + col + j));
    }
  }
  if (p.act == kActRelu) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = relu_f(v[j]);
  }
}

// NVFP4 copy of 16 output columns [col, col+16) of output row `row` (one block; the
// caller guarantees N % 32 == 0 and a row-major kernel orientation): block scale and
// codes exactly as the quantize kernels compute them, with the caller's global scale.
__device__ __forceinline__ void epi_quantize16(const GemmArgs& p, int row, int col, const float (&v)[16]) {
  const float g = *p.q_g;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  if (m >= 0x7F800000u) atomicOr(p.status, kStatusNonFinite);
  uint32_t sb;
  const float mul = nvfp4_block_scale(__uint_as_float(m), g, sb);
  float a[8], b[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = v[j] == 0.0f ? v[j] : __fmul_rn(v[j], mul);  // a zero stays zero if 1/denom overflowed
    b[j] = v[8 + j] == 0.0f ? v[8 + j] : __fmul_rn(v[8 + j], mul);
  }
  *reinterpret_cast<uint2*>(p.q_codes + static_cast<int64_t>(row) * (p.Nk / 2) + col / 2) =
      make_uint2(pack8<kE2M1Hardware>(a), pack8<kE2M1Hardware>(b));
  const int c = col / 16;
  p.q_scales[((row / 128) * p.q_atoms + c / 4) * 512 + (row % 32) * 16 + ((row % 128) / 32) * 4 + c % 4] =
      static_cast<uint8_t>(sb);
}

// Finishes 16 consecutive kernel columns of one kernel row: bias, activation, the
// BF16 / FP32 store and the NVFP4 copy.
__device__ __forceinline__ void epi_row16(const GemmArgs& p, int row, int col, float (&v)[16], uint32_t& tmax) {
  epi_bias_act(p, row, col, v);
  if (p.out) store_row16(p, row, col, v);
  if (p.q_codes && col < p.Nk) epi_quantize16(p, row, col, v);
  if (p.amax_out) {  // the result's amax, for the global scale of its next quantization
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (p.transposed || col + j < p.Nk) tmax = max(tmax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  }
}

// Reads 16 summed partials of one row (columns [col, col + 16)) of rows padded to whole float4s,
// and clears them.
__device__ __forceinline__ void take_raw16(float* row, int col, int n, uint32_t* v) {
#pragma unroll
  for (int j = 0; j < 16; j += 4) {
    float4* at = reinterpret_cast<float4*>(row + col + j);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col + j < n) {
      t = __ldcg(at);
      __stcg(at, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    v[j] = __float_as_uint(t.x);
    v[j + 1] = __float_as_uint(t.y);
    v[j + 2] = __float_as_uint(t.z);
    v[j + 3] = __float_as_uint(t.w);
  }
}

// Reads 16 summed partials of one row (columns [col, col + 16) of n), clears them, scales.
__device__ __forceinline__ void take_sums16(float* row, int col, int n, float scale, float (&v)[16]) {
  if ((n & 3) == 0 && col + 16 <= n) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      float4* at = reinterpret_cast<float4*>(row + col + j);
      const float4 t = __ldcg(at);
      __stcg(at, make_float4(0.f, 0.f, 0.f, 0.f));
      v[j] = t.x * scale;
      v[j + 1] = t.y * scale;
      v[j + 2] = t.z * scale;
      v[j + 3] = t.w * scale;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      v[j] = 0.0f;
      if (col + j < n) {
        v[j] = __ldcg(row + col + j) * scale;
        __stcg(row + col + j, 0.0f);
      }
    }
  }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// One 32-byte sector, 32-byte aligned.
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void ld_sector(const void* p, uint32_t* w) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}

// Where a warp of the long epilogues is: 32 rows from row0 (the first `rows` of them exist), this
// lane's row being row0 + lane, and `cols` (at most 16) columns from col.
struct EpiSpot {
  int row0, rows, lane;
  int col, cols;
  bool direct;   // whole sectors: each lane reads and writes its own row
  __device__ __forceinline__ bool row_ok() const { return lane < rows; }
};

// Transposes 8 x 8 words over groups of 8 lanes (its own inverse): word k of lane i becomes
// word i of lane k.
__device__ __forceinline__ void transpose8(uint32_t (&w)[8], int lane) {
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if ((k & d) == 0) {
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? w[k] : w[k | d], d);
        if (up) w[k] = got;
        else w[k | d] = got;
      }
  }
}

// Eight words of every lane's row, from element column `col` on (16 BF16 or 8 FP32 elements, of
// which `cols` exist), to or from the matrix.  Where all exist and rows start at 32-byte sectors
// (s.direct; known at compile time in the WHOLE kernels) each lane reads and writes whole sectors
// of its own row: 16-byte pieces, half a sector each, slowed the whole kernel down (8192 x 4096 x
// 4096 gated with G and U: 216 us against 189).  Else the words are transposed over 8 lanes, which
// then hold a run of one row each time, so that neighbouring lanes touch neighbouring words (8192 x
// 4097 x 4096 gated: 199 us, 441 with every lane's elements stored one by one).
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void put_words(const GemmArgs& p, const EpiSpot& s, void* out, int col, int cols, uint32_t (&w)[8]) {
  if (WHOLE || s.direct) {
    if (s.row_ok()) {
      const int64_t at = static_cast<int64_t>(s.row0 + s.lane) * p.ldo + col;
      st_sector(static_cast<uint8_t*>(out) + at * (BF16 ? 2 : 4), w);
    }
    return;
  }
  if constexpr (WHOLE) return;
  uint32_t x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = w[j];
  transpose8(x, s.lane);
  const int i = s.lane & 7, r0 = s.lane & ~7;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (r0 + j >= s.rows) continue;
    const int64_t at = static_cast<int64_t>(s.row0 + r0 + j) * p.ldo + col + (BF16 ? 2 * i : i);
    if constexpr (BF16) {
      uint16_t* dst = static_cast<uint16_t*>(out) + at;
      if (2 * i + 1 < cols && (at & 1) == 0) {
        *reinterpret_cast<uint32_t*>(dst) = x[j];
      } else {
        if (2 * i < cols) dst[0] = static_cast<uint16_t>(x[j]);
        if (2 * i + 1 < cols) dst[1] = static_cast<uint16_t>(x[j] >> 16);
      }
    } else {
      if (i < cols) static_cast<uint32_t*>(out)[at] = x[j];
    }
  }
}

template <bool BF16, bool WHOLE>
__device__ __forceinline__ void get_words(const GemmArgs& p, const EpiSpot& s, const void* in, int col, int cols, uint32_t (&w)[8]) {
  if (WHOLE || s.direct) {
    const int64_t at = static_cast<int64_t>(s.row0 + s.lane) * p.ldo + col;
    if (s.row_ok()) ld_sector(static_cast<const uint8_t*>(in) + at * (BF16 ? 2 : 4), w);
    return;
  }
  if constexpr (WHOLE) return;
  const int i = s.lane & 7, r0 = s.lane & ~7;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] = 0;
    if (r0 + j >= s.rows) continue;
    const int64_t at = static_cast<int64_t>(s.row0 + r0 + j) * p.ldo + col + (BF16 ? 2 * i : i);
    if constexpr (BF16) {
      const uint16_t* src = static_cast<const uint16_t*>(in) + at;
      if (2 * i + 1 < cols && (at & 1) == 0) {
        w[j] = *reinterpret_cast<const uint32_t*>(src);
      } else {
        if (2 * i < cols) w[j] = src[0];
        if (2 * i + 1 < cols) w[j] |= static_cast<uint32_t>(src[1]) << 16;
      }
    } else {
      if (i < cols) w[j] = static_cast<const uint32_t*>(in)[at];
    }
  }
  transpose8(w, s.lane);
}

// Stores 16 values of a row.
template <bool WHOLE>
__device__ __forceinline__ void put16(const GemmArgs& p, const EpiSpot& s, void* out, const float2 (&v)[8]) {
  uint32_t w[8];
  if (p.out_bf16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(v[j].x, v[j].y);
    put_words<true, WHOLE>(p, s, out, s.col, s.cols, w);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[2 * j] = __float_as_uint(v[4 * h + j].x);
        w[2 * j + 1] = __float_as_uint(v[4 * h + j].y);
      }
      put_words<false, WHOLE>(p, s, out, s.col + 8 * h, s.cols - 8 * h, w);
    }
  }
}

// 16 sums of a product, scaled, plus the bias (in shared memory, or null).
__device__ __forceinline__ void linear16(const uint32_t* sums, float scale, const float* bias, float2 (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = __fmul2_rn(make_float2(__uint_as_float(sums[2 * j]), __uint_as_float(sums[2 * j + 1])), pair(scale));
  if (bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 x = reinterpret_cast<const float4*>(bias)[j];
      v[2 * j] = __fadd2_rn(v[2 * j], make_float2(x.x, x.y));
      v[2 * j + 1] = __fadd2_rn(v[2 * j + 1], make_float2(x.z, x.w));
    }
  }
}

// The long epilogues: 16 consecutive columns of a warp's 32 rows, one row per lane, whose sums
// are in registers (gated: 16 gate sums, then 16 up sums).  Only the activation itself is in a
// switch: a copy of the whole per activation took minutes to compile and spilled.  All lanes take
// part.
template <bool GATED, bool WHOLE>
__device__ __forceinline__ void epi_rows(const GemmArgs& p, const EpiSpot& s, const float* bias, const float* bias2,
                                         float scale, float scale2, const uint32_t* sums, uint32_t& tmax) {
  uint32_t res[8], res2[8];
  if (!GATED && p.res) {
    if (p.res_bf16) {
      get_words<true, WHOLE>(p, s, p.res, s.col, s.cols, res);
    } else {
      get_words<false, WHOLE>(p, s, p.res, s.col, s.cols, res);
      get_words<false, WHOLE>(p, s, p.res, s.col + 8, s.cols - 8, res2);
    }
  }
  float2 v[8];
  linear16(sums, scale, bias, v);
  if (p.pre) put16<WHOLE>(p, s, p.pre, v);
  with_act(p.act, [&](auto tag) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = act_value2<decltype(tag)::value>(v[j]);
  });
  if constexpr (GATED) {
    float2 u[8];
    linear16(sums + 16, scale2, bias2, u);
    if (p.pre2) put16<WHOLE>(p, s, p.pre2, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul2_rn(v[j], u[j]);
  } else if (p.res) {
    if (p.res_bf16) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = __fadd2_rn(v[j], make_float2(__uint_as_float(res[j] << 16), __uint_as_float(res[j] & 0xFFFF0000u)));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = __fadd2_rn(v[j], make_float2(__uint_as_float(res[2 * j]), __uint_as_float(res[2 * j + 1])));
        v[4 + j] = __fadd2_rn(v[4 + j], make_float2(__uint_as_float(res2[2 * j]), __uint_as_float(res2[2 * j + 1])));
      }
    }
  }
  if (p.out) put16<WHOLE>(p, s, p.out, v);
  if (p.amax_out && s.row_ok()) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (WHOLE || 2 * j < s.cols) tmax = max(tmax, __float_as_uint(v[j].x) & 0x7FFFFFFFu);
      if (WHOLE || 2 * j + 1 < s.cols) tmax = max(tmax, __float_as_uint(v[j].y) & 0x7FFFFFFFu);
    }
  }
  if (p.q_codes && s.row_ok()) {
    float z[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[2 * j] = v[j].x;
      z[2 * j + 1] = v[j].y;
    }
    epi_quantize16(p, s.row0 + s.lane, s.col, z);
  }
}

// kEpiFull on small-N tiles, whose operands are swapped (kernel rows are output columns, so that
// neighbouring lanes touch neighbouring elements): finishes 16 consecutive kernel columns, i.e.
// output rows, of kernel row `row` (values already multiplied by the global scales).
__device__ __forceinline__ void epi_finish16(const GemmArgs& p, int row, int col, float (&v)[16]) {
  if (p.bias) {
    const float b = __ldg(p.bias + row);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __fadd_rn(v[j], b);
  }
  auto put = [&](void* out) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (col + j < p.Nk) {
        const int64_t at = static_cast<int64_t>(col + j) * p.ldo + row;
        if (p.out_bf16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v[j]);
        else static_cast<float*>(out)[at] = v[j];
      }
  };
  if (p.pre) put(p.pre);
  with_act(p.act, [&](auto tag) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = act_value<decltype(tag)::value>(v[j]);
  });
  if (p.res) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (col + j < p.Nk) {
        const int64_t at = static_cast<int64_t>(col + j) * p.ldo + row;
        v[j] += p.res_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.res)[at]) : static_cast<const float*>(p.res)[at];
      }
  }
  put(p.out);
}

// Named barrier among the epilogue threads of one pipeline.
__device__ __forceinline__ void epi_sync(int sub, int nthreads) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + sub), "r"(nthreads) : "memory");
}

// Operands as tensor maps (b2, sfb2: the up operand of a gated product).
struct GemmMaps {
  CUtensorMap a, b, sfa, sfb, b2, sfb2;
};

template <int BN, bool MX, int ACC, bool PAIR, bool F8 = false, int EPI = kEpiPlain>
__global__ void __launch_bounds__(Cfg<BN, MX, ACC, PAIR, F8, EPI>::kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSFA, const __grid_constant__ CUtensorMap tmSFB,
                    const __grid_constant__ CUtensorMap tmB2, const __grid_constant__ CUtensorMap tmSFB2,
                    const GemmArgs p) {
  using C = Cfg<BN, MX, ACC, PAIR, F8, EPI>;
  constexpr int S = C::kStages;
  constexpr bool kGated = C::kGated, kWhole = EPI == kEpiFullWhole || EPI == kEpiGatedWhole;
  using Schedule = Sched<BN, kGated ? BN / 2 : BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  const int sub = C::kP == 1 ? 0 : threadIdx.x / 192;  // pipeline of this thread
  const int lt = C::kP == 1 ? threadIdx.x : threadIdx.x % 192;
  const int warp = lt >> 5, lane = lt & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)) +
                  sub * C::kSubBytes;
  uint8_t* misc = smem + S * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + ACC;
  uint64_t* drain = acc_empty + ACC;
  uint64_t* sf_full = drain + 1;                // [kSFSlots]: stage scale factors are in TMEM slot i
  uint64_t* cp_drain = sf_full + C::kSFSlots;   // the copier warps' last copies have completed
  // [S]: a stage's scale factors have landed.  With a separate copier they complete on
  // their own barrier (and are issued first), so that the copier warps move them into TMEM
  // while the stage's operand tiles are still arriving; otherwise they complete on full.
  uint64_t* sf_landed = cp_drain + 1;
  volatile int* s_abort = reinterpret_cast<volatile int*>(sf_landed + S);
  volatile int* s_epi_fail = s_abort + 1;
  volatile int* s_last = s_abort + 2;  // stream-K: this pipeline completes the current tile
  int* s_mt = reinterpret_cast<int*>(misc + 1024);
  int* s_off = s_mt + (kMaxGroups + 1);
  int* s_pt = PAIR ? s_off + (kMaxGroups + 1) : nullptr;
  // A CTA pair (cluster of two) shares one 256 x 256 tile: rank 0, the leader, issues the
  // MMAs and scale-factor copies for both; each CTA loads its own 128 rows of A, its half
  // of B's rows, its A scales and all of the tile's B scales, and stores its 128 rows.
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const int vb = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x) * C::kP + sub;
  const int vg = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x) * C::kP;
  constexpr int kMTile = PAIR ? 256 : 128;
  const int sub_row = static_cast<int>(rank) * 128;

  // prologue (overlaps the tail of the previous kernel under programmatic launch)
  if (lt == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_landed[s], 1);
    }
    for (int a = 0; a < ACC; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], (PAIR ? 2 : 1) * C::kEpiWarps);  // a pair: both CTAs' epilogue warps
    }
    mbar_init(drain, 1);
    for (int i = 0; i < C::kSFSlots; ++i) mbar_init(&sf_full[i], C::kSepCp ? C::kCopiers : 1);
    mbar_init(cp_drain, C::kSepCp ? C::kCopiers : 1);
    *s_abort = 0;
    *s_epi_fail = 0;
    *s_last = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (kGated) tma_prefetch_desc(&tmB2);
    if (PAIR) {
      tma_prefetch_desc(&tmSFA);
      tma_prefetch_desc(&tmSFB);
    }
  }
  if (sub == 0 && warp == 1) {  // one allocation for all pipelines of the CTA
    if constexpr (PAIR) {       // the same columns in both CTAs of the pair
      tmem_alloc_pair(&s_tmem_base, C::kTmemAlloc);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&s_tmem_base, C::kTmemAlloc);
      tmem_relinquish();
    }
  }
  if (p.mode == kModeGrouped && warp == 2) {
    wait_prior_grids();  // the offsets may come from the previous kernel
    // m-tile prefix per group (= scale row-block prefix of the grouped A layout)
    const int E = p.num_groups;
    // (CTA pairs: also the prefix of 256-row tiles, by which they enumerate tiles)
    int carry = 0, carry2 = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      int cnt = 0, cnt2 = 0;
      if (e < E) {
        const int lo = p.offsets[e], hi = p.offsets[e + 1];
        s_off[e] = lo;
        cnt = (hi - lo + 127) / 128;
        cnt2 = (hi - lo + 255) / 256;
      }
      int incl = cnt, incl2 = cnt2;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        const int t2 = __shfl_up_sync(0xFFFFFFFFu, incl2, d);
        if (lane >= d) {
          incl += t;
          incl2 += t2;
        }
      }
      if (e < E) {
        s_mt[e] = carry + incl - cnt;
        if (PAIR) s_pt[e] = carry2 + incl2 - cnt2;
      }
      carry += __shfl_sync(0xFFFFFFFFu, incl, 31);
      carry2 += __shfl_sync(0xFFFFFFFFu, incl2, 31);
    }
    if (lane == 0) {
      s_mt[E] = carry;
      if (PAIR) s_pt[E] = carry2;
      s_off[E] = p.offsets[E];
    }
  }
  tc_fence_before();
  __syncthreads();
  // a pair: the peer's barriers are initialised before this CTA's loads and arrivals reach them
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base + sub * C::kTmemCols;
  const uint32_t sf_col0 = ACC * BN;
  // copies one stage's scale-factor atoms (A's, then B's row-blocks) into a TMEM slot
  auto copy_stage_sf = [&](uint32_t st, uint32_t sfa_t, int kb) {
    const uint32_t sfb_t = sfa_t + C::kSFACols;
    const int atoms = min(C::kAtomsKT, p.sf_atoms_k - kb * C::kAtomsKT);
    for (int a = 0; a < atoms; ++a) tc_cp_sf_atom(sfa_t + a * 4, smem_desc_sf(st + C::kABytes + C::kBBytes + a * 512));
#pragma unroll
    for (int rb = 0; rb < C::kNRB; ++rb)
      for (int a = 0; a < atoms; ++a)
        tc_cp_sf_atom(sfb_t + (a * C::kNRB + rb) * 4,
                      smem_desc_sf(st + C::kABytes + C::kBBytes + C::kSFABytes + (rb * C::kAtomsKT + a) * 512));
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ producer
      // swapped decode: the weights (A here) are read once -> evict first; the small
      // activations (B) are re-read by every CTA -> keep
      // otherwise both operands are re-read by other tiles -> keep (the output is stored
      // with the streaming hint, so that it does not push them out of L2)
      const uint64_t pol_a = p.transposed ? l2_policy_evict_first() : l2_policy_evict_last();
      const uint64_t pol_b = l2_policy_evict_last();
      // Loads of one stage: the A box and A scales ("a" side), the B box and B scales.
      auto load_side = [&](int st_idx, const Work& w, int kb, bool side_a) {
        uint8_t* st = smem + st_idx * C::kStageBytes;
        const int atoms = min(C::kAtomsKT, p.sf_atoms_k - kb * C::kAtomsKT);
        const uint32_t sf_bytes = static_cast<uint32_t>(atoms) * 512u;
        const int64_t koff = static_cast<int64_t>(kb) * C::kAtomsKT * 512;
        if constexpr (PAIR) {
          // every box in full (out-of-range rows read as zero), so that the leader can
          // expect a fixed byte count from both CTAs on its own barriers
          const uint32_t c_full = cluster_addr(smem_u32(&full[st_idx]), 0);
          const uint32_t c_sf = cluster_addr(smem_u32(&sf_landed[st_idx]), 0);
          if (side_a) {
            tma_load_2d_pair(st + C::kABytes + C::kBBytes, &tmSFA, c_sf, 0,
                             static_cast<int>((w.sfa_rb * p.sfa_rb_bytes + koff) / 256), pol_a);
            tma_load_2d_pair(st, &tmA, c_full, kb * 128, w.a_row, pol_a);
          } else {
#pragma unroll
            for (int rb = 0; rb < C::kNRB; ++rb)
              tma_load_2d_pair(st + C::kABytes + C::kBBytes + C::kSFABytes + rb * C::kAtomsKT * 512,
                               kGated && rb ? &tmSFB2 : &tmSFB, c_sf, 0,
                               static_cast<int>((w.sfb_off + (kGated ? 0 : rb) * p.sfb_rb_bytes + koff) / 256), pol_b);
            // gated: the leader holds the tile's gate rows, the other CTA its up rows
            tma_load_2d_pair(st + C::kABytes, kGated && !leader ? &tmB2 : &tmB, c_full, kb * 128, w.b_row, pol_b);
          }
          (void)sf_bytes;
          return;
        }
        uint64_t* sf_bar = C::kSepCp ? &sf_landed[st_idx] : &full[st_idx];
        if (side_a) {
          bulk_load(st + C::kABytes + C::kBBytes, p.sfa + w.sfa_rb * p.sfa_rb_bytes + koff, sf_bytes, sf_bar, pol_a);
          tma_load_2d(st, &tmA, &full[st_idx], kb * 128, w.a_row, pol_a);
        } else {
          if constexpr (kGated) {
            bulk_load(st + C::kABytes + C::kBBytes + C::kSFABytes, p.sfb + w.sfb_off + koff, sf_bytes, sf_bar, pol_b);
            bulk_load(st + C::kABytes + C::kBBytes + C::kSFABytes + C::kAtomsKT * 512, p.sfb2 + w.sfb_off + koff,
                      sf_bytes, sf_bar, pol_b);
            tma_load_2d(st + C::kABytes, &tmB, &full[st_idx], kb * 128, w.b_row, pol_b);
            tma_load_2d(st + C::kABytes + C::kBBytes / 2, &tmB2, &full[st_idx], kb * 128, w.b_row, pol_b);
            return;
          }
          const int rb0 = w.n0 / 128;
#pragma unroll
          for (int rb = 0; rb < C::kNRB; ++rb)
            if (rb0 + rb < p.sfb_rbs)
              bulk_load(st + C::kABytes + C::kBBytes + C::kSFABytes + rb * C::kAtomsKT * 512,
                        p.sfb + w.sfb_off + rb * p.sfb_rb_bytes + koff, sf_bytes, sf_bar, pol_b);
          tma_load_2d(st + C::kABytes, &tmB, &full[st_idx], kb * 128, w.b_row, pol_b);
        }
      };
      auto stage_sf_bytes = [&](const Work& w, int kb) -> uint32_t {
        const int atoms = min(C::kAtomsKT, p.sf_atoms_k - kb * C::kAtomsKT);
        const uint32_t sf_bytes = static_cast<uint32_t>(atoms) * 512u;
        if (kGated) return sf_bytes * 3;
        const int rb0 = w.n0 / 128;
        int nrb = 0;
#pragma unroll
        for (int rb = 0; rb < C::kNRB; ++rb) nrb += (rb0 + rb < p.sfb_rbs) ? 1 : 0;
        return sf_bytes * (1 + nrb);
      };
      // With an independent operand, the first ring-full of stages loads only that side,
      // then waits for the preceding kernel, then issues the other side of those stages.
      const bool early = p.indep != 0;
      const bool early_a = p.indep == 1;
      int npend = 0;
      bool replayed = !early;
      auto replay = [&]() {
        wait_prior_grids();
        Schedule rs(p, s_mt, s_off, vb, vg, kMTile, sub_row, s_pt);
        Work rw;
        int j = 0;
        while (j < npend && rs.next(rw))
          for (int kb = rw.kb0; kb < rw.kb1 && j < npend; ++kb, ++j) load_side(j, rw, kb, !early_a);
        replayed = true;
      };
      if (!early) wait_prior_grids();
      Schedule sch(p, s_mt, s_off, vb, vg, kMTile, sub_row, s_pt);
      Work w;
      int stage = 0;
      uint32_t phase = 0, issued = 0, issued_par = 0;
      bool ok = true;
      // operand bytes a stage's tensor copies complete: a 4-bit operand of the mixed-format
      // MMA counts its packed bytes (half its footprint in shared memory)
      uint32_t ab_tx = C::kABytes + C::kBBytes;
      if constexpr (F8)
        ab_tx = ((p.f8_fmt & 7u) == kFmtE2M1 ? C::kABytes / 2 : C::kABytes) +
                (((p.f8_fmt >> 3) & 7u) == kFmtE2M1 ? C::kBBytes / 2 : C::kBBytes);
      while (ok && sch.next(w)) {
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, s_abort)) {
            latch_timeout(s_abort, p.status);
            ok = false;
            break;
          }
          if constexpr (PAIR) {
            if (leader) {  // the leader's barriers count the boxes of both CTAs
              mbar_arrive_expect_tx(&sf_landed[stage], 2 * (C::kSFABytes + C::kSFBBytes));
              mbar_arrive_expect_tx(&full[stage], 2 * ab_tx);
            }
          } else if constexpr (C::kSepCp) {
            mbar_arrive_expect_tx(&sf_landed[stage], stage_sf_bytes(w, kb));
            mbar_arrive_expect_tx(&full[stage], ab_tx);
          } else {
            mbar_arrive_expect_tx(&full[stage], C::kABytes + C::kBBytes + stage_sf_bytes(w, kb));
          }
          if (!replayed) {
            load_side(stage, w, kb, early_a);
            if (++npend == S) replay();
          } else {
            load_side(stage, w, kb, true);
            load_side(stage, w, kb, false);
          }
          issued |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (ok && !replayed) replay();
      // let every issued copy land before the CTA's shared memory goes away (a pair's
      // leader waits for both CTAs' boxes: they complete on its barriers)
      if (*s_abort && leader) {
        for (int s = 0; s < S; ++s)
          if (issued & (1u << s)) {
            volatile int no_abort = 0;
            mbar_wait(&full[s], (issued_par >> s) & 1u, &no_abort);
            if (C::kSepCp) mbar_wait(&sf_landed[s], (issued_par >> s) & 1u, &no_abort);
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ MMA issuer
      Schedule sch(p, s_mt, s_off, vb, vg, kMTile, sub_row, s_pt);
      const uint32_t smem_base = smem_u32(smem);
      Work w;
      int stage = 0, iter = 0, nstage = 0;
      uint32_t phase = 0, slot = 0;
      bool ok = true;
      while (ok && sch.next(w)) {
        const int acc = iter % ACC;
        if (!mbar_wait(&acc_empty[acc], ((iter / ACC) & 1) ^ 1, s_abort)) {
          latch_timeout(s_abort, p.status);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * BN;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, s_abort)) {
            latch_timeout(s_abort, p.status);
            ok = false;
            break;
          }
          const uint32_t st = smem_base + stage * C::kStageBytes;
          const uint32_t sfa_t = tmem + sf_col0 + slot * C::kSFSlot;
          const uint32_t sfb_t = sfa_t + C::kSFACols;
          if constexpr (C::kSepCp) {
            // the copier warps have put this stage's scale factors into the slot
            if (!mbar_wait(&sf_full[slot], (nstage / C::kSFSlots) & 1, s_abort)) {
              latch_timeout(s_abort, p.status);
              ok = false;
              break;
            }
            tc_fence_after();
          } else {
            tc_fence_after();
            copy_stage_sf(st, sfa_t, kb);
          }
          ++nstage;
          const int krem = p.K - kb * (F8 ? 128 : 256);
          const int nk = F8 ? (krem >= 128 ? 4 : (krem + 31) / 32) : (krem >= 256 ? 4 : (krem + 63) / 64);
          const uint64_t adesc = smem_desc_sw128(st);
          const uint64_t bdesc = smem_desc_sw128(st + C::kABytes);
          if constexpr (F8) {
            // four K = 32 MMAs over the stage's 128-byte rows (one byte per element of
            // either format); MMA k reads byte k of each row's 32-bit scale word
            for (int k = 0; k < nk; ++k) {
              const uint32_t sfid = static_cast<uint32_t>(k);
              const uint32_t idesc = mma_idesc_f8(BN, p.f8_fmt & 7u, (p.f8_fmt >> 3) & 7u, sfid, sfid, kMTile);
              const uint32_t accum = (kb > w.kb0 || k > 0) ? 1u : 0u;
              if constexpr (PAIR)
                tc_mma_mxf8f6f4_pair(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, sfa_t | (sfid << 30),
                                     sfb_t | (sfid << 30), accum);
              else
                tc_mma_mxf8f6f4(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, sfa_t | (sfid << 30),
                                sfb_t | (sfid << 30), accum);
            }
          } else {
          for (int k = 0; k < nk; ++k) {
            const uint32_t a_idx = MX ? (k >> 1) : k;
            const uint32_t sfid = MX ? (k & 1) * 2 : 0;
            const uint32_t idesc = mma_idesc(BN, MX, sfid, sfid, kMTile);
            const uint32_t accum = (kb > w.kb0 || k > 0) ? 1u : 0u;
            const uint32_t ta = (sfa_t + a_idx * 4) | (sfid << 30);
            const uint32_t tb = (sfb_t + a_idx * C::kNRB * 4) | (sfid << 30);
            if constexpr (PAIR && MX)
              tc_mma_mxfp4_pair(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, ta, tb, accum);
            else if constexpr (PAIR)
              tc_mma_nvfp4_pair(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, ta, tb, accum);
            else if constexpr (MX)
              tc_mma_mxfp4(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, ta, tb, accum);
            else
              tc_mma_nvfp4(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, ta, tb, accum);
          }
          }
          if constexpr (PAIR)
            tc_commit_pair_mc(&empty[stage], 3);  // frees the stage in both CTAs
          else
            tc_commit(&empty[stage]);
          if (++slot == C::kSFSlots) slot = 0;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (PAIR)
          tc_commit_pair_mc(&acc_full[acc], 3);  // both CTAs' epilogues
        else
          tc_commit(&acc_full[acc]);
        ++iter;
      }
      // make sure no MMA still writes TMEM when it is freed
      if constexpr (PAIR)
        tc_commit_pair(drain);
      else
        tc_commit(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort);
    }
  } else if (C::kSepCp && warp >= 2 + C::kEpiWarps) {
    const int cw = warp - 2 - C::kEpiWarps;  // 0: A's atoms; 1 + rb: B's row-block rb
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ scale-factor copier
      // Stage n's atoms go to TMEM slot n % kSFSlots once they have landed and the
      // MMAs of stage n - kSFSlots (the slot's previous user) have completed; each slot's
      // copies are committed to sf_full[slot] for the MMA thread.
      Schedule sch(p, s_mt, s_off, vb, vg, kMTile, sub_row, s_pt);
      const uint32_t smem_base = smem_u32(smem);
      Work w;
      int stage = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && sch.next(w)) {
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&sf_landed[stage], phase, s_abort)) {
            latch_timeout(s_abort, p.status);
            ok = false;
            break;
          }
          if (n >= C::kSFSlots) {
            const int prev = n - C::kSFSlots;
            if (!mbar_wait(&empty[prev % S], (prev / S) & 1, s_abort)) {
              latch_timeout(s_abort, p.status);
              ok = false;
              break;
            }
          }
          tc_fence_after();
          const uint32_t sl = n % C::kSFSlots;
          {
            const uint32_t st = smem_base + stage * C::kStageBytes;
            const uint32_t sfa_t = tmem + sf_col0 + sl * C::kSFSlot;
            const int atoms = min(C::kAtomsKT, p.sf_atoms_k - kb * C::kAtomsKT);
            auto cp = [&](uint32_t taddr, uint64_t sdesc) {
              if constexpr (PAIR)
                tc_cp_sf_atom_pair(taddr, sdesc);
              else
                tc_cp_sf_atom(taddr, sdesc);
            };
            if (cw == 0) {
              for (int a = 0; a < atoms; ++a) cp(sfa_t + a * 4, smem_desc_sf(st + C::kABytes + C::kBBytes + a * 512));
            } else {
              const int rb = cw - 1;
              for (int a = 0; a < atoms; ++a)
                cp(sfa_t + C::kSFACols + (a * C::kNRB + rb) * 4,
                   smem_desc_sf(st + C::kABytes + C::kBBytes + C::kSFABytes + (rb * C::kAtomsKT + a) * 512));
            }
          }
          if constexpr (PAIR)
            tc_commit_pair(&sf_full[sl]);
          else
            tc_commit(&sf_full[sl]);
          ++n;
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      // no copy may still write TMEM when it is freed
      if constexpr (PAIR)
        tc_commit_pair(cp_drain);
      else
        tc_commit(cp_drain);
      volatile int no_abort = 0;
      mbar_wait(cp_drain, 0, &no_abort);
    }
  } else if (warp >= 2 && warp < 2 + C::kEpiWarps) {
    // ------------------------------------------------------------ epilogue
    // a warp reads the TMEM lane quarter given by its warp index in the CTA, modulo 4,
    // and (with eight epilogue warps) the column half given by its warp index over 4
    const int q = (threadIdx.x >> 5) & 3;
    const int rl = q * 32 + lane;     // accumulator row (TMEM lane) of this thread
    const int et = lt - 32 * 2;  // 0 .. 32 * kEpiWarps - 1
    constexpr int CH = C::kEpiCols;
    const int c0 = ((warp - 2) >> 2) * CH;  // first accumulator column of this thread
    // BF16 row-major tiles whose columns are all in range are converted into registers
    // and TMEM is handed back to the MMA thread before the stores, so that they overlap
    // the next tile's MMAs
    const bool early_release = C::kSepCp && p.mode != kModeStreamK && p.out && p.out_bf16 && !p.transposed &&
                               p.vec_store && !p.q_codes;
    // hands an accumulator back to the MMA thread (a pair's leader counts both CTAs' warps)
    auto release_acc = [&](int a) {
      if constexpr (PAIR)
        mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[a]), 0));
      else
        mbar_arrive(&acc_empty[a]);
    };
    wait_prior_grids();               // the global scales come from earlier kernels
    allow_dependents();
    const float ga = p.ga ? *p.ga : 1.0f;
    uint32_t tmax = 0;                // max |result| over this thread's values (amax_out)
    Schedule sch(p, s_mt, s_off, vb, vg, kMTile, sub_row, s_pt);
    Work w;
    int iter = 0;
    while (sch.next(w)) {
      const int acc = iter % ACC;
      const uint32_t par = (iter / ACC) & 1;
      if constexpr (C::kLong && !kGated) {
        // this thread's piece of the residual comes into L2 while the tile is being multiplied
        if (p.res && p.mode != kModeStreamK && rl < w.rows_valid && w.n0 + c0 < p.Nk) {
          const int64_t at = static_cast<int64_t>(w.out_row0 + rl) * p.ldo + w.n0 + c0;
          const uint8_t* r = static_cast<const uint8_t*>(p.res) + at * (p.res_bf16 ? 2 : 4);
          prefetch_l2(r);
          if (!p.res_bf16 && w.n0 + c0 + 32 < p.Nk) prefetch_l2(r + 128);
        }
      }
      float* const s_bias = reinterpret_cast<float*>(misc + (C::kLong ? C::kBiasOff : 0)) + (iter & 1) * BN;
      if constexpr (C::kLong) {
        // the tile's biases, before the barrier below (two buffers: a warp may still read the
        // last tile's, but not the one's before)
        if (et < BN && p.bias_any) {
          const float* b = kGated && et >= BN / 2 ? p.bias2 : p.bias;
          const int col = w.n0 + (kGated ? et % (BN / 2) : et);
          s_bias[et] = b && col < p.Nk ? __ldg(b + w.group * p.bias_group + col) : 0.0f;
        }
      }
      // the epilogue warps decide together whether to go on, so that none of them
      // is left behind at a named barrier
      if (et == 0 && !mbar_wait(&acc_full[acc], par, s_abort)) {
        latch_timeout(s_abort, p.status);
        *s_epi_fail = 1;
      }
      epi_sync(sub, 32 * C::kEpiWarps);
      if (*s_epi_fail) break;
      tc_fence_after();
      const float gb = p.gb ? p.gb[w.group] : 1.0f;
      const float scale = ga * gb;
      float scale2 = 0.0f;  // the up columns' scale
      if constexpr (kGated) scale2 = ga * (p.gb2 ? p.gb2[w.group] : 1.0f);
      const bool row_ok = rl < w.rows_valid;
      const int row = w.out_row0 + rl;
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
      bool released = false;
      if constexpr (EPI != kEpiPlain) {
        if constexpr (C::kLong) {
          const int rows = max(0, min(32, w.rows_valid - q * 32));  // of this warp
          bool finish = true;
          if (!kWhole && p.mode == kModeStreamK) {
            // Partial sums to the workspace (rows of ws_ld floats; gated: G's, then U's).  The
            // pipeline whose sums complete the tile's K range finishes it (as below).
#pragma unroll 1
            for (int cw = c0; cw < c0 + CH; cw += 32) {
              uint32_t rr[32];
              tmem_ld32(taddr + cw, rr);
              tmem_ld_wait();
              const int half = kGated && cw >= BN / 2 ? 1 : 0;
              const int col = w.n0 + cw - half * (BN / 2);
              float* dst = p.ws + (static_cast<int64_t>(half) * p.Mk + row) * p.ws_ld + col;
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                if (row_ok && col + j < p.ws_ld)
                  red_add_v4(dst + j, __uint_as_float(rr[j]), __uint_as_float(rr[j + 1]), __uint_as_float(rr[j + 2]),
                             __uint_as_float(rr[j + 3]));
              __syncwarp();  // the next TMEM load takes the whole warp
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) release_acc(acc);
            __threadfence();
            epi_sync(sub, 32 * C::kEpiWarps);
            if (et == 0) {
              __threadfence();
              const int covered = w.kb1 - w.kb0;
              const int before = atomicAdd(p.tile_cnt + w.tile, covered);
              *s_last = before + covered == p.num_kb ? 1 : 0;
            }
            epi_sync(sub, 32 * C::kEpiWarps);
            finish = *s_last;
            if (finish) {
              __threadfence();
              if (et == 0) p.tile_cnt[w.tile] = 0;
            }
          }
          // 32 sums per thread at a time; the last 32 are in registers when TMEM goes back to the
          // MMA thread, so that their work overlaps the next tile's MMAs
          constexpr int kOut = kGated ? 16 : 32;  // output columns per step
          const int oc = kGated ? c0 / 2 : c0;
          if (finish) {
#pragma unroll 1
            for (int b = 0; b < CH / 32; ++b) {
              uint32_t rr[32];
              const int o = oc + b * kOut;
              if (!kWhole && p.mode == kModeStreamK) {
                if (row_ok) {
                  float* src = p.ws + static_cast<int64_t>(row) * p.ws_ld;
                  take_raw16(src, w.n0 + o, p.ws_ld, rr);
                  take_raw16(kGated ? src + static_cast<int64_t>(p.Mk) * p.ws_ld : src, w.n0 + o + (kGated ? 0 : 16),
                             p.ws_ld, rr + 16);
                }
              } else {
                // (One site of these loads: copies of it, per activation or per kind of tile,
                // spill whatever the register budget.  Warps without a valid row read TMEM all
                // the same: the loads stay convergent.)
                if constexpr (kGated) {
                  tmem_ld16(taddr + o, *reinterpret_cast<uint32_t(*)[16]>(rr));
                  tmem_ld16(taddr + BN / 2 + o, *reinterpret_cast<uint32_t(*)[16]>(rr + 16));
                } else {
                  tmem_ld32(taddr + o, rr);
                }
                tmem_ld_wait();
                if (b == CH / 32 - 1) {
                  tc_fence_before();
                  __syncwarp();
                  if (lane == 0) release_acc(acc);
                }
              }
#pragma unroll
              for (int c = 0; c < kOut; c += 16) {
                const int col = w.n0 + o + c, cols = min(16, p.Nk - col);  // (whole: 16, or none)
                if (rows > 0 && cols > 0) {  // warp-uniform
                  const EpiSpot spot{row - lane, rows, lane, col, cols, p.sectors && cols == 16};
                  const float* b1 = p.bias ? s_bias + o + c : nullptr;
                  const float* b2 = kGated && p.bias2 ? s_bias + BN / 2 + o + c : nullptr;
                  epi_rows<kGated, kWhole>(p, spot, b1, b2, scale, scale2, rr + c, tmax);
                }
              }
              __syncwarp();  // the next TMEM load takes the whole warp
            }
          }
          ++iter;
          continue;
        } else if (p.mode != kModeStreamK) {
          // small-N tiles: finished as they are read
          if (q * 32 < w.rows_valid) {  // warp-uniform
#pragma unroll 1
            for (int c = c0; c < c0 + CH; c += 16) {
              uint32_t rg[16];
              tmem_ld16(taddr + c, rg);
              tmem_ld_wait();
              const int col = w.n0 + c;
              if (row_ok && col < p.Nk) {
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(rg[j]) * scale;
                epi_finish16(p, row, col, v);
              }
              __syncwarp();  // the next TMEM load takes the whole warp
            }
          }
        } else if (q * 32 < w.rows_valid) {
          // small-N tiles, stream-K: partial sums to the workspace
#pragma unroll 1
          for (int c = c0; c < c0 + CH; c += 16) {
            uint32_t rr[16];
            tmem_ld16(taddr + c, rr);
            tmem_ld_wait();
            const int col = w.n0 + c;
            if (row_ok && col < p.Nk) {
              float* dst = p.ws + static_cast<int64_t>(row) * p.Nk + col;
              if ((p.Nk & 3) == 0 && col + 16 <= p.Nk) {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                  red_add_v4(dst + j, __uint_as_float(rr[j]), __uint_as_float(rr[j + 1]), __uint_as_float(rr[j + 2]),
                             __uint_as_float(rr[j + 3]));
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (col + j < p.Nk) atomicAdd(dst + j, __uint_as_float(rr[j]));
              }
            }
            __syncwarp();  // the next TMEM load takes the whole warp
          }
        }
      } else
      if (q * 32 < w.rows_valid && early_release && w.n0 + BN <= p.Nk) {  // warp-uniform
        uint32_t pk[CH / 2];  // this thread's columns [c0, c0 + CH) as scaled BF16 pairs
        // 32-column TMEM loads, one wait per load: the hand-back of the accumulator
        // waits for few TMEM round trips
        constexpr int kLdBatch = CH >= 32 ? 32 : CH;
        static_assert(CH % kLdBatch == 0 && kLdBatch % 16 == 0, "TMEM load batches");
#pragma unroll
        for (int cb = 0; cb < CH; cb += kLdBatch) {
          uint32_t rr[kLdBatch];
          if constexpr (kLdBatch % 32 == 0) {
#pragma unroll
            for (int h = 0; h < kLdBatch; h += 32) tmem_ld32(taddr + c0 + cb + h, rr + h);
          } else {
            tmem_ld16(taddr + c0 + cb, *reinterpret_cast<uint32_t(*)[16]>(rr));
          }
          tmem_ld_wait();
#pragma unroll
          for (int cw = 0; cw < kLdBatch; cw += 16) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(rr[cw + j]) * scale;
            if (p.bias || p.act) epi_bias_act(p, row, w.n0 + c0 + cb + cw, v);
            if (p.amax_out) {  // (a mask, no branch by rows: the next TMEM load takes the whole warp)
              const uint32_t keep = row_ok ? 0x7FFFFFFFu : 0u;
#pragma unroll
              for (int j = 0; j < 16; ++j) tmax = max(tmax, __float_as_uint(v[j]) & keep);
            }
#pragma unroll
            for (int j = 0; j < 16; j += 2) pk[(cb + cw + j) / 2] = pack_bf16x2(v[j], v[j + 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) release_acc(acc);
        released = true;
        if (row_ok) {
          __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(p.out) + static_cast<int64_t>(row) * p.ldo;
#pragma unroll
          for (int c = 0; c < CH; c += 8)  // streaming stores: the output is not read back here
            __stcs(reinterpret_cast<uint4*>(orow + w.n0 + c0 + c),
                   make_uint4(pk[c / 2], pk[c / 2 + 1], pk[c / 2 + 2], pk[c / 2 + 3]));
        }
      } else if (q * 32 < w.rows_valid) {  // warp-uniform: warps without a valid row skip TMEM
        // up to 64 columns per TMEM round trip (32 with eight epilogue warps), one wait
        constexpr int CW = C::kSepCp ? 32 : CH >= 64 ? 64 : CH;
#pragma unroll 1
        for (int cw = c0; cw < c0 + CH; cw += CW) {
          uint32_t rr[CW / 16][16];
#pragma unroll
          for (int h = 0; h < CW / 16; ++h) tmem_ld16(taddr + cw + h * 16, rr[h]);
          tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < CW / 16; ++h) {
          const int c = cw + h * 16;
          const uint32_t (&r)[16] = rr[h];
          const int col = w.n0 + c;
          if (!row_ok || col >= p.Nk) continue;
          if (p.mode == kModeStreamK) {
            float* dst = p.ws + static_cast<int64_t>(row) * p.Nk + col;
            if ((p.Nk & 3) == 0 && col + 16 <= p.Nk) {
#pragma unroll
              for (int j = 0; j < 16; j += 4)
                red_add_v4(dst + j, __uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]),
                           __uint_as_float(r[j + 3]));
            } else {
              for (int j = 0; j < 16 && col + j < p.Nk; ++j) atomicAdd(dst + j, __uint_as_float(r[j]));
            }
          } else {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]) * scale;
            epi_row16(p, row, col, v, tmax);
          }
        }
          __syncwarp();  // the next TMEM loads take the whole warp
        }
      }
      if (!released) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) release_acc(acc);
      }
      ++iter;
      if (p.mode == kModeStreamK) {
        // The pipeline whose partial sums complete the tile's K range writes the tile:
        // every pipeline publishes its reductions (fence), then adds the K steps it
        // covered to the tile's counter; the one that brings it to num_kb reads the
        // sums back from L2, scales, converts, stores, and clears sums and counter.
        __threadfence();
        epi_sync(sub, 32 * C::kEpiWarps);
        if (et == 0) {
          __threadfence();
          const int covered = w.kb1 - w.kb0;
          const int before = atomicAdd(p.tile_cnt + w.tile, covered);
          *s_last = before + covered == p.num_kb ? 1 : 0;
        }
        epi_sync(sub, 32 * C::kEpiWarps);
        if (*s_last) {
          __threadfence();
          if constexpr (EPI != kEpiPlain) {
            if (row_ok) {
#pragma unroll 1
              for (int c = c0; c < c0 + CH; c += 16) {
                const int col = w.n0 + c;
                if (col >= p.Nk) break;
                float v[16];
                take_sums16(p.ws + static_cast<int64_t>(row) * p.Nk, col, p.Nk, scale, v);
                epi_finish16(p, row, col, v);
              }
            }
          } else
          if (row_ok) {
            float* src = p.ws + static_cast<int64_t>(row) * p.Nk;
            for (int c = c0; c < c0 + CH; c += 16) {
              const int col = w.n0 + c;
              if (col >= p.Nk) break;
              float v[16];
              if ((p.Nk & 3) == 0 && col + 16 <= p.Nk) {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  const float4 t = __ldcg(reinterpret_cast<const float4*>(src + col + j));
                  __stcg(reinterpret_cast<float4*>(src + col + j), make_float4(0.f, 0.f, 0.f, 0.f));
                  v[j] = t.x * scale;
                  v[j + 1] = t.y * scale;
                  v[j + 2] = t.z * scale;
                  v[j + 3] = t.w * scale;
                }
              } else {
                for (int j = 0; j < 16; ++j) {
                  v[j] = 0.0f;
                  if (col + j < p.Nk) {
                    v[j] = __ldcg(src + col + j) * scale;
                    __stcg(src + col + j, 0.0f);
                  }
                }
              }
              epi_row16(p, row, col, v, tmax);
            }
          }
          if (et == 0) p.tile_cnt[w.tile] = 0;
        }
      }
    }
    if (p.amax_out) {  // one atomic per warp: non-negative float bits order as integers
      tmax = __reduce_max_sync(0xFFFFFFFFu, tmax);
      if (lane == 0 && tmax) atomicMax(p.amax_out, tmax);
    }
  }

  tc_fence_before();
  __syncthreads();
  // a pair: neither CTA frees TMEM or leaves (its shared memory is the peer's operand and
  // barrier target) before both are done
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  if (sub == 0 && warp == 1) {
    __syncwarp();
    if constexpr (PAIR)
      tmem_dealloc_pair(s_tmem_base, C::kTmemAlloc);
    else
      tmem_dealloc(s_tmem_base, C::kTmemAlloc);
  }
}

template <int BN, bool MX, int ACC, bool PAIR, bool F8 = false, int EPI = kEpiPlain>
static cudaError_t run(const GemmMaps& tm, const GemmArgs& a, int64_t units, cudaStream_t st) {
  using C = Cfg<BN, MX, ACC, PAIR, F8, EPI>;
  auto kern = fp4_gemm_kernel<BN, MX, ACC, PAIR, F8, EPI>;
  // the shared-memory opt-in is per device; set it once per (kernel, device)
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = cudaSuccess;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  // programmatic dependent launch: the prologue (barriers, TMEM, descriptor prefetch,
  // and loads of an operand the caller marked as ready) overlaps the previous kernel on
  // the stream; everything else waits for it
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int grid = 0;
  if constexpr (PAIR) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    // persistent: as many pairs as can be resident at once (asked once per device)
    static int max_pairs[64] = {0};
    int pairs = (dev >= 0 && dev < 64) ? max_pairs[dev] : 0;
    if (pairs <= 0) {
      cfg.gridDim = dim3(2 * static_cast<unsigned>(num_sms() / 2));
      e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (pairs <= 0) return cudaErrorInvalidConfiguration;
      if (dev >= 0 && dev < 64) max_pairs[dev] = pairs;
    }
    // (grouped schedules count their tiles on the device: every pair)
    grid = 2 * static_cast<int>(a.mode == kModeGrouped ? pairs : std::max<int64_t>(1, std::min<int64_t>(units, pairs)));
  } else {
    grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((units + C::kP - 1) / C::kP, num_sms())));
    if (a.mode == kModeGrouped) grid = num_sms();
  }
  cfg.gridDim = dim3(grid);
  return cudaLaunchKernelEx(&cfg, kern, tm.a, tm.b, tm.sfa, tm.sfb, tm.b2, tm.sfb2, a);
}

}  // namespace fp4
