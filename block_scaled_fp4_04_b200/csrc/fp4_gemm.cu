// fp4_gemm.cu -- block-scaled FP4 GEMM on the sm_100a tensor cores (tcgen05).
//
// Computes D = gA * gB * (A_hat . B_hat^T) where A_hat / B_hat are E2M1 codes times
// their block scales ("Rubin FP4 GEMM overview", yfxerp.com, 3.1: the block scale
// factors are re-applied on the FP32 accumulators; 3.2: global -> shared -> tensor core
// -> FP32 accumulators -> epilogue; 4.2: the global scale product is fused into the
// epilogue so no extra pass over memory is needed).
//
// Structure (one CTA per SM, persistent).  128/256-wide tiles, one pipeline per CTA:
//   warp 0      TMA producer: per 256-wide K step, one 128 x 128-byte box of A, one
//               BN x 128-byte box of B (both 128-byte swizzled) on the stage's barrier,
//               and the matching 512-byte scale-factor atoms (issued first) on a
//               barrier of their own, into a STAGES-deep ring.
//   warp 1      TMEM owner; lane 0 issues tcgen05.mma.kind::mxf4nvf4 (NVFP4,
//               scale_vec::4X, UE4M3) or kind::mxf4 (MXFP4, scale_vec::2X, UE8M0),
//               M=128, N=BN, K=64 each, accumulating in TMEM; commits free the ring
//               slot and, at the end of a tile, hand the accumulator to the epilogue.
//   warps 2..9  epilogue: two warps per TMEM lane quarter (warp w reads lanes
//               32*(w%4)..+31), one per column half; multiply by gA*gB, BF16 (RNE) or
//               FP32 stores.  BF16 row-major tiles are packed into registers and the
//               accumulator is handed back before the stores.
//   warps 10..  scale-factor copiers (one for A's atoms, one per 128-row block of B's):
//               tcgen05.cp of a stage's atoms into a TMEM slot, replicated to the four
//               sub-partitions, while the MMA thread works on earlier stages.
// 256-wide tiles with M >= 256 run on CTA pairs (clusters of two): the pair computes a
// 256 x 256 tile with M=256 MMAs (tcgen05 .cta_group::2) issued by the leader; each CTA
// loads its own 128 rows of A and half of B's rows (so each SM moves a third fewer
// operand bytes per MMA), all TMA bytes complete on the leader's barriers, and the
// leader's commits arrive on both CTAs' barriers.
// Small-N tiles (16..64) run two independent pipelines of 6 warps per CTA, whose MMA
// thread also issues the scale-factor copies.
// Schedules: whole tiles (grouped raster for L2 reuse); stream-K over (tile, K-step)
// units when there are too few tiles to fill the SMs -- each CTA adds its FP32 partial
// tiles into a workspace with vector reductions, and the one whose part completes a
// tile's K range reads it back, scales, converts, stores and clears it; grouped MoE
// tiles enumerated on the device from the expert offsets.
// Decode-sized M (<= 64) runs with the operands swapped: the weight rows fill MMA-M and
// the few activation rows are MMA-N (16/32/64), which keeps the tensor-core work held per
// pipeline stage small and therefore many stages of weights in flight.
// Scale-factor TMEM addresses are always multiples of 4 columns (one 128-row atom per
// 4 columns); the hardware faults on other alignments.
// Launched with programmatic dependent launch: the prologue overlaps the previous
// kernel; global memory is touched only after griddepcontrol.wait.
// No TMA multicast is used anywhere.  Every wait is bounded (fp4_ptx.cuh); on a timeout
// the CTA latches the status word, drains its in-flight copies and MMAs, frees TMEM and
// returns.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "fp4_gemm_kernel.cuh"
#include "fp4_gemm_host.h"

namespace fp4 {

// ---------------------------------------------------------------------- host side
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
}

// [rows, inner_bytes] uint8 matrix, boxes of box_rows x 128 bytes, 128-byte swizzle,
// out-of-bounds elements read as zero.
static bool encode_map(CUtensorMap* m, const void* base, uint64_t inner_bytes, uint64_t rows, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {inner_bytes, rows};
  const cuuint64_t strides[1] = {inner_bytes};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, k] E2M1 codes, packed two per byte in global memory (row pitch k / 2 bytes),
// copied into shared memory one byte per element: each 16 codes (8 bytes) followed by an
// 8-byte gap, the operand layout of the kind::mxf8f6f4 MMA.  CUDA's documented limits for
// this data type: a 32-byte aligned base, k a multiple of 128, a row pitch that is a
// multiple of 32 bytes, and boxes 128 elements wide.
static bool encode_map_u4(CUtensorMap* m, const void* base, uint64_t k, uint64_t rows, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {k, rows};
  const cuuint64_t strides[1] = {k / 2};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Small host cache of encoded tensor maps keyed by (address, shape, box): decode-style
// callers pass the same buffers every step, and encoding costs host time on every call.
// A map only describes addresses, so a stale entry is just another valid encoding.
namespace {
struct MapCacheEntry {
  const void* base;
  uint64_t inner, rows;
  uint32_t box;
  CUtensorMap map;
};
}  // namespace
bool make_tensor_map_u8(CUtensorMap* m, const void* base, uint64_t inner_bytes, uint64_t rows, uint32_t box_rows) {
  constexpr int kEntries = 32;
  static MapCacheEntry cache[kEntries];
  static int used = 0, next = 0;
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i) {
      const MapCacheEntry& e = cache[i];
      if (e.base == base && e.inner == inner_bytes && e.rows == rows && e.box == box_rows) {
        *m = e.map;
        return true;
      }
    }
  }
  if (!encode_map(m, base, inner_bytes, rows, box_rows)) return false;
  std::lock_guard<std::mutex> lock(mu);
  MapCacheEntry& e = cache[next];
  e.base = base;
  e.inner = inner_bytes;
  e.rows = rows;
  e.box = box_rows;
  e.map = *m;
  next = (next + 1) % kEntries;
  if (used < kEntries) ++used;
  return true;
}

// A scale-factor buffer as a [bytes / 256, 256] uint8 matrix, boxes of box_rows x 256
// bytes, no swizzle, rows past the end read as zero: a CTA pair loads a stage's scale
// atoms with tensor copies (their completion can be counted on the leader's barrier).
static bool encode_sf_map(CUtensorMap* m, const void* base, uint64_t bytes, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {256, bytes / 256};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {256, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_sf_map(CUtensorMap* m, const void* base, uint64_t bytes, uint32_t box_rows) {
  constexpr int kEntries = 16;
  static MapCacheEntry cache[kEntries];
  static int used = 0, next = 0;
  static std::mutex mu;
  {
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i) {
      const MapCacheEntry& e = cache[i];
      if (e.base == base && e.inner == 256 && e.rows == bytes / 256 && e.box == box_rows) {
        *m = e.map;
        return true;
      }
    }
  }
  if (!encode_sf_map(m, base, bytes, box_rows)) return false;
  std::lock_guard<std::mutex> lock(mu);
  MapCacheEntry& e = cache[next];
  e.base = base;
  e.inner = 256;
  e.rows = bytes / 256;
  e.box = box_rows;
  e.map = *m;
  next = (next + 1) % kEntries;
  if (used < kEntries) ++used;
  return true;
}

// `groups` is the number of experts of a grouped problem, 0 for a plain GEMM.
Plan make_plan(int64_t M, int64_t N, int64_t K, int groups, int mx, bool row_major_out) {
  Plan pl{};
  pl.num_kb = static_cast<int>((K + 255) / 256);
  (void)mx;
  if (groups) {
    // 256-wide tiles: per MMA the scale-factor copies into TMEM cost less than with
    // 128-wide ones (an expert's last N-tile may be half empty; its extra columns, read
    // from the next expert's rows, are never stored)
    pl.swap = false;
    pl.BN = N >= 256 ? 256 : 128;
    pl.ACC = pl.BN == 256 ? 1 : 2;
    // 256 x 256 tiles on CTA pairs load a third fewer bytes per MMA, but an expert's last
    // row tile is on average half empty: 128 rows of padding per expert instead of 64.
    // With experts of a few hundred rows (top-k routing of a few thousand tokens) the
    // padding costs more than the pairs save (measured on 32 experts of ~512 rows:
    // 128-row tiles 5% faster per clock); pairs from 1280 rows per expert on average.
    pl.pair = pl.BN == 256 && M >= 1280 * static_cast<int64_t>(groups);
    pl.mode = kModeGrouped;
    pl.Mk = M;
    pl.Nk = N;
    pl.tiles_n = static_cast<int>((N + pl.BN - 1) / pl.BN);
    pl.ws_bytes = 0;
    return pl;
  }
  if (M <= 64 && !row_major_out) {  // decode: weight rows fill MMA-M, the few activation rows are MMA-N
    pl.swap = true;
    pl.Mk = N;
    pl.Nk = M;
    pl.BN = M <= 16 ? 16 : M <= 32 ? 32 : 64;
    pl.ACC = 2;
  } else {
    pl.swap = false;
    pl.Mk = M;
    pl.Nk = N;
    // 256-wide tiles when there are enough of them to fill the SMs, else 128-wide
    const int64_t tiles256 = ((M + 127) / 128) * ((N + 255) / 256);
    pl.BN = (N >= 256 && tiles256 >= num_sms()) ? 256 : 128;
    pl.ACC = pl.BN == 256 ? 1 : 2;
  }
  pl.tiles_m = static_cast<int>((pl.Mk + 127) / 128);
  pl.tiles_n = static_cast<int>((pl.Nk + pl.BN - 1) / pl.BN);
  const int64_t tiles = static_cast<int64_t>(pl.tiles_m) * pl.tiles_n;
  const int sms = num_sms();
  // Too few tiles to fill the SMs: split every tile's K range across CTAs (stream-K).
  // Swapped (decode-like) shapes split whenever tiles are scarce; the others only when
  // K is long enough that the split's partial-sum traffic stays small against the MMAs.
  if (tiles < 2 * sms && pl.num_kb >= 4 && (pl.swap || (2 * tiles < sms && pl.num_kb >= 16))) {
    pl.mode = kModeStreamK;
    pl.units = tiles * pl.num_kb;
    pl.ws_bytes = (static_cast<size_t>(M * N) * 4 + 255) / 256 * 256 + (static_cast<size_t>(tiles) * 4 + 255) / 256 * 256;
  } else {
    pl.mode = kModeTile;
    pl.units = tiles;
    pl.ws_bytes = 0;
    // 256-wide tiles with at least two 128-row blocks: CTA pairs share 256 x 256 tiles,
    // so that each SM loads a third fewer operand bytes per MMA
    if (pl.BN == 256 && !pl.swap && M >= 256) {
      pl.pair = true;
      pl.tiles_m = static_cast<int>((pl.Mk + 255) / 256);
      pl.units = static_cast<int64_t>(pl.tiles_m) * pl.tiles_n;
    }
  }
  return pl;
}

size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int mx, bool fp4_out) {
  if (!mx && !fp4_out && decode_eligible(M, N, K)) return decode_workspace_bytes(M, N);
  return make_plan(M, N, K, 0, mx, fp4_out).ws_bytes;
}

size_t gemm_workspace_align(int64_t M, int64_t N, int64_t K, int mx, bool fp4_out) {
  int64_t row = M;  // floats per row of partial sums
  if (mx || fp4_out || !decode_eligible(M, N, K)) {
    const Plan pl = make_plan(M, N, K, 0, mx, fp4_out);
    if (pl.mode != kModeStreamK) return 1;
    row = pl.Nk;
  }
  return row % 4 == 0 ? 16 : 4;
}

// Whether the long epilogue's operands stay in place: for outputs by rows, and for the few rows of
// NVFP4 that have a K too long for the decode kernel (its small-N kernels are for MXFP4).
static bool full_in_place(int64_t M, int mx, bool fp4_out) { return fp4_out || (!mx && M <= 32); }

// The long epilogue keeps its partial sums in rows of whole float4s.
static size_t full_ws_bytes(const Plan& pl, int64_t M) {
  if (pl.mode != kModeStreamK || pl.swap) return pl.ws_bytes;
  return pl.ws_bytes + static_cast<size_t>(M) * 3 * 4 + 256;  // at most three floats more per row
}

size_t gemm_full_workspace_bytes(int64_t M, int64_t N, int64_t K, int mx, bool fp4_out) {
  if (!mx && !fp4_out && decode_eligible(M, N, K)) return decode_workspace_bytes(M, N);
  return full_ws_bytes(make_plan(M, N, K, 0, mx, full_in_place(M, mx, fp4_out)), M);
}

// the quantize workspace (tensor amax), then the GEMM's
size_t gemm_bf16a_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return (kQuantWorkspaceBytes + 255) / 256 * 256 + gemm_workspace_bytes(M, N, K, 0);
}

template <bool MX>
static cudaError_t dispatch(const Plan& pl, const GemmMaps& tm, const GemmArgs& a, cudaStream_t st) {
  // one CTA per SM at most; a CTA holds pipes_per_cta<BN>() pipelines
  switch (pl.BN) {
    case 16: return run<16, MX, 2, false>(tm, a, pl.units, st);
    case 32: return run<32, MX, 2, false>(tm, a, pl.units, st);
    case 64: return run<64, MX, 2, false>(tm, a, pl.units, st);
    case 128: return run<128, MX, 2, false>(tm, a, pl.units, st);
    default:
      return pl.pair ? run<256, MX, 1, true>(tm, a, pl.units, st) : run<256, MX, 1, false>(tm, a, pl.units, st);
  }
}

int launch_gemm(const GemmProblem& g0, unsigned* status, cudaStream_t st, const char** why, cudaError_t* err) {
  return launch_gemm_full(GemmProblemFull{g0, nullptr}, status, st, why, err);
}

int launch_gemm_full(const GemmProblemFull& g, unsigned* status, cudaStream_t st, const char** why, cudaError_t* err) {
  const int grouped = g.num_groups > 0;
  if (!grouped && !g.mx && !g.q_codes && !g.amax_out && decode_eligible(g.M, g.N, g.K)) {
    // a few activation rows: the decode kernel (the weights are problem B)
    DecodeProblem q{};
    q.W = g.B;
    q.sW = g.sB;
    q.gW = g.gB;
    q.Xq = g.A;
    q.Xs = g.sA;
    q.gX = g.gA;
    q.M = g.M;
    q.N = g.N;
    q.K = g.K;
    q.D = g.D;
    q.out_bf16 = g.out_bf16;
    q.ws = g.ws;
    q.ws_bytes = g.ws_bytes;
    q.weights_ready = g.weights_ready;
    q.bias = g.bias;
    q.act = g.act;
    if (g.full) {
      DecodeExtra x{};
      x.res = g.full->res;
      x.res_bf16 = g.full->res_bf16;
      x.pre = g.full->pre;
      return launch_decode_extra(q, x, status, st, why, err);
    }
    return launch_decode(q, status, st, why, err);
  }
  // the NVFP4 copy of the result is written by rows: keep the operands in place
  const bool by_rows = g.q_codes != nullptr || g.amax_out != nullptr;
  const Plan pl = make_plan(g.M, g.N, g.K, g.num_groups, g.mx, g.full ? full_in_place(g.M, g.mx, by_rows) : by_rows);
  const size_t need = g.full ? full_ws_bytes(pl, g.M) : pl.ws_bytes;
  if (g.ws_bytes < need || (need && !g.ws)) {
    *why = "workspace too small (see fp4_gemm_workspace_size)";
    return 1;
  }
  const int64_t sf_cols = g.K / (g.mx ? 32 : 16);
  const int64_t atoms_k = (sf_cols + 3) / 4;
  const uint8_t *kA = g.A, *kB = g.B, *kSA = g.sA, *kSB = g.sB;
  const float *kgA = g.gA, *kgB = g.gB;
  int64_t rowsA = g.M, rowsB = grouped ? static_cast<int64_t>(g.num_groups) * g.N : g.N;
  if (pl.swap) {
    std::swap(kA, kB);
    std::swap(kSA, kSB);
    std::swap(kgA, kgB);
    std::swap(rowsA, rowsB);
  }
  GemmMaps tm;
  if (!make_tensor_map_u8(&tm.a, kA, static_cast<uint64_t>(g.K / 2), static_cast<uint64_t>(rowsA), 128) ||
      !make_tensor_map_u8(&tm.b, kB, static_cast<uint64_t>(g.K / 2), static_cast<uint64_t>(rowsB),
                          static_cast<uint32_t>(pl.pair ? pl.BN / 2 : pl.BN))) {
    *why = "cuTensorMapEncodeTiled failed (alignment or driver)";
    return 1;
  }
  tm.sfa = tm.sfb = tm.a;  // unused unless CTA pairs load the scale factors with tensor copies
  tm.b2 = tm.sfb2 = tm.a;  // unused: the gated products' second operand
  if (pl.pair) {
    // one box = one stage's atoms of one 128-row block (4 atoms NVFP4, 2 MXFP4)
    const uint32_t box_rows = (g.mx ? 2u : 4u) * 512u / 256u;
    // grouped A scales: the capacity fp4_scales_bytes_grouped gives (every 128-row block
    // of every group plus one pad block per group), which the caller's buffer holds
    const int64_t sfa_blocks = (rowsA + 127) / 128 + (grouped ? g.num_groups : 0);
    if (!make_sf_map(&tm.sfa, kSA, static_cast<uint64_t>(sfa_blocks) * atoms_k * 512, box_rows) ||
        !make_sf_map(&tm.sfb, kSB, static_cast<uint64_t>((rowsB + 127) / 128) * atoms_k * 512, box_rows)) {
      *why = "cuTensorMapEncodeTiled failed for the scale factors (alignment or driver)";
      return 1;
    }
  }
  GemmArgs a{};
  a.sfa = kSA;
  a.sfb = kSB;
  a.sfa_rb_bytes = atoms_k * 512;
  a.sfb_rb_bytes = atoms_k * 512;
  a.sf_atoms_k = static_cast<int>(atoms_k);
  a.ga = kgA;
  a.gb = kgB;
  a.Mk = static_cast<int>(pl.Mk);
  a.Nk = static_cast<int>(pl.Nk);
  a.K = static_cast<int>(g.K);
  a.num_kb = pl.num_kb;
  a.out = g.D;
  a.out_bf16 = g.out_bf16;
  a.transposed = pl.swap ? 1 : 0;
  // the weights (problem B) are kernel A when the operands are swapped
  a.indep = g.weights_ready ? (pl.swap ? 1 : 2) : 0;
  a.ldo = g.N;
  const int esz = g.out_bf16 ? 2 : 4;
  a.vec_store = ((g.N * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(g.D) & 15) == 0) ? 1 : 0;
  a.mode = pl.mode;
  a.tiles_m = pl.tiles_m;
  a.tiles_n = pl.tiles_n;
  a.group_m = 16;
  a.total_units = pl.units;
  a.status = status;
  a.bias = g.bias;
  a.act = g.act;
  a.q_codes = g.q_codes;
  a.q_scales = g.q_scales;
  a.q_g = g.q_g;
  a.q_atoms = (g.N / 16 + 3) / 4;
  a.amax_out = reinterpret_cast<unsigned*>(g.amax_out);
  if (pl.mode == kModeStreamK) {
    a.ws = static_cast<float*>(g.ws);
    a.ws_ld = static_cast<int>(g.full && !pl.swap ? (g.N + 3) / 4 * 4 : g.N);
    a.tile_cnt = reinterpret_cast<int*>(static_cast<uint8_t*>(g.ws) + (static_cast<size_t>(g.M * a.ws_ld) * 4 + 255) / 256 * 256);
  }
  if (grouped) {
    a.num_groups = g.num_groups;
    a.offsets = g.offsets;
    a.b_rows_per_group = static_cast<int>(g.N);
    a.sfb_rbs = static_cast<int>((g.N + 127) / 128);
    a.sfb_group_bytes = static_cast<int64_t>(a.sfb_rbs) * atoms_k * 512;
  } else {
    a.sfb_rbs = static_cast<int>((rowsB + 127) / 128);
  }
  cudaError_t e;
  if (g.full) {
    a.res = g.full->res;
    a.res_bf16 = g.full->res_bf16;
    a.pre = g.full->pre;
    auto al32 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; };
    a.sectors = (g.N * esz) % 32 == 0 && al32(g.D) && al32(a.pre) &&
                (!a.res || ((g.N * (a.res_bf16 ? 2 : 4)) % 32 == 0 && al32(a.res)));
    a.bias_any = a.bias != nullptr;
    e = dispatch_full(pl, g.mx, tm, a, st);
  } else {
    e = g.mx ? dispatch<true>(pl, tm, a, st) : dispatch<false>(pl, tm, a, st);
  }
  if (e != cudaSuccess) {
    *err = e;
    return 2;
  }
  return 0;
}

// FP4 x FP8 ("Rubin FP4 GEMM overview" 3.4: an FP4 operand opposite an FP8 one): A and
// B each MXFP4 or MXFP8, D = A B^T on kind::mxf8f6f4 MMAs.  Dense, whole tiles on single
// CTAs; K a multiple of 128.
int launch_gemm_mixed(const GemmProblem& g, int a_fp8, int b_fp8, unsigned* status, cudaStream_t st,
                      const char** why, cudaError_t* err) {
  const int sms = num_sms();
  const int64_t tiles256 = ((g.M + 127) / 128) * ((g.N + 255) / 256);
  const int BN = (g.N >= 256 && tiles256 >= sms) ? 256 : 128;
  // 256-wide tiles with at least two 128-row blocks run on CTA pairs, as the FP4 GEMM's do
  const bool pair = BN == 256 && g.M >= 256;
  GemmMaps tm;
  const bool ok_a = a_fp8 ? make_tensor_map_u8(&tm.a, g.A, static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.M), 128)
                          : encode_map_u4(&tm.a, g.A, static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.M), 128);
  const bool ok_b = b_fp8 ? make_tensor_map_u8(&tm.b, g.B, static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.N),
                                               static_cast<uint32_t>(pair ? BN / 2 : BN))
                          : encode_map_u4(&tm.b, g.B, static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.N),
                                          static_cast<uint32_t>(pair ? BN / 2 : BN));
  if (!ok_a || !ok_b) {
    *why = "cuTensorMapEncodeTiled failed (alignment or driver)";
    return 1;
  }
  const int64_t atoms_k = g.K / 128;  // one E8M0 per 32 K elements, four per atom row
  tm.sfa = tm.sfb = tm.b2 = tm.sfb2 = tm.a;
  // a pair loads a stage's scale atoms (one per 128-row block: 512 bytes, two 256-byte rows)
  // with tensor copies that complete on the leader's barrier
  if (pair && (!make_sf_map(&tm.sfa, g.sA, static_cast<uint64_t>((g.M + 127) / 128) * atoms_k * 512, 2) ||
               !make_sf_map(&tm.sfb, g.sB, static_cast<uint64_t>((g.N + 127) / 128) * atoms_k * 512, 2))) {
    *why = "cuTensorMapEncodeTiled failed for the scale factors (alignment or driver)";
    return 1;
  }
  GemmArgs a{};
  a.sfa = g.sA;
  a.sfb = g.sB;
  a.sfa_rb_bytes = atoms_k * 512;
  a.sfb_rb_bytes = atoms_k * 512;
  a.sf_atoms_k = static_cast<int>(atoms_k);
  a.sfb_rbs = static_cast<int>((g.N + 127) / 128);
  a.Mk = static_cast<int>(g.M);
  a.Nk = static_cast<int>(g.N);
  a.K = static_cast<int>(g.K);
  a.num_kb = static_cast<int>(g.K / 128);
  a.out = g.D;
  a.out_bf16 = g.out_bf16;
  a.ldo = g.N;
  const int esz = g.out_bf16 ? 2 : 4;
  a.vec_store = ((g.N * esz) % 16 == 0 && (reinterpret_cast<uintptr_t>(g.D) & 15) == 0) ? 1 : 0;
  a.mode = kModeTile;
  a.tiles_m = static_cast<int>((g.M + (pair ? 255 : 127)) / (pair ? 256 : 128));
  a.tiles_n = static_cast<int>((g.N + BN - 1) / BN);
  a.group_m = 16;
  a.total_units = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
  a.status = status;
  a.f8_fmt = (a_fp8 ? kFmtE4M3 : kFmtE2M1) | ((b_fp8 ? kFmtE4M3 : kFmtE2M1) << 3);
  const cudaError_t e = pair        ? run<256, true, 1, true, true>(tm, a, a.total_units, st)
                        : BN == 256 ? run<256, true, 1, false, true>(tm, a, a.total_units, st)
                                    : run<128, true, 2, false, true>(tm, a, a.total_units, st);
  if (e != cudaSuccess) {
    *err = e;
    return 2;
  }
  return 0;
}

}  // namespace fp4
