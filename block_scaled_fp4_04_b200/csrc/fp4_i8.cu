// fp4_i8.cu -- matrix product in 8-bit integers with a scale for each token and each channel:
//   D[m, n] = act(sA[m] sB[n] sum_k A[m, k] B[n, k] + bias[n])
// dense, or by experts (rows [offsets[e], offsets[e + 1]) of A with weights number e).
//
// The sums are 32-bit integers on the tensor cores (tcgen05.mma.kind::i8): exact, so that partial
// sums can meet in any order and the result has the same bits every time.
//
// One orientation for all sizes: the weights' rows fill the MMA's 128 rows (256 over a pair of
// CTAs), the tokens are its BN columns.  A lane of the epilogue then owns one channel (scale and
// bias in registers), neighbouring lanes write neighbouring outputs of a token, and the tile's
// width follows the number of tokens: 16 for a decode step, so that almost all of the shared
// memory's ring is weights in flight.
//
// Structure, one CTA (or one CTA of a pair) per SM, persistent:
//   warp 0      loads, by TMA: per K step of 128 bytes one 128 x 128-byte box of weights and one box
//               of tokens, both with the 128-byte swizzle, into a ring of stages of one K step
//               (pairs: two)
//   warp 1      owns TMEM; one lane issues four K = 32 MMAs a K step
//   warps 2..   epilogue, four warps (one per TMEM lane quarter), or eight from 64 tokens on, which
//               share out the columns; two accumulators, so that it overlaps the next tile
// Wider tiles are shared by a pair of CTAs: 256 channels x up to 256 tokens, each CTA loading
// its 128 channels and half of the tokens.  Its width is the tokens that share weights (one
// expert's, or all) in equal parts, rounded up to 64: 530 rows are 3 x 192, not 2 x 256 and a rest.
//
// Schedules: pairs take whole tiles, strided over the grid.  Single CTAs split: the K steps of all
// tiles form one sequence that is cut evenly over the grid.  A CTA then leaves the sums of a tile that
// it has only a piece of in the workspace (one slot for a tile that it ends, one for a tile that
// it starts); the one whose piece completes the tile's K steps adds up the others' slots, clears
// them, and finishes the tile.  No CTA waits for another one.
//
// Measured: 8192 x 8192 x 8192 334 us in short bursts, 3.29e15 operations a second (the MMA loop alone
// reaches 4.2 to 4.5e15, 128 cycles per 128 x 256 x 32), 385 to 400 us under the power cap at 1.3 GHz, where
// the loop's own limit is 345; the tensor pipe is 90% busy at 4096 x 8192 x 8192.  16 x 28672 x 8192 streams its
// weights at 5.1e12 bytes a second.  A pair's K step of 256 channels x 256 tokens moves as many bytes into
// shared memory as the MMAs read from it, together what its bandwidth allows: narrower tiles are
// bound by it, and the epilogue stays out of shared memory.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp4_act.cuh"
#include "fp4_i8.cuh"
#include "fp4_moe.h"

namespace fp4 {
namespace {

struct I8Args {
  const float *sx, *sw, *bias;
  int act;
  int M, N, K, num_kb;
  void* out;
  int out_bf16;
  int wide;            // BF16 outputs of an even width
  int early_w;         // weights may be read before the preceding kernel finishes
  // A weight's tokens fit one tile (by experts: on average, whatever the offsets say): it need not stay in
  // L2.  Asking each tile on the device instead made no difference for even experts, nor for 64 rows of one
  // of 64 experts of 5760 x 2880, and 100 rows of one of 100 experts of 28672 x 8192 took 254 us for 248
  // (medians of 62 bursts in turn, 248-270 and 225-264).
  int weights_once;
  int split;
  int tiles_w, tiles_t;  // tiles along the channels, along the tokens (dense)
  int num_groups;
  const int32_t* offsets;
  int* cnt;            // split: K steps done of the tile that each CTA starts, per warp; zero between calls
  int4* sums;          // split: two slots per CTA of BN x 128 sums, zero between calls
  unsigned* status;
};

struct I8Work {
  int w_row, x_row;    // first rows of the tile's boxes (of this CTA's)
  int n0, n_valid;     // this CTA's channels
  int t0, t_valid;     // the tile's tokens
  int width;           // its MMA columns
  int group;
  int kb0, kb1;
  int first, last;     // split: the CTAs that hold its first and last K step
};

template <int BN, bool PAIR>
struct I8Cfg {
  static constexpr int kEpiWarps = BN >= 64 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kSteps = PAIR ? 2 : 1;  // K steps of 128 bytes a stage
  static constexpr int kWBytes = 128 * 128;
  static constexpr int kXBytes = (PAIR ? BN / 2 : BN) * 128;
  static constexpr int kStageBytes = kSteps * (kWBytes + kXBytes);
  static constexpr int kScaleOff = 1024;                        // barriers and flags before it
  static constexpr int kGroupOff = kScaleOff + 2 * BN * 4;      // two tiles' token scales
  static constexpr int kMiscBytes = kGroupOff + 2 * (kMaxGroups + 1) * 4;
  static constexpr int kFit = (227 * 1024 - 1024 - 256 - kMiscBytes) / kStageBytes;
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static constexpr int kSmemBytes = kStages * kStageBytes + kMiscBytes + 1024;
  static constexpr int kTmemCols = 2 * BN;  // 32 .. 512, a power of two
  static constexpr int kChunk = BN * 4 / kEpiWarps;  // accumulator columns of an epilogue thread
  static constexpr int kLoad = PAIR ? 32 : 16;  // that it takes at once
  static_assert(32 * kEpiWarps >= BN, "a token scale per epilogue thread");
  static_assert(PAIR ? BN == 256 : BN == 16 || BN == 32 || BN == 64, "tile width");
  static_assert(kXBytes % 1024 == 0 && kStageBytes % 1024 == 0, "the 128-byte swizzle's alignment");
  static_assert(kStages >= 3 && kSmemBytes + 256 <= 227 * 1024, "shared memory");
  static_assert((2 * kStages + 5) * 8 + 16 <= kScaleOff, "barriers");
};

// A pair's tile width: the rows that share weights in `tiles` equal parts, rounded up to 64.  (Unsigned: the
// sum passes 2^31 below the largest number of rows.)
__host__ __device__ __forceinline__ int pair_width(uint32_t rows, uint32_t tiles) {
  return static_cast<int>((rows + tiles - 1) / tiles + 63) / 64 * 64;
}

// Token rows of a pair's boxes: half of a tile's width of 64, 128, 192 or 256.
struct I8TokenMaps {
  CUtensorMap box[4];
};

template <int BN, bool PAIR>
struct I8Sched {
  static constexpr int kRows = PAIR ? 256 : 128;
  const I8Args& p;
  const int *s_off, *s_tiles;  // by experts: row offsets, prefix of token tiles
  int vb, vg, sub_row;
  uint32_t u, end, units;  // (32 bits: divisions are taken for every tile, and the host sees to it that they do)

  __device__ I8Sched(const I8Args& a, const int* off, const int* tl, int vb_, int vg_, int sub)
      : p(a), s_off(off), s_tiles(tl), vb(vb_), vg(vg_), sub_row(sub) {
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_w) * (p.num_groups ? s_tiles[p.num_groups] : p.tiles_t);
    units = tiles * p.num_kb;
    u = p.split ? units * vb / vg : vb;
    end = p.split ? units * (vb + 1) / vg : tiles;
  }

  __device__ bool next(I8Work& w) {
    if (u >= end) return false;
    uint32_t tile = u;
    w.kb0 = 0;
    w.kb1 = p.num_kb;
    if (p.split) {
      tile = u / p.num_kb;
      w.kb0 = static_cast<int>(u - tile * p.num_kb);
      w.kb1 = static_cast<int>(min(static_cast<uint32_t>(p.num_kb), w.kb0 + (end - u)));
      // the CTA c whose units [units c / vg, units (c + 1) / vg) hold unit x is ((x + 1) vg - 1) / units
      w.first = static_cast<int>(((tile * p.num_kb + 1) * vg - 1) / units);
      w.last = static_cast<int>(((tile + 1) * p.num_kb * vg - 1) / units);
      u += w.kb1 - w.kb0;
    } else {
      u += vg;
    }
    int wt, tt, tts, row0, row_end;
    if (p.num_groups) {
      int lo = 0, hi = p.num_groups - 1;  // the last expert whose tiles start at or before this one
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<uint32_t>(s_tiles[mid]) * p.tiles_w <= tile) lo = mid;
        else hi = mid - 1;
      }
      tts = s_tiles[lo + 1] - s_tiles[lo];
      const uint32_t local = tile - static_cast<uint32_t>(s_tiles[lo]) * p.tiles_w;
      wt = static_cast<int>(local / tts);
      tt = static_cast<int>(local - wt * tts);
      w.group = lo;
      row0 = s_off[lo];
      row_end = s_off[lo + 1];
    } else {
      // groups of sixteen token tiles, so that tiles that run at once share boxes in L2
      constexpr uint32_t kBand = 16;
      const uint32_t band = tile / (kBand * p.tiles_w), first = band * kBand;
      const uint32_t size = min(kBand, p.tiles_t - first), r = tile - first * p.tiles_w;
      wt = static_cast<int>(r / size);
      tt = static_cast<int>(first + r - wt * size);
      tts = p.tiles_t;
      w.group = 0;
      row0 = 0;
      row_end = p.M;
    }
    w.n0 = wt * kRows + sub_row;
    w.n_valid = max(0, min(128, p.N - w.n0));
    w.w_row = w.group * p.N + w.n0;
    w.width = PAIR ? pair_width(row_end - row0, tts) : BN;
    w.t0 = row0 + tt * w.width;
    w.t_valid = min(w.width, row_end - w.t0);
    w.x_row = w.t0 + (sub_row ? w.width / 2 : 0);
    return true;
  }
};

// Stores 16 tokens of a warp's 32 channels: v[i] holds tokens `token` + 2i and + 2i + 1 (of which
// `tokens` exist) of channel `ch` + lane (of which `chs` exist).  FP32 rows are whole lines as they
// are.  BF16 ones of an even width leave in words of two channels: neighbouring lanes exchange
// halves, so that even lanes hold even tokens.  (Meeting in shared memory for 16-byte words costs
// bandwidth that the MMAs and their loads need: experts 32 x 16384 x 5760 x 2880 300 us under the power
// cap, so 295; 8192 x 8192 x 256 73.5 and 66.9.)
__device__ __forceinline__ void store_tokens16(const I8Args& p, int64_t token, int tokens, int ch, int chs, int lane,
                                               const float2 (&v)[8]) {
  const bool on = lane < chs;
  if (!p.out_bf16) {
    float* out = static_cast<float*>(p.out) + token * p.N + ch + lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (on && 2 * i < tokens) __stcs(out, v[i].x);
      if (on && 2 * i + 1 < tokens) __stcs(out + p.N, v[i].y);
      out += 2 * static_cast<int64_t>(p.N);
    }
    return;
  }
  const int odd = p.wide ? lane & 1 : 0;
  uint16_t* out = static_cast<uint16_t*>(p.out) + (token + odd) * p.N + ch + (p.wide ? lane & ~1 : lane);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
    const uint32_t w = *reinterpret_cast<const uint32_t*>(&h);
    if (p.wide) {
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
      const uint32_t two = __byte_perm(w, got, odd ? 0x3276 : 0x5410);
      if (on && 2 * i + odd < tokens) __stcs(reinterpret_cast<uint32_t*>(out), two);
    } else {
      if (on && 2 * i < tokens) out[0] = static_cast<uint16_t>(w);
      if (on && 2 * i + 1 < tokens) out[p.N] = static_cast<uint16_t>(w >> 16);
    }
    out += 2 * static_cast<int64_t>(p.N);
  }
}

__device__ __forceinline__ void i8_timeout(volatile int* abort, unsigned* status) {
  *abort = 1;
  atomicOr(status, kStatusTimeout);
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(I8Cfg<BN, PAIR>::kThreads, 1)
    fp4_i8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ I8TokenMaps tmX, const I8Args p) {
  using C = I8Cfg<BN, PAIR>;
  using Schedule = I8Sched<BN, PAIR>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* misc = smem + S * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  volatile int* s_abort = reinterpret_cast<volatile int*>(drain + 1);
  volatile int* s_fail = s_abort + 1;
  float* s_scale = reinterpret_cast<float*>(misc + C::kScaleOff);
  int* s_off = reinterpret_cast<int*>(misc + C::kGroupOff);
  int* s_tiles = s_off + kMaxGroups + 1;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const int vb = PAIR ? blockIdx.x / 2 : blockIdx.x, vg = PAIR ? gridDim.x / 2 : gridDim.x;
  const int sub_row = static_cast<int>(rank) * 128;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], (PAIR ? 2 : 1) * C::kEpiWarps);
    }
    mbar_init(drain, 1);
    *s_abort = 0;
    *s_fail = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    if constexpr (!PAIR) tma_prefetch_desc(&tmX.box[0]);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&s_tmem_base, C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&s_tmem_base, C::kTmemCols);
      tmem_relinquish();
    }
  }
  if (p.num_groups && warp == 2) {  // the prefix of token tiles over the experts
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int carry = 0;
    for (int base = 0; base < p.num_groups; base += 32) {
      const int e = base + lane;
      int n = 0;
      if (e < p.num_groups) {
        const int lo = p.offsets[e];
        s_off[e] = lo;
        n = (p.offsets[e + 1] - lo + BN - 1) / BN;
      }
      int in = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, in, d);
        if (lane >= d) in += t;
      }
      if (e < p.num_groups) s_tiles[e] = carry + in - n;
      carry += __shfl_sync(0xFFFFFFFFu, in, 31);
    }
    if (lane == 0) {
      s_tiles[p.num_groups] = carry;
      s_off[p.num_groups] = p.offsets[p.num_groups];
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ loads
      const uint64_t pol_w = p.weights_once ? l2_policy_evict_first() : l2_policy_evict_last();
      const uint64_t pol_x = l2_policy_evict_last();
      auto load = [&](int stage, const I8Work& w, int kb, bool weights) {
        uint8_t* st = smem + stage * C::kStageBytes + (weights ? 0 : C::kSteps * C::kWBytes);
#pragma unroll
        for (int h = 0; h < C::kSteps; ++h) {
          const int x = (kb * C::kSteps + h) * 128;
          if constexpr (PAIR) {
            const uint32_t bar = cluster_addr(smem_u32(&full[stage]), 0);
            if (weights) tma_load_2d_pair(st + h * C::kWBytes, &tmW, bar, x, w.w_row, pol_w);
            else tma_load_2d_pair(st + h * C::kXBytes, &tmX.box[w.width / 64 - 1], bar, x, w.x_row, pol_x);
          } else {
            if (weights) tma_load_2d(st + h * C::kWBytes, &tmW, &full[stage], x, w.w_row, pol_w);
            else tma_load_2d(st + h * C::kXBytes, &tmX.box[0], &full[stage], x, w.x_row, pol_x);
          }
        }
      };
      // with weights that are ready, the first ring-full of stages asks for them, then waits for
      // the preceding kernel, then asks for the tokens
      bool waited = !p.early_w;
      if (waited) asm volatile("griddepcontrol.wait;" ::: "memory");
      int pending = 0;
      auto tokens = [&]() {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        Schedule again(p, s_off, s_tiles, vb, vg, sub_row);
        I8Work w;
        int j = 0;
        while (j < pending && again.next(w))
          for (int kb = w.kb0; kb < w.kb1 && j < pending; ++kb, ++j) load(j, w, kb, false);
        waited = true;
      };
      Schedule sch(p, s_off, s_tiles, vb, vg, sub_row);
      I8Work w;
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      while (ok && sch.next(w)) {
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, s_abort)) {
            i8_timeout(s_abort, p.status);
            ok = false;
            break;
          }
          // a pair's leader counts the boxes of both CTAs (out-of-range rows read as zero)
          if (leader)
            mbar_arrive_expect_tx(&full[stage], PAIR ? C::kSteps * (2 * C::kWBytes + w.width * 128) : C::kStageBytes);
          load(stage, w, kb, true);
          if (waited) load(stage, w, kb, false);
          else if (++pending == S) tokens();
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!waited) tokens();
      // after a timeout: let what was asked for land before the shared memory goes away
      if (*s_abort && leader)
        for (int s = 0; s < S; ++s)
          if (issued & (1u << s)) {
            volatile int go_on = 0;
            mbar_wait(&full[s], (parity >> s) & 1u, &go_on);
          }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ MMAs
      Schedule sch(p, s_off, s_tiles, vb, vg, sub_row);
      I8Work w;
      int stage = 0, iter = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && sch.next(w)) {
        const int acc = iter & 1;
        if (!mbar_wait(&acc_empty[acc], ((iter >> 1) & 1) ^ 1, s_abort)) {
          i8_timeout(s_abort, p.status);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * BN;
        const uint32_t idesc = mma_idesc_i8(PAIR ? w.width : BN, PAIR ? 256 : 128);
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, s_abort)) {
            i8_timeout(s_abort, p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem) + stage * C::kStageBytes;
          const uint64_t adesc = smem_desc_sw128(st), bdesc = smem_desc_sw128(st + C::kSteps * C::kWBytes);
          const int left = (p.K - kb * C::kSteps * 128 + 31) / 32;  // MMAs up to the end of K
#pragma unroll
          for (int k = 0; k < 4 * C::kSteps; ++k) {
            if (k >= left) break;
            const uint64_t ad = adesc + (k / 4) * (C::kWBytes / 16) + 2 * (k % 4);
            const uint64_t bd = bdesc + (k / 4) * (C::kXBytes / 16) + 2 * (k % 4);
            const uint32_t accum = kb > w.kb0 || k > 0 ? 1u : 0u;
            if constexpr (PAIR) tc_mma_i8_pair(d_tmem, ad, bd, idesc, accum);
            else tc_mma_i8(d_tmem, ad, bd, idesc, accum);
          }
          if constexpr (PAIR) tc_commit_pair_mc(&empty[stage], 3);
          else tc_commit(&empty[stage]);
          if (++stage == S) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if constexpr (PAIR) tc_commit_pair_mc(&acc_full[acc], 3);
        else tc_commit(&acc_full[acc]);
        ++iter;
      }
      // no MMA may still write TMEM when it is freed
      if constexpr (PAIR) tc_commit_pair(drain);
      else tc_commit(drain);
      volatile int go_on = 0;
      mbar_wait(drain, 0, &go_on);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int q = warp & 3;                       // TMEM lane quarter
    const int et = threadIdx.x - 64;
    const int c0 = ((warp - 2) >> 2) * C::kChunk;  // this thread's first column
    const int rl = q * 32 + lane;                 // its channel within the tile
    Schedule sch(p, s_off, s_tiles, vb, vg, sub_row);
    I8Work w, next;
    // a tile's scales and biases are asked for one tile ahead
    float next_x = 0.0f, next_w = 0.0f, next_b = 0.0f;
    auto ahead = [&]() {
      if (!sch.next(next)) return false;
      next_x = et < next.t_valid ? __ldg(p.sx + next.t0 + et) : 0.0f;
      if (rl < next.n_valid) {
        const int64_t ch = static_cast<int64_t>(next.group) * p.N + next.n0 + rl;
        next_w = __ldg(p.sw + ch);
        if (p.bias) next_b = __ldg(p.bias + ch);
      }
      return true;
    };
    bool more = ahead();
    int iter = 0;
    while (more) {
      w = next;
      const int acc = iter & 1;
      float* xs = s_scale + acc * BN;
      if (et < BN) xs[et] = next_x;
      const float sw = next_w, b = next_b;
      more = ahead();
      // the warps decide together whether to go on, so that none is left at a barrier
      if (et == 0 && !mbar_wait(&acc_full[acc], (iter >> 1) & 1, s_abort)) {
        i8_timeout(s_abort, p.status);
        *s_fail = 1;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kEpiWarps) : "memory");
      if (*s_fail) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
      // 16 tokens of this thread's channel (all lanes take part)
      const int chs = max(0, min(32, w.n_valid - q * 32));
      auto finish = [&](int c, const uint32_t* r) __attribute__((always_inline)) {
        float2 z[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 x = *reinterpret_cast<const float4*>(xs + c + 2 * j);
          const int* a = reinterpret_cast<const int*>(r) + 2 * j;
          z[j] = __fmul2_rn(make_float2(__int2float_rn(a[0]), __int2float_rn(a[1])), make_float2(x.x, x.y));
          z[j + 1] = __fmul2_rn(make_float2(__int2float_rn(a[2]), __int2float_rn(a[3])), make_float2(x.z, x.w));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = __fmul2_rn(z[j], pair(sw));
        if (p.bias) {
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = __fadd2_rn(z[j], pair(b));
        }
        with_act(p.act, [&](auto tag) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = act_value2<decltype(tag)::value>(z[j]);
        });
        store_tokens16(p, w.t0 + c, w.t_valid - c, w.n0 + q * 32, chs, lane, z);
      };
      auto load = [&](int c, uint32_t* r) __attribute__((always_inline)) {
        if constexpr (C::kLoad == 32) tmem_ld32(taddr + c, r);
        else tmem_ld16(taddr + c, *reinterpret_cast<uint32_t(*)[16]>(r));
        tmem_ld_wait();
      };
      const int c1 = min(c0 + C::kChunk, w.t_valid);
      bool done = true;
      const bool piece = !PAIR && w.kb1 - w.kb0 < p.num_kb;
      // this thread's sums in the slot of CTA `who`: the one for the tile that it starts, or ends
      auto slot = [&](int who) { return p.sums + (2 * who + (who == w.first)) * static_cast<int64_t>(BN * 32) + rl; };
      if (piece) {
        int4* mine = slot(vb);
#pragma unroll 1
        for (int c = c0; c < c1; c += C::kLoad) {  // c1 is the same for all lanes
          int r[C::kLoad];
          load(c, reinterpret_cast<uint32_t*>(r));
#pragma unroll
          for (int j = 0; j < C::kLoad; j += 4)
            __stcg(mine + (c + j) / 4 * 128, make_int4(r[j], r[j + 1], r[j + 2], r[j + 3]));
        }
        // every warp for itself: the warps of this number in the tile's CTAs have the same sums to add
        // (with barriers over the CTA 64 x 8192 x 8192 took 28.8 us, so 21.8)
        __syncwarp();
        if (lane == 0) {
          __threadfence();
          int* cnt = p.cnt + w.first * C::kEpiWarps + warp - 2;
          const int all = atomicAdd(cnt, w.kb1 - w.kb0) + w.kb1 - w.kb0;
          done = all == p.num_kb;
          if (done) *cnt = 0;
          __threadfence();
        }
        done = __shfl_sync(0xFFFFFFFFu, done, 0);
        __syncwarp();  // lane 0's fences hold for the warp: the sums before its count, the others' after
      }
      if (done) {
#pragma unroll 1
        for (int c = c0; c < c1; c += C::kLoad) {
          uint32_t r[C::kLoad];
          load(c, r);
          if (piece) {
            constexpr int kAsk = 4, kWords = C::kLoad / 4;  // slots that are asked for at once
            for (int who = w.first; who <= w.last; who += kAsk) {
              int4 t[kAsk][kWords];
#pragma unroll
              for (int h = 0; h < kAsk; ++h) {
                const int4* from = slot(who + h) + c / 4 * 128;
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                  t[h][j] = who + h <= w.last && who + h != vb ? __ldcg(from + j * 128) : make_int4(0, 0, 0, 0);
              }
#pragma unroll
              for (int h = 0; h < kAsk; ++h) {
                if (who + h > w.last) break;
                int4* from = slot(who + h) + c / 4 * 128;
#pragma unroll
                for (int j = 0; j < kWords; ++j) {
                  r[4 * j] += t[h][j].x;
                  r[4 * j + 1] += t[h][j].y;
                  r[4 * j + 2] += t[h][j].z;
                  r[4 * j + 3] += t[h][j].w;
                  __stcg(from + j * 128, make_int4(0, 0, 0, 0));
                }
              }
            }
          }
          finish(c, r);
          if constexpr (C::kLoad == 32) {
            if (c + 16 < w.t_valid) finish(c + 16, r + 16);
          }
          __syncwarp();  // the next TMEM load takes the whole warp
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[acc]), 0));
        else mbar_arrive(&acc_empty[acc]);
      }
      ++iter;
    }
  }

  tc_fence_before();
  __syncthreads();
  // a pair: neither CTA leaves while its shared memory or TMEM is still used by the other
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    if constexpr (PAIR) tmem_dealloc_pair(s_tmem_base, C::kTmemCols);
    else tmem_dealloc(s_tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------- host side
struct I8Plan {
  int BN;
  bool pair, split;
  int64_t tiles_w, tiles_t;  // (by experts: an estimate of the token tiles, the offsets are on the device)
  int64_t rows;              // tokens that share their weights
  int64_t units;             // K steps of all tiles, at most
  int num_kb;
  int grid;                  // CTAs or pairs
};

I8Plan i8_plan(int64_t M, int64_t N, int64_t K, int groups) {
  I8Plan pl{};
  const int sms = num_sms(), pairs = sms / 2;
  const int64_t used = groups ? std::min<int64_t>(groups, M) : 1;  // experts with rows, at most
  pl.rows = (M + used - 1) / used;
  if (groups) {
    // Experts' rows fall unevenly: a tile that is wide enough for twice the average and more costs
    // little, a second tile of an expert reads its weights again.  (32 experts of 5760 x 2880, tiles of
    // 16 / 64 / pairs: 32 rows in all 59 / 69 / 57 us, 512 rows 113 / 87 / 92, 2048 rows 354 / 112 / 93.)
    pl.pair = pl.rows > 32;
    pl.BN = pl.pair ? 256 : pl.rows > 1 ? 64 : 16;
  } else {
    // Above 16 tokens a pair's whole tiles beat the pieces' sum where they are few and short.
    // (64 x 5760 x 2880: pairs 11.9 us, split 14.8; 64 x 4096 x 4096 13.4 and 15.3; 64 x 8192 x 8192
    // 22.5 and 21.3; 64 x 1024 x 8192 25.8 and 18.2; 16 x 4096 x 4096 12.3 and 10.4.)
    pl.pair = pl.rows > 64 || (pl.rows > 16 && K <= 4096 && (N + 255) / 256 <= pairs);
    pl.BN = pl.pair ? 256 : pl.rows <= 16 ? 16 : pl.rows <= 32 ? 32 : 64;
  }
  const int step = pl.pair ? 256 : 128;
  pl.num_kb = static_cast<int>((K + step - 1) / step);
  pl.tiles_w = (N + step - 1) / step;
  int width = pl.BN;
  if (pl.pair && !groups) {
    // A K step of a pair moves 256 + width rows into and out of shared memory, which takes longer
    // than its MMAs up to a width of 256 (measured: as 320 + width), and all pairs wait for the last
    // round of tiles: the width with the shortest rounds in all.  (256 x 4096 x 4096: widths
    // 64 / 128 / 256 take 15.1 / 16.6 / 18.5 us, 1024 x 8192 x 8192 115 / 73 / 50.)
    int64_t best = INT64_MAX;
    for (int w = 64; w <= 256; w += 64) {
      const int64_t tiles = pl.tiles_w * ((M + w - 1) / w), cost = (tiles + pairs - 1) / pairs * (320 + w);
      if (cost <= best) {
        best = cost;
        width = w;
      }
    }
  }
  pl.tiles_t = used * ((pl.rows + width - 1) / width);
  const int64_t tiles = pl.tiles_w * pl.tiles_t;
  // (units times CTAs fit 32 bits; so many units have enough tiles without a split.  Experts' rows that
  // fall unevenly make at most one more tile each.)
  pl.units = (tiles + (groups ? groups * pl.tiles_w : 0)) * pl.num_kb;
  pl.split = !pl.pair && pl.num_kb > 1 && pl.units < (1ll << 32) / (sms + 1);
  pl.grid = pl.pair ? pairs : sms;
  if (pl.split) {
    // A tile's pieces are added up by one CTA, so that with many of them their sum takes longer
    // than their K steps: about the square root of the K steps is the best number.
    int64_t pieces = 2;
    while ((pieces + 1) * (pieces + 1) <= pl.num_kb) ++pieces;
    pl.grid = static_cast<int>(std::min<int64_t>(pl.grid, tiles * std::min<int64_t>(pieces, pl.num_kb)));
  } else if (!groups) {
    pl.grid = static_cast<int>(std::min<int64_t>(pl.grid, tiles));
  }
  return pl;
}

constexpr int64_t kStepMargin = 1024;   // a CTA's step past the last tile
constexpr size_t kCountBytes = 16384;   // counters of each CTA's epilogue warps, before the slots

size_t plan_workspace(const I8Plan& pl) {
  return pl.split ? kCountBytes + static_cast<size_t>(pl.grid) * 2 * pl.BN * 128 * 4 : 0;
}

template <int BN, bool PAIR>
cudaError_t run_i8(const CUtensorMap& w, const I8TokenMaps& x, const I8Args& a, int grid, cudaStream_t st) {
  using C = I8Cfg<BN, PAIR>;
  auto kern = fp4_i8_kernel<BN, PAIR>;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t e = cudaSuccess;
  if (dev < 0 || dev >= 64 || !attr_done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (PAIR) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    static int max_pairs[64] = {0};  // pairs that can be resident at once, asked once per device
    int pairs = dev >= 0 && dev < 64 ? max_pairs[dev] : 0;
    if (pairs <= 0) {
      cfg.gridDim = dim3(2 * static_cast<unsigned>(num_sms() / 2));
      e = cudaOccupancyMaxActiveClusters(&pairs, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (pairs <= 0) return cudaErrorInvalidConfiguration;
      if (dev >= 0 && dev < 64) max_pairs[dev] = pairs;
    }
    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min(grid, pairs)));
  } else {
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
  }
  return cudaLaunchKernelEx(&cfg, kern, w, x, a);
}

}  // namespace

size_t i8_workspace_bytes(int64_t M, int64_t N, int64_t K, int num_groups) {
  if (M <= 0 || N <= 0 || K <= 0 || num_groups < 0) return 0;
  return plan_workspace(i8_plan(M, N, K, num_groups));
}

int launch_gemm_i8(const I8Problem& g, unsigned* status, cudaStream_t st, const char** why, cudaError_t* err) {
  const I8Plan pl = i8_plan(g.M, g.N, g.K, g.num_groups);
  const size_t need = plan_workspace(pl);
  if (need && (!g.ws || g.ws_bytes < need || (reinterpret_cast<uintptr_t>(g.ws) & 15))) {
    *why = "workspace too small or misaligned (see fp4_gemm_i8_workspace_size)";
    return 1;
  }
  if (pl.units / pl.num_kb + kStepMargin > (1ll << 31)) {
    *why = "too many tiles";
    return 1;
  }
  const int64_t rows_w = g.N * std::max(1, g.num_groups);
  const int width = pair_width(static_cast<uint32_t>(g.M), static_cast<uint32_t>(pl.tiles_t));
  CUtensorMap w;
  I8TokenMaps x{};
  bool ok = make_tensor_map_u8(&w, g.B, static_cast<uint64_t>(g.K), static_cast<uint64_t>(rows_w), 128);
  for (int i = 0; ok && i < 4; ++i) {
    // dense pairs have one width, experts' may have any
    if (pl.pair ? !g.num_groups && width != 64 * (i + 1) : i > 0) continue;
    ok = make_tensor_map_u8(&x.box[i], g.A, static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.M),
                            static_cast<uint32_t>(pl.pair ? 32 * (i + 1) : pl.BN));
  }
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed (alignment or driver)";
    return 1;
  }
  I8Args a{};
  a.sx = g.sA;
  a.sw = g.sB;
  a.bias = g.bias;
  a.act = g.act;
  a.M = static_cast<int>(g.M);
  a.N = static_cast<int>(g.N);
  a.K = static_cast<int>(g.K);
  a.num_kb = pl.num_kb;
  a.out = g.D;
  a.out_bf16 = g.out_bf16;
  a.wide = g.N % 2 == 0;
  a.early_w = g.weights_ready && !g.num_groups;
  a.weights_once = g.num_groups ? pl.rows <= pl.BN : pl.tiles_t == 1;
  a.split = pl.split;
  a.tiles_w = static_cast<int>(pl.tiles_w);
  a.tiles_t = static_cast<int>(pl.tiles_t);
  a.num_groups = g.num_groups;
  a.offsets = g.offsets;
  if (pl.split) {
    a.cnt = static_cast<int*>(g.ws);
    a.sums = reinterpret_cast<int4*>(static_cast<uint8_t*>(g.ws) + kCountBytes);
  }
  a.status = status;
  switch (pl.BN) {
    case 16: *err = run_i8<16, false>(w, x, a, pl.grid, st); break;
    case 32: *err = run_i8<32, false>(w, x, a, pl.grid, st); break;
    case 64: *err = run_i8<64, false>(w, x, a, pl.grid, st); break;
    default: *err = run_i8<256, true>(w, x, a, pl.grid, st); break;
  }
  return *err == cudaSuccess ? 0 : 2;
}

}  // namespace fp4
