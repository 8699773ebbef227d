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
//               of BN (pair: BN / 2) tokens, both with the 128-byte swizzle, into a ring of stages
//   warp 1      owns TMEM; one lane issues four K = 32 MMAs a stage
//   warps 2..   epilogue, four warps (tiles up to 64 tokens) or eight (two per TMEM lane quarter,
//               one per half of the columns); two accumulators, so that it overlaps the next tile
//
// Schedules: whole tiles, strided over the grid; or a split, where the K steps of all tiles form one
// sequence that is cut evenly over the grid.  A tile cut in pieces has its partial sums added up
// in the workspace, in the slot of the CTA that starts it; the CTA whose piece completes the K
// steps takes them from there, clears slot and counter, and finishes the tile.  No CTA waits for
// another one.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp4_act.cuh"
#include "fp4_moe.h"
#include "fp4_ptx.cuh"

namespace fp4 {
namespace {

struct I8Args {
  const float *sx, *sw, *bias;
  int act;
  int M, N, K, num_kb;
  void* out;
  int out_bf16;
  int early_w;         // weights may be read before the preceding kernel finishes
  int split;
  int tiles_w, tiles_t;  // tiles along the channels, along the tokens (dense)
  int num_groups;
  const int32_t* offsets;
  int* cnt;            // split: K steps summed so far in each slot, zero between calls
  int* sums;           // split: [grid][BN][128] partial sums, zero between calls
  unsigned* status;
};

struct I8Work {
  int w_row, x_row;    // first rows of the tile's boxes (of this CTA's)
  int n0, n_valid;     // this CTA's channels
  int t0, t_valid;     // the tile's tokens
  int group;
  int kb0, kb1;
  int slot;            // split: the CTA that starts the tile
};

template <int BN, bool PAIR>
struct I8Cfg {
  static constexpr int kEpiWarps = BN >= 128 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kWBytes = 128 * 128;
  static constexpr int kXRows = PAIR ? BN / 2 : BN;
  static constexpr int kXBytes = kXRows * 128;
  static constexpr int kStageBytes = kWBytes + kXBytes;
  static constexpr int kScaleOff = 1024;                        // barriers and flags before it
  static constexpr int kGroupOff = kScaleOff + 2 * BN * 4;      // two tiles' token scales
  static constexpr int kMiscBytes = kGroupOff + 2 * (kMaxGroups + 1) * 4;
  static constexpr int kFit = (227 * 1024 - 1024 - 256 - kMiscBytes) / kStageBytes;
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static constexpr int kSmemBytes = kStages * kStageBytes + kMiscBytes + 1024;
  static constexpr int kTmemCols = 2 * BN;  // 32 .. 512, a power of two
  static constexpr int kChunk = BN * 4 / kEpiWarps;  // accumulator columns of an epilogue thread
  static_assert(BN == 16 || BN == 32 || BN == 64 || BN == 128 || BN == 256, "tile width");
  static_assert(!PAIR || BN == 256, "pairs run 256 x 256 tiles");
  static_assert(kStageBytes % 1024 == 0, "the 128-byte swizzle's alignment");
  static_assert(kStages >= 3 && kSmemBytes + 256 <= 227 * 1024, "shared memory");
  static_assert((2 * kStages + 5) * 8 + 16 <= kScaleOff, "barriers");
};

template <int BN, bool PAIR>
struct I8Sched {
  static constexpr int kRows = PAIR ? 256 : 128;
  const I8Args& p;
  const int *s_off, *s_tiles;  // by experts: row offsets, prefix of token tiles
  int vb, vg, sub_row;
  int64_t u, end, tiles, units;

  __device__ I8Sched(const I8Args& a, const int* off, const int* tl, int vb_, int vg_, int sub)
      : p(a), s_off(off), s_tiles(tl), vb(vb_), vg(vg_), sub_row(sub) {
    tiles = static_cast<int64_t>(p.tiles_w) * (p.num_groups ? s_tiles[p.num_groups] : p.tiles_t);
    units = tiles * p.num_kb;
    u = p.split ? units * vb / vg : vb;
    end = p.split ? units * (vb + 1) / vg : tiles;
  }

  __device__ bool next(I8Work& w) {
    if (u >= end) return false;
    int64_t tile = u;
    w.kb0 = 0;
    w.kb1 = p.num_kb;
    w.slot = 0;
    if (p.split) {
      tile = u / p.num_kb;
      w.kb0 = static_cast<int>(u - tile * p.num_kb);
      w.kb1 = static_cast<int>(min(static_cast<int64_t>(p.num_kb), w.kb0 + (end - u)));
      // the CTA c whose units [units c / vg, units (c + 1) / vg) hold the tile's first one
      w.slot = static_cast<int>(((tile * p.num_kb + 1) * vg - 1) / units);
      u += w.kb1 - w.kb0;
    } else {
      u += vg;
    }
    int wt, tt, row0, row_end;
    if (p.num_groups) {
      int lo = 0, hi = p.num_groups - 1;  // the last expert whose tiles start at or before this one
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<int64_t>(s_tiles[mid]) * p.tiles_w <= tile) lo = mid;
        else hi = mid - 1;
      }
      const int mine = s_tiles[lo + 1] - s_tiles[lo];
      const int64_t local = tile - static_cast<int64_t>(s_tiles[lo]) * p.tiles_w;
      wt = static_cast<int>(local / mine);
      tt = static_cast<int>(local % mine);
      w.group = lo;
      row0 = s_off[lo];
      row_end = s_off[lo + 1];
    } else {
      // groups of eight token tiles, so that tiles that run at once share boxes in L2
      constexpr int kBand = 8;
      const int64_t band = static_cast<int64_t>(kBand) * p.tiles_w;
      const int first = static_cast<int>(tile / band) * kBand;
      const int size = min(kBand, p.tiles_t - first);
      const int r = static_cast<int>(tile % band);
      wt = r / size;
      tt = first + r % size;
      w.group = 0;
      row0 = 0;
      row_end = p.M;
    }
    w.n0 = wt * kRows + sub_row;
    w.n_valid = max(0, min(128, p.N - w.n0));
    w.w_row = w.group * p.N + w.n0;
    w.t0 = row0 + tt * BN;
    w.t_valid = min(BN, row_end - w.t0);
    w.x_row = w.t0 + (PAIR ? sub_row : 0);
    return true;
  }
};

__device__ __forceinline__ void i8_timeout(volatile int* abort, unsigned* status) {
  *abort = 1;
  atomicOr(status, kStatusTimeout);
}

template <int BN, bool PAIR>
__global__ void __launch_bounds__(I8Cfg<BN, PAIR>::kThreads, 1)
    fp4_i8_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const I8Args p) {
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
  volatile int* s_last = s_abort + 2;
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
    *s_last = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
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
      // weights that one band of tokens reads once need not stay in L2
      const uint64_t pol_w = p.tiles_t == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
      const uint64_t pol_x = l2_policy_evict_last();
      auto load = [&](int stage, const I8Work& w, int kb, bool weights) {
        uint8_t* st = smem + stage * C::kStageBytes;
        if constexpr (PAIR) {
          const uint32_t bar = cluster_addr(smem_u32(&full[stage]), 0);
          if (weights) tma_load_2d_pair(st, &tmW, bar, kb * 128, w.w_row, pol_w);
          else tma_load_2d_pair(st + C::kWBytes, &tmX, bar, kb * 128, w.x_row, pol_x);
        } else {
          if (weights) tma_load_2d(st, &tmW, &full[stage], kb * 128, w.w_row, pol_w);
          else tma_load_2d(st + C::kWBytes, &tmX, &full[stage], kb * 128, w.x_row, pol_x);
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
          if (leader) mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * C::kStageBytes);
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
      constexpr uint32_t idesc_rows = PAIR ? 256 : 128;
      const uint32_t idesc = mma_idesc_i8(BN, idesc_rows);
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
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&full[stage], phase, s_abort)) {
            i8_timeout(s_abort, p.status);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem) + stage * C::kStageBytes;
          const uint64_t adesc = smem_desc_sw128(st), bdesc = smem_desc_sw128(st + C::kWBytes);
          const int nk = min(4, (p.K - kb * 128 + 31) / 32);
          for (int k = 0; k < nk; ++k) {
            const uint32_t accum = kb > w.kb0 || k > 0 ? 1u : 0u;
            if constexpr (PAIR) tc_mma_i8_pair(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, accum);
            else tc_mma_i8(d_tmem, adesc + 2 * k, bdesc + 2 * k, idesc, accum);
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
    I8Work w;
    int iter = 0;
    while (sch.next(w)) {
      const int acc = iter & 1;
      float* xs = s_scale + acc * BN;
      for (int c = et; c < BN; c += 32 * C::kEpiWarps) xs[c] = c < w.t_valid ? __ldg(p.sx + w.t0 + c) : 0.0f;
      const bool ch_ok = rl < w.n_valid;
      float sw = 0.0f, b = 0.0f;
      if (ch_ok) {
        const int64_t ch = static_cast<int64_t>(w.group) * p.N + w.n0 + rl;
        sw = __ldg(p.sw + ch);
        if (p.bias) b = __ldg(p.bias + ch);
      }
      // the warps decide together whether to go on, so that none is left at a barrier
      if (et == 0 && !mbar_wait(&acc_full[acc], (iter >> 1) & 1, s_abort)) {
        i8_timeout(s_abort, p.status);
        *s_fail = 1;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kEpiWarps) : "memory");
      if (*s_fail) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * BN;
      // 16 tokens of this thread's channel
      auto finish = [&](int c, const uint32_t (&r)[16]) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(r[j])), xs[c + j]), sw);
        if (p.bias) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __fadd_rn(v[j], b);
        }
        with_act(p.act, [&](auto tag) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = act_value<decltype(tag)::value>(v[j]);
        });
        if (!ch_ok) return;
        const int64_t at = static_cast<int64_t>(w.t0 + c) * p.N + w.n0 + rl;
        if (p.out_bf16) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < w.t_valid) o[static_cast<int64_t>(j) * p.N] = __float2bfloat16_rn(v[j]);
        } else {
          float* o = static_cast<float*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < w.t_valid) o[static_cast<int64_t>(j) * p.N] = v[j];
        }
      };
      const bool piece = w.kb1 - w.kb0 < p.num_kb;
      int* slot = p.sums + static_cast<int64_t>(w.slot) * (BN * 128) + rl;
#pragma unroll 1
      for (int c = c0; c < c0 + C::kChunk; c += 16) {
        if (c >= w.t_valid) break;  // the same for all lanes
        uint32_t r[16];
        tmem_ld16(taddr + c, r);
        tmem_ld_wait();
        if (!PAIR && piece) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (ch_ok && c + j < w.t_valid) atomicAdd(slot + (c + j) * 128, static_cast<int>(r[j]));
        } else {
          finish(c, r);
        }
        __syncwarp();  // the next TMEM load takes the whole warp
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[acc]), 0));
        else mbar_arrive(&acc_empty[acc]);
      }
      ++iter;
      if (PAIR || !piece) continue;
      // this piece's sums are out; the one that completes the tile's K steps finishes it
      __threadfence();
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kEpiWarps) : "memory");
      if (et == 0) {
        __threadfence();
        const int before = atomicAdd(p.cnt + w.slot, w.kb1 - w.kb0);
        *s_last = before + (w.kb1 - w.kb0) == p.num_kb;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(32 * C::kEpiWarps) : "memory");
      if (!*s_last) continue;
      __threadfence();
      if (et == 0) p.cnt[w.slot] = 0;
#pragma unroll 1
      for (int c = c0; c < c0 + C::kChunk && c < w.t_valid; c += 16) {
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          r[j] = 0;
          if (ch_ok && c + j < w.t_valid) {
            r[j] = static_cast<uint32_t>(__ldcg(slot + (c + j) * 128));
            __stcg(slot + (c + j) * 128, 0);
          }
        }
        finish(c, r);
      }
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
  int num_kb;
  int grid;                  // CTAs or pairs; split: slots
};

I8Plan i8_plan(int64_t M, int64_t N, int64_t K, int groups) {
  I8Plan pl{};
  const int sms = num_sms();
  const int64_t used = groups ? std::min<int64_t>(groups, M) : 1;  // experts with rows, at most
  const int64_t rows = (M + used - 1) / used;                      // tokens that share their weights
  pl.num_kb = static_cast<int>((K + 127) / 128);
  auto tiles_t = [&](int bn) { return used * ((rows + bn - 1) / bn); };
  pl.BN = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  if (rows > 128 && N > 128 && (N + 255) / 256 * tiles_t(256) >= sms / 4) {
    pl.BN = 256;
    pl.pair = true;
  }
  pl.tiles_w = (N + (pl.pair ? 255 : 127)) / (pl.pair ? 256 : 128);
  pl.tiles_t = tiles_t(pl.BN);
  const int64_t tiles = pl.tiles_w * pl.tiles_t;
  pl.split = !pl.pair && pl.num_kb > 1 && (pl.BN <= 64 || tiles < 2 * sms);
  pl.grid = pl.pair ? sms / 2 : sms;
  if (!groups) pl.grid = static_cast<int>(std::min<int64_t>(pl.grid, pl.split ? tiles * pl.num_kb : tiles));
  return pl;
}

constexpr size_t kCountBytes = 4096;  // the slots' counters, before their sums

size_t plan_workspace(const I8Plan& pl) {
  return pl.split ? kCountBytes + static_cast<size_t>(pl.grid) * pl.BN * 128 * 4 : 0;
}

template <int BN, bool PAIR>
cudaError_t run_i8(const CUtensorMap& w, const CUtensorMap& x, const I8Args& a, int grid, cudaStream_t st) {
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
  const int64_t rows_w = g.N * std::max(1, g.num_groups);
  CUtensorMap w, x;
  if (!make_tensor_map_u8(&w, g.B, static_cast<uint64_t>(g.K), static_cast<uint64_t>(rows_w), 128) ||
      !make_tensor_map_u8(&x, g.A, static_cast<uint64_t>(g.K), static_cast<uint64_t>(g.M),
                          static_cast<uint32_t>(pl.pair ? pl.BN / 2 : pl.BN))) {
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
  a.early_w = g.weights_ready && !g.num_groups;
  a.split = pl.split;
  a.tiles_w = static_cast<int>(pl.tiles_w);
  a.tiles_t = static_cast<int>(pl.tiles_t);
  a.num_groups = g.num_groups;
  a.offsets = g.offsets;
  if (pl.split) {
    a.cnt = static_cast<int*>(g.ws);
    a.sums = reinterpret_cast<int*>(static_cast<uint8_t*>(g.ws) + kCountBytes);
  }
  a.status = status;
  switch (pl.pair ? 256 : pl.BN) {
    case 16: *err = run_i8<16, false>(w, x, a, pl.grid, st); break;
    case 32: *err = run_i8<32, false>(w, x, a, pl.grid, st); break;
    case 64: *err = run_i8<64, false>(w, x, a, pl.grid, st); break;
    case 128: *err = run_i8<128, false>(w, x, a, pl.grid, st); break;
    default: *err = run_i8<256, true>(w, x, a, pl.grid, st); break;
  }
  return *err == cudaSuccess ? 0 : 2;
}

}  // namespace fp4
