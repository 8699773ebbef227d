// fp4_norm.cu -- layer norm over the columns of a row-major [rows, cols] tensor, forward and
// backward, and the column sums that end a weight gradient.  Memory-bound: every row is read
// once and kept in registers between the reductions.
//
//   forward   mean = sum x / n, var = sum (x - mean)^2 / n (two passes over the registers: no
//             difference of large squares), rstd = 1 / sqrt(var + eps),
//             y = (x - mean) rstd w + b
//   backward  xh = (x - mean) rstd, a = dy w,
//             dx = rstd (a - mean(a) - xh mean(a xh)) + dres, dw = sum_r dy xh, db = sum_r dy
//
// All sums are FP32.  Sums over a row go through a fixed tree, sums over rows through a fixed
// split of the rows into partial sums that a second kernel adds in order: no atomics, the
// same bits every time.
#include "fp4_ops.h"
#include "fp4_rows.cuh"

namespace fp4 {

struct LnArgs {
  const void* x;
  int64_t rows;
  int n;
  const float *w, *b;
  float eps;
  void* y;
  int y_bf16;
  float *mean, *rstd;
  RowCodes q;
  unsigned* amax;
  unsigned* status;
};

// Sum over the WPR warps of one row; every thread of the row gets it.  Rows of one warp need
// no shared memory; others meet on the named barrier `bar`.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* s, int wr, int lane, int bar) {
  v = warp_sum(v);
  if constexpr (WPR > 1) {
    if (lane == 0) s[wr] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(WPR * 32) : "memory");
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += s[i];
  }
  return v;
}

// WPR warps per row, C chunks of V elements per thread held in registers; C = 0: rows of any
// length, read again for every pass.
template <typename T, int V, int WPR, int C, int FMT>
__global__ void __launch_bounds__((WPR < 4 ? 4 : WPR) * 32) ln_forward_kernel(const LnArgs p) {
  constexpr int kWarps = WPR < 4 ? 4 : WPR;
  constexpr int kRows = kWarps / WPR;  // rows per CTA
  constexpr int kCh = C > 0 ? C : 1;
  __shared__ float s_red[2][kRows][WPR];
  rows_wait_prior();
  rows_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / WPR, wr = warp % WPR, bar = 1 + group;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group;
  const bool row_ok = row < p.rows;
  const T* x = static_cast<const T*>(p.x) + (row_ok ? row : 0) * p.n;
  const int first = (wr * 32 + lane) * V;      // this thread's first element
  constexpr int kStep = WPR * 32 * V;
  const int loops = C > 0 ? C : (p.n + kStep - 1) / kStep;

  RowVec<T, V> raw[kCh];
  auto load = [&](int j, RowVec<T, V>& r) {
    const int col = first + j * kStep;
    if (row_ok && col < p.n) r.load(x + col);
    else r.zero();
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int j = 0; j < C; ++j) load(j, raw[j]);
  }
  // f(chunk, values, whether they exist)
  auto each = [&](auto&& f) {
    if constexpr (C > 0) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float v[V];
        raw[j].unpack(v);
        f(first + j * kStep, v, row_ok && first + j * kStep < p.n);
      }
    } else {
      for (int j = 0; j < loops; ++j) {
        float v[V];
        load(j, raw[0]);
        raw[0].unpack(v);
        f(first + j * kStep, v, row_ok && first + j * kStep < p.n);
      }
    }
  };
  const float inv_n = 1.0f / static_cast<float>(p.n);
  float s = 0.0f;
  each([&](int, const float (&v)[V], bool) {
#pragma unroll
    for (int i = 0; i < V; ++i) s += v[i];  // missing elements are zero
  });
  const float mean = row_sum<WPR>(s, s_red[0][group], wr, lane, bar) * inv_n;
  float ss = 0.0f;
  each([&](int, const float (&v)[V], bool ok) {
    if (ok) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = v[i] - mean;
        ss += d * d;
      }
    }
  });
  const float var = row_sum<WPR>(ss, s_red[1][group], wr, lane, bar) * inv_n;
  const float rstd = 1.0f / sqrtf(var + p.eps);
  if (row_ok && wr == 0 && lane == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  float g = 1.0f;
  if constexpr (FMT == kCodesNv) g = *p.q.g;
  uint32_t m = 0;
  bool bad = false;
  each([&](int col, const float (&v)[V], bool ok) {
    float o[V];
    if (ok) {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = (v[i] - mean) * rstd;
      if (p.w) {
        float w[V];
        load_params<V>(p.w + col, w);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] *= w[i];
      }
      if (p.b) {
        float b[V];
        load_params<V>(p.b + col, b);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] += b[i];
      }
      if (p.y) store_row_vec<V>(p.y, p.y_bf16, row * p.n + col, o);
      if (p.amax) {
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, abs_bits_of(o[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = 0.0f;
    }
    if constexpr (FMT != kCodesNone) bad |= encode_row_vec<FMT, V>(p.q, g, row, col, ok, o);
  });
  if (p.amax) {
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0 && m) atomicMax(p.amax, m);
  }
  if (FMT != kCodesNone && bad) atomicOr(p.status, kStatusNonFinite);
}

// ------------------------------------------------------------------ rows through a ring
// With many rows: one CTA per SM whose groups of WPR warps walk over rows of their own.  Each
// group has a ring of row slots in shared memory that bulk copies fill several rows ahead, so
// that the loads in flight do not depend on how far its arithmetic is, and a thread keeps the
// parameters of its columns in registers from row to row.  A group's first thread refills a
// slot after the row sum's barrier, by when every thread has read the slot.
constexpr int kRingWarps = 16;
constexpr int kRingSlots = 8;                       // at most, per group
constexpr size_t kRingBytes = 200 * 1024;           // shared memory for the slots of a CTA
constexpr int kRingHeader = 1024;                   // barriers, row sums

struct RingPlan {
  int slots;      // per group
  size_t smem;
  int grid;
};
static RingPlan ring_plan(int groups, size_t slot_bytes, int64_t rows) {
  RingPlan r{};
  r.slots = static_cast<int>(std::min<size_t>(kRingSlots, kRingBytes / (groups * slot_bytes)));
  r.smem = kRingHeader + static_cast<size_t>(r.slots) * groups * slot_bytes;
  r.grid = static_cast<int>(std::min<int64_t>(num_sms(), (rows + groups - 1) / groups));
  return r;
}

struct Ring {
  uint64_t* full;          // [slots] of this group
  uint8_t* slot0;          // this group's slots
  uint32_t slot_bytes;
  int slots;
  volatile int* abort;
  unsigned* status;
  int at;                  // slot of the current row
  uint32_t phase;
  // Waits for the current row.  After a timeout (latched) the group goes on with what is there,
  // so that its barriers still match; the outputs are then unspecified.
  __device__ __forceinline__ void wait() {
    if (!mbar_wait(&full[at], phase, abort) && !*abort) {
      *abort = 1;
      atomicOr(status, kStatusTimeout);
    }
  }
  __device__ __forceinline__ const uint8_t* row() const { return slot0 + static_cast<size_t>(at) * slot_bytes; }
  __device__ __forceinline__ void next() {
    if (++at == slots) {
      at = 0;
      phase ^= 1;
    }
  }
};

template <typename T, int V>
__device__ __forceinline__ void ring_read(RowVec<T, V>& r, const uint8_t* row, int col) {
  const uint4 t = *reinterpret_cast<const uint4*>(row + static_cast<size_t>(col) * sizeof(T));
  r.w[0] = t.x;
  r.w[1] = t.y;
  r.w[2] = t.z;
  r.w[3] = t.w;
}

// R rows at a time per group (a slot holds R consecutive rows): their chains of shuffles and
// their one barrier overlap.  One barrier gives mean and variance: each warp takes the mean m_w
// and the sum of squares about it of its own n_w columns, and the row's sum of squares is
// sum_w M2_w + n_w (m_w - mean)^2 -- no difference of large squares.
// A vector's elements as FP32 pairs: the paired FP32 instructions do two at once.
template <typename T, int V>
__device__ __forceinline__ void unpack2(const RowVec<T, V>& r, float2 (&v)[V / 2]) {
  float t[V];
  r.unpack(t);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) v[i] = make_float2(t[2 * i], t[2 * i + 1]);
}

template <typename T, int V, int W, int WPR, int C, int R, int FMT>
__global__ void __launch_bounds__(W * 32, 1) ln_forward_ring_kernel(const LnArgs p, int slots) {
  constexpr int G = W / WPR;
  constexpr int kStep = WPR * 32 * V;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ float2 s_stat[2][G][WPR][R];
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / WPR, wr = warp % WPR, bar = 1 + group;
  const int first = (wr * 32 + lane) * V;
  const uint32_t row_bytes = static_cast<uint32_t>(p.n) * sizeof(T);
  Ring ring{reinterpret_cast<uint64_t*>(s_ring) + group * kRingSlots,
            s_ring + kRingHeader + static_cast<size_t>(group) * slots * R * row_bytes, R * row_bytes, slots, &s_abort, p.status,
            0, 0};
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < G * kRingSlots; ++i) mbar_init(reinterpret_cast<uint64_t*>(s_ring) + i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  rows_wait_prior();
  rows_allow_dependents();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * G * R;
  int64_t row = (static_cast<int64_t>(blockIdx.x) * G + group) * R;
  const bool loader = wr == 0 && lane == 0;
  const uint64_t pol = l2_policy_evict_first();
  auto load_rows = [&](int slot, int64_t r) {
    const uint32_t bytes = static_cast<uint32_t>(min(static_cast<int64_t>(R), p.rows - r)) * row_bytes;
    mbar_arrive_expect_tx(&ring.full[slot], bytes);
    bulk_load(ring.slot0 + static_cast<size_t>(slot) * R * row_bytes, static_cast<const T*>(p.x) + r * p.n, bytes,
              &ring.full[slot], pol);
  };
  if (loader)
    for (int i = 0; i < slots && row + i * stride < p.rows; ++i) load_rows(i, row + i * stride);
  float2 w[C][V / 2], b[C][V / 2];
  int n_w = 0;  // columns of this warp
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int col = first + j * kStep;
    float tw[V], tb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      tw[i] = 1.0f;
      tb[i] = 0.0f;
    }
    if (col < p.n) {
      if (p.w) load_params<V>(p.w + col, tw);
      if (p.b) load_params<V>(p.b + col, tb);
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      w[j][i] = make_float2(tw[2 * i], tw[2 * i + 1]);
      b[j][i] = make_float2(tb[2 * i], tb[2 * i + 1]);
    }
    n_w += max(0, min(32 * V, p.n - (wr * 32 * V + j * kStep)));
  }
  const float inv_n = 1.0f / static_cast<float>(p.n);
  const float inv_nw = n_w ? 1.0f / static_cast<float>(n_w) : 0.0f;
  // columns of warp lane % WPR of the group, for combining the warps' statistics
  constexpr int kEntries = WPR * R, kSets = kEntries > 32 ? kEntries / 32 : 1;
  float lane_n = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j)
    lane_n += static_cast<float>(max(0, min(32 * V, p.n - ((lane % WPR) * 32 * V + j * kStep))));
  const float lane_inv = lane_n > 0.0f ? 1.0f / lane_n : 0.0f;
  float g = 1.0f;
  if constexpr (FMT == kCodesNv) g = *p.q.g;
  uint32_t m = 0;
  bool bad = false;
  for (int par = 0; row < p.rows; row += stride, par ^= 1) {
    ring.wait();
    RowVec<T, V> raw[R][C];
    float s[R], q[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 a[2] = {};
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int col = first + j * kStep;
        // (rows past the last one: what the slot held before; never stored)
        if (col < p.n) ring_read<T, V>(raw[r][j], ring.row() + static_cast<size_t>(r) * row_bytes, col);
        else raw[r][j].zero();
        float2 v[V / 2];
        unpack2(raw[r][j], v);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) a[i & 1] = __fadd2_rn(a[i & 1], v[i]);
      }
      s[r] = (a[0].x + a[0].y) + (a[1].x + a[1].y);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], d);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float mw = s[r] * inv_nw;
      const float2 neg = make_float2(-mw, -mw);
      float2 a[2] = {};
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (first + j * kStep < p.n) {
          float2 v[V / 2];
          unpack2(raw[r][j], v);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const float2 e = __fadd2_rn(v[i], neg);
            a[i & 1] = __ffma2_rn(e, e, a[i & 1]);
          }
        }
      q[r] = (a[0].x + a[0].y) + (a[1].x + a[1].y);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) q[r] += __shfl_xor_sync(0xFFFFFFFFu, q[r], d);
    if (lane == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) s_stat[par][group][wr][r] = make_float2(s[r], q[r]);
    }
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(WPR * 32) : "memory");
    if (loader && row + slots * stride < p.rows) load_rows(ring.at, row + slots * stride);
    ring.next();
    // lane e (and e + 32, ...) holds what warp e % WPR found for row e / WPR
    float mean[R], rstd[R];
#pragma unroll
    for (int k = 0; k < kSets; ++k) {
      const int e = (lane + 32 * k) % kEntries;
      const float2 t = s_stat[par][group][e % WPR][e / WPR];
      float sum = t.x;
#pragma unroll
      for (int d = 1; d < WPR; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
      const float mu = sum * inv_n;
      const float dev = fmaf(t.x, lane_inv, -mu);
      float sq = fmaf(dev * dev, lane_n, t.y);
#pragma unroll
      for (int d = 1; d < WPR; d <<= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, d);
      const float rs = 1.0f / sqrtf(sq * inv_n + p.eps);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r * WPR / 32 == k) {
          mean[r] = __shfl_sync(0xFFFFFFFFu, mu, r * WPR % 32);
          rstd[r] = __shfl_sync(0xFFFFFFFFu, rs, r * WPR % 32);
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool row_ok = row + r < p.rows;
      if (loader && row_ok) {
        if (p.mean) p.mean[row + r] = mean[r];
        if (p.rstd) p.rstd[row + r] = rstd[r];
      }
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int col = first + j * kStep;
        const bool ok = row_ok && col < p.n;
        float2 v[V / 2];
        float o[V];
        unpack2(raw[r][j], v);
        const float2 neg = make_float2(-mean[r], -mean[r]), rs = make_float2(rstd[r], rstd[r]);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const float2 y = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[i], neg), rs), w[j][i], b[j][i]);
          o[2 * i] = ok ? y.x : 0.0f;
          o[2 * i + 1] = ok ? y.y : 0.0f;
        }
        if (ok) {
          if (p.y) store_row_vec<V>(p.y, p.y_bf16, (row + r) * p.n + col, o);
          if (p.amax) {
#pragma unroll
            for (int i = 0; i < V; ++i) m = max(m, abs_bits_of(o[i]));
          }
        }
        if constexpr (FMT != kCodesNone) bad |= encode_row_vec<FMT, V>(p.q, g, row + r, col, ok, o);
      }
    }
  }
  if (p.amax) {
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0 && m) atomicMax(p.amax, m);
  }
  if (FMT != kCodesNone && bad) atomicOr(p.status, kStatusNonFinite);
  if (s_abort && loader) {  // copies still in flight land before the shared memory goes away
    volatile int no_abort = 0;
    for (int i = 0; i < slots; ++i) mbar_wait(&ring.full[i], ring.phase ^ (i < ring.at ? 1u : 0u), &no_abort);
  }
}

template <typename K>
static cudaError_t ring_attr(K kern, bool (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(kRingHeader + kRingBytes));
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

template <typename T, int V, int W, int WPR, int C, int R, int FMT>
static cudaError_t run_ln_ring(const LnArgs& a, cudaStream_t st) {
  constexpr int G = W / WPR;
  static bool done[64] = {false};
  const cudaError_t e = ring_attr(ln_forward_ring_kernel<T, V, W, WPR, C, R, FMT>, done);
  if (e != cudaSuccess) return e;
  const RingPlan r = ring_plan(G, static_cast<size_t>(a.n) * sizeof(T) * R, (a.rows + R - 1) / R);
  return launch_rows(ln_forward_ring_kernel<T, V, W, WPR, C, R, FMT>, dim3(static_cast<unsigned>(r.grid)), W * 32,
                     r.smem, st, a, r.slots);
}

// Rows and lengths the ring serves: BF16 rows that fill their groups' lanes, several steps for
// every group in the grid.  Measured against a CTA per row (us): 8192 x 8192 BF16 48.8 / 60.8,
// 16384 x 4096 48.9 / 56.4, 16384 x 2880 36.8 / 43.2, 32768 x 1024 27.9 / 28.1, 2400 x 4096
// 10.7 / 11.4, but 1200 x 4096 6.4 / 6.1.  FP32 has half the arithmetic per byte and does not
// need it: 4096 x 8192 49.7 / 43.6, 8192 x 2880 35.0 / 32.4.
template <typename T, int V, int FMT>
static bool pick_ln_ring(const LnArgs& a, cudaStream_t st, cudaError_t* e) {
  if constexpr (V != 8) {
    return false;
  } else {
    const int nch = (a.n + V - 1) / V;
    if (a.rows < 16 * static_cast<int64_t>(num_sms()) || nch < 96 || nch > 2048) return false;
    if (nch <= 128) *e = run_ln_ring<T, V, 16, 2, 2, 2, FMT>(a, st);
    else if (nch <= 192) *e = run_ln_ring<T, V, 16, 2, 3, 2, FMT>(a, st);
    else if (nch <= 256) *e = run_ln_ring<T, V, 16, 4, 2, 2, FMT>(a, st);
    else if (nch <= 384) *e = run_ln_ring<T, V, 16, 4, 3, 2, FMT>(a, st);
    else if (nch <= 512) *e = run_ln_ring<T, V, 16, 8, 2, 2, FMT>(a, st);
    else if (nch <= 768) *e = run_ln_ring<T, V, 16, 8, 3, 2, FMT>(a, st);
    else if (nch <= 1024) *e = run_ln_ring<T, V, 16, 16, 2, 2, FMT>(a, st);
    else if (nch <= 1536) *e = run_ln_ring<T, V, 16, 16, 3, 2, FMT>(a, st);
    else *e = run_ln_ring<T, V, 16, 16, 4, 1, FMT>(a, st);
    return true;
  }
}

template <typename T, int V, int WPR, int C, int FMT>
static cudaError_t run_ln(const LnArgs& a, cudaStream_t st) {
  constexpr int kWarps = WPR < 4 ? 4 : WPR, kRows = kWarps / WPR;
  return launch_rows(ln_forward_kernel<T, V, WPR, C, FMT>, dim3(static_cast<unsigned>((a.rows + kRows - 1) / kRows)),
                     kWarps * 32, 0, st, a);
}

// Warps per row by the row's length, so that a thread holds at most four chunks.
template <typename T, int V, int FMT>
static cudaError_t pick_ln(const LnArgs& a, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  if (pick_ln_ring<T, V, FMT>(a, st, &e)) return e;
  const int nch = (a.n + V - 1) / V;
  if (nch <= 32) return run_ln<T, V, 1, 1, FMT>(a, st);
  // Single elements and pairs: sixteen elements a thread, for fewer warps per row (4096 x 2881
  // BF16: 31.7 us, 45.6 with four on 16 warps).
  if constexpr (V < 4) {
    constexpr int C = 16 / V;
    if (nch <= 128) return run_ln<T, V, 1, 4, FMT>(a, st);
    if (nch <= 32 * C) return run_ln<T, V, 1, C, FMT>(a, st);
    if (nch <= 128 * C) return run_ln<T, V, 4, C, FMT>(a, st);
    if (nch <= 256 * C) return run_ln<T, V, 8, C, FMT>(a, st);
    if (nch <= 512 * C) return run_ln<T, V, 16, C, FMT>(a, st);
    return run_ln<T, V, 16, 0, FMT>(a, st);
  }
  if (nch <= 64) return run_ln<T, V, 1, 2, FMT>(a, st);
  if (nch <= 128) return run_ln<T, V, 1, 4, FMT>(a, st);
  if (nch <= 512) return run_ln<T, V, 4, 4, FMT>(a, st);
  if (nch <= 1024) return run_ln<T, V, 8, 4, FMT>(a, st);
  if (nch <= 2048) return run_ln<T, V, 16, 4, FMT>(a, st);
  return run_ln<T, V, 16, 0, FMT>(a, st);
}

static bool aligned16_rows(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
// rows of pairs: even lengths (the matrices themselves are 16-byte aligned), parameters at 8 bytes
static bool pairs_ok(int n, const void* w, const void* b) {
  return n % 2 == 0 && ((reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(b)) & 7) == 0;
}

template <typename T>
static cudaError_t pick_ln_vec(const LayerNormProblem& p, const LnArgs& a, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  // whole 16-byte words of x and of the parameters; y rows are then aligned too
  const bool vec = a.n % V == 0 && aligned16_rows(a.x) && aligned16_rows(a.y) && aligned16_rows(a.w) && aligned16_rows(a.b);
  if (p.q.fmt == kCodesNv) return vec ? pick_ln<T, V, kCodesNv>(a, st) : cudaErrorInvalidValue;
  if (p.q.fmt == kCodesMx) return vec ? pick_ln<T, V, kCodesMx>(a, st) : cudaErrorInvalidValue;
  if (vec) return pick_ln<T, V, kCodesNone>(a, st);
  return pairs_ok(a.n, a.w, a.b) ? pick_ln<T, 2, kCodesNone>(a, st) : pick_ln<T, 1, kCodesNone>(a, st);
}

cudaError_t launch_layernorm(const LayerNormProblem& p, unsigned* status, cudaStream_t st) {
  LnArgs a{};
  a.x = p.x;
  a.rows = p.rows;
  a.n = static_cast<int>(p.cols);
  a.w = p.weight;
  a.b = p.bias;
  a.eps = p.eps;
  a.y = p.y;
  a.y_bf16 = p.y_bf16;
  a.mean = p.mean;
  a.rstd = p.rstd;
  a.q = RowCodes{p.q.codes, p.q.scales, p.q.g, p.cols, (p.cols / (p.q.fmt == kCodesMx ? 32 : 16) + 3) / 4};
  a.amax = reinterpret_cast<unsigned*>(p.amax_out);
  a.status = status;
  return p.bf16 ? pick_ln_vec<__nv_bfloat16>(p, a, st) : pick_ln_vec<float>(p, a, st);
}

// ------------------------------------------------------------------ backward
struct LnGradArgs {
  const void *dy, *x, *dres;
  int64_t rows;
  int n;
  const float *w, *mean, *rstd;
  void* dx;
  int dx_bf16;
  float* part;  // [grid][2][n] partial sums of dy xh and dy, or null
};

// A CTA takes rows blockIdx.x * kRows + group, + gridDim.x * kRows, ... and keeps the sums of
// its columns in registers over all of them.
template <typename T, int V, int WPR, int C>
__global__ void __launch_bounds__((WPR < 8 ? 8 : WPR) * 32) ln_backward_kernel(const LnGradArgs p) {
  constexpr int kWarps = WPR < 8 ? 8 : WPR;
  constexpr int kRows = kWarps / WPR;
  constexpr int kStep = WPR * 32 * V;
  __shared__ float s_red[2][2][kRows][WPR];
  rows_wait_prior();
  rows_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / WPR, wr = warp % WPR, bar = 1 + group;
  const int first = (wr * 32 + lane) * V;
  const float inv_n = 1.0f / static_cast<float>(p.n);
  float dw[C][V], db[C][V];
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[j][i] = db[j][i] = 0.0f;
  int par = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + group; row < p.rows;
       row += static_cast<int64_t>(gridDim.x) * kRows, par ^= 1) {
    const int64_t base = row * p.n;
    RowVec<T, V> rx[C], rd[C];
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = first + j * kStep;
      if (col < p.n) {
        rx[j].load(static_cast<const T*>(p.x) + base + col);
        rd[j].load(static_cast<const T*>(p.dy) + base + col);
      } else {
        rx[j].zero();
        rd[j].zero();
      }
    }
    const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = first + j * kStep;
      if (col < p.n) {
        float x[V], d[V], w[V];
        rx[j].unpack(x);
        rd[j].unpack(d);
        if (p.w) load_params<V>(p.w + col, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (x[i] - mean) * rstd;
          dw[j][i] += d[i] * xh;
          db[j][i] += d[i];
          const float a = p.w ? d[i] * w[i] : d[i];
          s1 += a;
          s2 += a * xh;
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (WPR > 1) {
      // two buffers in turn: a warp may be one row ahead of the others, not two
      float* r1 = s_red[par][0][group];
      float* r2 = s_red[par][1][group];
      if (lane == 0) {
        r1[wr] = s1;
        r2[wr] = s2;
      }
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(WPR * 32) : "memory");
      s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        s1 += r1[i];
        s2 += r2[i];
      }
    }
    const float c1 = s1 * inv_n, c2 = s2 * inv_n;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = first + j * kStep;
      if (col < p.n) {
        float x[V], d[V], w[V], o[V];
        rx[j].unpack(x);
        rd[j].unpack(d);
        if (p.w) load_params<V>(p.w + col, w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (x[i] - mean) * rstd;
          const float a = p.w ? d[i] * w[i] : d[i];
          o[i] = rstd * (a - c1 - xh * c2);
        }
        if (p.dres) {
          RowVec<T, V> rr;
          float r[V];
          rr.load(static_cast<const T*>(p.dres) + base + col);
          rr.unpack(r);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += r[i];
        }
        store_row_vec<V>(p.dx, p.dx_bf16, base + col, o);
      }
    }
  }
  if (!p.part) return;
  // the CTA's groups of rows add up in shared memory, in the order of the groups
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.n;
  if constexpr (kRows > 1) {
    extern __shared__ float s_part[];  // [2][n]
    for (int gi = 0; gi < kRows; ++gi) {
      if (group == gi) {
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int col = first + j * kStep + i;
            if (col < p.n) {
              s_part[col] = gi ? s_part[col] + dw[j][i] : dw[j][i];
              s_part[p.n + col] = gi ? s_part[p.n + col] + db[j][i] : db[j][i];
            }
          }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * p.n; c += kWarps * 32) out[c] = s_part[c];
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = first + j * kStep;
      if (col < p.n) {
        if constexpr (V < 4) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            out[col + i] = dw[j][i];
            out[p.n + col + i] = db[j][i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            *reinterpret_cast<float4*>(out + col + i) = make_float4(dw[j][i], dw[j][i + 1], dw[j][i + 2], dw[j][i + 3]);
            *reinterpret_cast<float4*>(out + p.n + col + i) =
                make_float4(db[j][i], db[j][i + 1], db[j][i + 2], db[j][i + 3]);
          }
        }
      }
    }
  }
}

// The same through a ring of rows (x, dy and the residual's gradient side by side in a slot).
// SUMS: the column sums too (else p.part is ignored).
template <typename T, int V, int WPR, int C, bool RES, bool SUMS>
__global__ void __launch_bounds__(kRingWarps * 32, 1) ln_backward_ring_kernel(const LnGradArgs p, int slots, unsigned* status) {
  constexpr int G = kRingWarps / WPR;
  constexpr int kStep = WPR * 32 * V;
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ float s_red[2][2][G][WPR];
  __shared__ volatile int s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / WPR, wr = warp % WPR, bar = 1 + group;
  const int first = (wr * 32 + lane) * V;
  const uint32_t row_bytes = static_cast<uint32_t>(p.n) * sizeof(T);
  const uint32_t slot_bytes = row_bytes * (RES ? 3 : 2);
  Ring ring{reinterpret_cast<uint64_t*>(s_ring) + group * kRingSlots,
            s_ring + kRingHeader + static_cast<size_t>(group) * slots * slot_bytes, slot_bytes, slots, &s_abort, status, 0, 0};
  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < G * kRingSlots; ++i) mbar_init(reinterpret_cast<uint64_t*>(s_ring) + i, 1);
    fence_mbar_init();
  }
  __syncthreads();
  rows_wait_prior();
  rows_allow_dependents();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * G;
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + group;
  const bool loader = wr == 0 && lane == 0;
  const uint64_t pol = l2_policy_evict_first();
  auto load_row = [&](int slot, int64_t r) {
    uint8_t* dst = ring.slot0 + static_cast<size_t>(slot) * slot_bytes;
    uint64_t* full = &ring.full[slot];
    mbar_arrive_expect_tx(full, slot_bytes);
    bulk_load(dst, static_cast<const T*>(p.x) + r * p.n, row_bytes, full, pol);
    bulk_load(dst + row_bytes, static_cast<const T*>(p.dy) + r * p.n, row_bytes, full, pol);
    if (RES) bulk_load(dst + 2 * row_bytes, static_cast<const T*>(p.dres) + r * p.n, row_bytes, full, pol);
  };
  if (loader)
    for (int i = 0; i < slots && row + i * stride < p.rows; ++i) load_row(i, row + i * stride);
  float w[C][V], dw[C][V], db[C][V];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int col = first + j * kStep;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      w[j][i] = 1.0f;
      dw[j][i] = db[j][i] = 0.0f;
    }
    if (p.w && col < p.n) load_params<V>(p.w + col, w[j]);
  }
  const float inv_n = 1.0f / static_cast<float>(p.n);
  float mean_n = 0.0f, rstd_n = 0.0f;
  if (row < p.rows) {
    mean_n = __ldg(p.mean + row);
    rstd_n = __ldg(p.rstd + row);
  }
  for (int par = 0; row < p.rows; row += stride, par ^= 1) {
    const float mean = mean_n, rstd = rstd_n;
    if (row + stride < p.rows) {  // the next row's, a row ahead
      mean_n = __ldg(p.mean + row + stride);
      rstd_n = __ldg(p.rstd + row + stride);
    }
    ring.wait();
    RowVec<T, V> rx[C], rd[C], rr[RES ? C : 1];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = first + j * kStep;
      if (col < p.n) {
        ring_read<T, V>(rx[j], ring.row(), col);
        ring_read<T, V>(rd[j], ring.row() + row_bytes, col);
        if constexpr (RES) ring_read<T, V>(rr[j], ring.row() + 2 * row_bytes, col);
        float x[V], d[V];
        rx[j].unpack(x);
        rd[j].unpack(d);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float xh = (x[i] - mean) * rstd;
          if constexpr (SUMS) {
            dw[j][i] += d[i] * xh;
            db[j][i] += d[i];
          }
          const float a = d[i] * w[j][i];
          s1 += a;
          s2 += a * xh;
        }
      }
    }
    s1 = warp_sum(s1);
    s2 = warp_sum(s2);
    if constexpr (WPR > 1) {
      float* r1 = s_red[par][0][group];
      float* r2 = s_red[par][1][group];
      if (lane == 0) {
        r1[wr] = s1;
        r2[wr] = s2;
      }
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(WPR * 32) : "memory");
      s1 = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        s1 += r1[i];
        s2 += r2[i];
      }
    } else {
      __syncwarp();
    }
    if (loader && row + slots * stride < p.rows) load_row(ring.at, row + slots * stride);
    ring.next();
    const float c1 = s1 * inv_n, c2 = s2 * inv_n;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int col = first + j * kStep;
      if (col < p.n) {
        float x[V], d[V], o[V];
        rx[j].unpack(x);
        rd[j].unpack(d);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = rstd * (d[i] * w[j][i] - c1 - (x[i] - mean) * rstd * c2);
        if constexpr (RES) {
          float r[V];
          rr[j].unpack(r);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += r[i];
        }
        store_row_vec<V>(p.dx, p.dx_bf16, row * p.n + col, o);
      }
    }
  }
  if (s_abort && loader) {  // copies still in flight land before the shared memory is used again
    volatile int no_abort = 0;
    for (int i = 0; i < slots; ++i) mbar_wait(&ring.full[i], ring.phase ^ (i < ring.at ? 1u : 0u), &no_abort);
  }
  if constexpr (!SUMS) return;
  if (!p.part) return;
  // The groups' sums meet in shared memory (within the ring, which is done with), each thread's
  // element k a row apart, padded so that both the writes and the sums by columns are free of
  // bank conflicts; they add up in the order of the groups.
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.n;
  constexpr int kLine = WPR * 32 + 32 / V, kPlane = C * V * kLine;
  static_assert(sizeof(float) * 2 * G * kPlane <= kRingBytes, "the groups' sums fit the ring");
  float* s_part = reinterpret_cast<float*>(s_ring);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float* at = s_part + 2 * group * kPlane + (j * V + i) * kLine + wr * 32 + lane;
      at[0] = dw[j][i];
      at[kPlane] = db[j][i];
    }
  __syncthreads();
  for (int c = threadIdx.x; c < p.n; c += kRingWarps * 32) {
    const float* at = s_part + ((c / kStep) * V + c % V) * kLine + c % kStep / V;
    float vw = 0.0f, vb = 0.0f;
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      vw += at[2 * gi * kPlane];
      vb += at[(2 * gi + 1) * kPlane];
    }
    out[c] = vw;
    out[p.n + c] = vb;
  }
}

template <typename T, int V, int WPR, int C, bool RES, bool SUMS = true>
static cudaError_t run_ln_grad_ring(const LnGradArgs& a, int* parts, unsigned* status, cudaStream_t st) {
  static bool done[64] = {false};
  const cudaError_t e = ring_attr(ln_backward_ring_kernel<T, V, WPR, C, RES, SUMS>, done);
  if (e != cudaSuccess) return e;
  RingPlan r = ring_plan(kRingWarps / WPR, static_cast<size_t>(a.n) * sizeof(T) * (RES ? 3 : 2), a.rows);
  r.smem = kRingHeader + kRingBytes;  // the groups' sums may take more than the slots
  *parts = r.grid;
  return launch_rows(ln_backward_ring_kernel<T, V, WPR, C, RES, SUMS>, dim3(static_cast<unsigned>(r.grid)), kRingWarps * 32,
                     r.smem, st, a, r.slots, status);
}

template <typename T, int V, bool RES>
static bool pick_ln_grad_ring(const LnGradArgs& a, int* parts, unsigned* status, cudaStream_t st, cudaError_t* e) {
  const int nch = (a.n + V - 1) / V;
  if (a.rows < 8 * static_cast<int64_t>(num_sms()) || nch < 96) return false;
  if constexpr (V == 8) {  // two chunks of 8 columns per thread at most
    if (nch <= 128) *e = run_ln_grad_ring<T, V, 2, 2, RES>(a, parts, status, st);
    else if (nch <= 256) *e = run_ln_grad_ring<T, V, 4, 2, RES>(a, parts, status, st);
    else if (nch <= 512) *e = run_ln_grad_ring<T, V, 8, 2, RES>(a, parts, status, st);
    else if (nch <= 1024) *e = run_ln_grad_ring<T, V, 16, 2, RES>(a, parts, status, st);
    else return false;
  } else {  // four of 4 columns
    if (nch <= 128) *e = run_ln_grad_ring<T, V, 2, 2, RES>(a, parts, status, st);
    else if (nch <= 256) *e = run_ln_grad_ring<T, V, 2, 4, RES>(a, parts, status, st);
    else if (nch <= 384) *e = run_ln_grad_ring<T, V, 4, 3, RES>(a, parts, status, st);
    else if (nch <= 512) *e = run_ln_grad_ring<T, V, 4, 4, RES>(a, parts, status, st);
    else if (nch <= 768) *e = run_ln_grad_ring<T, V, 8, 3, RES>(a, parts, status, st);
    else if (nch <= 1024) *e = run_ln_grad_ring<T, V, 8, 4, RES>(a, parts, status, st);
    else if (nch <= 1536) *e = run_ln_grad_ring<T, V, 16, 3, RES>(a, parts, status, st);
    else if (nch <= 2048) *e = run_ln_grad_ring<T, V, 16, 4, RES>(a, parts, status, st);
    else return false;
  }
  return true;
}

// Rows longer than a CTA's registers: the column sums by a kernel of their own, and dx by a
// CTA per row that reads the row twice.
template <typename T>
__global__ void __launch_bounds__(512) ln_backward_long_kernel(const LnGradArgs p) {
  __shared__ float s_red[2][16];
  rows_wait_prior();
  rows_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv_n = 1.0f / static_cast<float>(p.n);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * p.n;
  const float mean = __ldg(p.mean + blockIdx.x), rstd = __ldg(p.rstd + blockIdx.x);
  auto value = [&](const void* t, int col) {
    RowVec<T, 1> r;
    float v[1];
    r.load(static_cast<const T*>(t) + base + col);
    r.unpack(v);
    return v[0];
  };
  float s1 = 0.0f, s2 = 0.0f;
  for (int col = threadIdx.x; col < p.n; col += 512) {
    const float a = value(p.dy, col) * (p.w ? __ldg(p.w + col) : 1.0f);
    s1 += a;
    s2 += a * ((value(p.x, col) - mean) * rstd);
  }
  s1 = warp_sum(s1);
  s2 = warp_sum(s2);
  if (lane == 0) {
    s_red[0][warp] = s1;
    s_red[1][warp] = s2;
  }
  __syncthreads();
  s1 = s2 = 0.0f;
  for (int i = 0; i < 16; ++i) {
    s1 += s_red[0][i];
    s2 += s_red[1][i];
  }
  const float c1 = s1 * inv_n, c2 = s2 * inv_n;
  for (int col = threadIdx.x; col < p.n; col += 512) {
    const float a = value(p.dy, col) * (p.w ? __ldg(p.w + col) : 1.0f);
    const float xh = (value(p.x, col) - mean) * rstd;
    float o[1] = {rstd * (a - c1 - xh * c2)};
    if (p.dres) o[0] += value(p.dres, col);
    store_row_vec<1>(p.dx, p.dx_bf16, base + col, o);
  }
}

constexpr int kLongWarps = 8;

// A CTA takes 32 V columns and a slab of rows; warp w the slab's rows w, w + 8, ...
template <typename T, int V>
__global__ void __launch_bounds__(kLongWarps * 32) ln_columns_long_kernel(const LnGradArgs p, int64_t rows_per_part) {
  __shared__ float s_sum[kLongWarps][2][V][32];
  rows_wait_prior();
  rows_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = (blockIdx.x * 32 + lane) * V;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_part;
  const int64_t r1 = min(p.rows, r0 + rows_per_part);
  float dw[V], db[V];
#pragma unroll
  for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.0f;
  if (col < p.n) {
#pragma unroll 4
    for (int64_t r = r0 + warp; r < r1; r += kLongWarps) {
      RowVec<T, V> rx, rd;
      float x[V], d[V];
      rx.load(static_cast<const T*>(p.x) + r * p.n + col);
      rd.load(static_cast<const T*>(p.dy) + r * p.n + col);
      const float mean = __ldg(p.mean + r), rstd = __ldg(p.rstd + r);
      rx.unpack(x);
      rd.unpack(d);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dw[i] += d[i] * ((x[i] - mean) * rstd);
        db[i] += d[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    s_sum[warp][0][i][lane] = dw[i];
    s_sum[warp][1][i][lane] = db[i];
  }
  __syncthreads();
  float* out = p.part + static_cast<int64_t>(blockIdx.y) * 2 * p.n;
  for (int t = threadIdx.x; t < 2 * 32 * V; t += kLongWarps * 32) {
    const int h = t / (32 * V), k = t % (32 * V), c = blockIdx.x * 32 * V + k;
    if (c >= p.n) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kLongWarps; ++w) v += s_sum[w][h][k % V][k / V];
    out[static_cast<int64_t>(h) * p.n + c] = v;
  }
}

// ------------------------------------------------------------------ column sums
// 32 columns per CTA; each of its warps adds its share of the partial sums, in order, and the
// shares are added in order.  (Sixteen warps: at the usual 148 parts a thread's ten loads are in
// flight together.)  The partial sums are cleared behind it: a zero-filled workspace that other
// calls share stays so.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) column_sums_kernel(float* part, int parts, int64_t width, int64_t n0,
                                                                     float* out0, float* out1) {
  __shared__ float s[kSumWarps][32];
  rows_wait_prior();
  rows_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float v = 0.0f;
  if (c < width) {
    const int p0 = parts * warp / kSumWarps, p1 = parts * (warp + 1) / kSumWarps;
#pragma unroll 10
    for (int q = p0; q < p1; ++q) v += __ldcg(part + static_cast<int64_t>(q) * width + c);
    for (int q = p0; q < p1; ++q) __stcg(part + static_cast<int64_t>(q) * width + c, 0.0f);
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < width) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumWarps; ++i) v += s[i][lane];
    if (c < n0) {
      if (out0) out0[c] = v;
    } else if (out1) {
      out1[c - n0] = v;
    }
  }
}

cudaError_t launch_column_sums(float* part, int parts, int64_t width, int64_t n0, float* out0, float* out1,
                               cudaStream_t st) {
  return launch_rows(column_sums_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), kSumWarps * 32, 0, st, part,
                     parts, width, n0, out0, out1);
}

constexpr int kLnMaxParts = 2 * 148;

// CTAs of the backward kernel (and partial sums): two per SM, no more than groups of rows.
static int ln_parts(int64_t rows) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rows, std::min(2 * num_sms(), kLnMaxParts))));
}

size_t layernorm_grad_workspace_bytes(int64_t rows, int64_t cols) {
  return static_cast<size_t>(std::min<int64_t>(rows, kLnMaxParts)) * 2 * cols * sizeof(float);
}

template <typename T, int V, int WPR, int C>
static cudaError_t run_ln_grad(const LnGradArgs& a, int parts, cudaStream_t st) {
  constexpr int kWarps = WPR < 8 ? 8 : WPR, kRows = kWarps / WPR;
  const size_t smem = kRows > 1 && a.part ? 2 * static_cast<size_t>(a.n) * sizeof(float) : 0;
  return launch_rows(ln_backward_kernel<T, V, WPR, C>, dim3(static_cast<unsigned>(parts)), kWarps * 32, smem, st, a);
}

// Returns false where the row is too long for the registers of a CTA.
template <typename T, int V>
static bool pick_ln_grad(const LnGradArgs& a, int parts, cudaStream_t st, cudaError_t* e) {
  const int nch = (a.n + V - 1) / V;
  // at most 16 columns per thread; single elements and pairs fewer, on more warps per row, where
  // that reaches (4096 x 2881 BF16: 16 elements a thread 115 us, 4 to 8 on 16 warps 63)
  constexpr int C = V == 8 ? 2 : 4;
  if constexpr (V < 4) {
    if (nch > 2048 && nch <= 4096) {
      *e = run_ln_grad<T, V, 16, 8>(a, parts, st);
      return true;
    }
    if constexpr (V == 1) {
      if (nch > 4096 && nch <= 8192) {
        *e = run_ln_grad<T, V, 16, 16>(a, parts, st);
        return true;
      }
    }
  }
  if (nch <= 32) *e = run_ln_grad<T, V, 1, 1>(a, parts, st);
  else if (nch <= 32 * C) *e = run_ln_grad<T, V, 1, C>(a, parts, st);
  else if (nch <= 128 * C) *e = run_ln_grad<T, V, 4, C>(a, parts, st);
  else if (nch <= 256 * C) *e = run_ln_grad<T, V, 8, C>(a, parts, st);
  else if (nch <= 512 * C) *e = run_ln_grad<T, V, 16, C>(a, parts, st);
  else return false;
  return true;
}

template <typename T>
static cudaError_t ln_grad(const LnGradArgs& a, float* dw, float* db, unsigned* status, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = a.n % V == 0 && aligned16_rows(a.x) && aligned16_rows(a.dy) && aligned16_rows(a.dres) &&
                   aligned16_rows(a.dx) && aligned16_rows(a.w);
  int parts = ln_parts(a.rows);
  cudaError_t e = cudaSuccess;
  if (vec && (a.dres ? pick_ln_grad_ring<T, V, true>(a, &parts, status, st, &e)
                     : pick_ln_grad_ring<T, V, false>(a, &parts, status, st, &e))) {
    if (e != cudaSuccess || !a.part) return e;
    return launch_column_sums(a.part, parts, 2 * static_cast<int64_t>(a.n), a.n, dw, db, st);
  }
  const bool two = !vec && pairs_ok(a.n, a.w, nullptr);
  if (!(vec   ? pick_ln_grad<T, V>(a, parts, st, &e)
        : two ? pick_ln_grad<T, 2>(a, parts, st, &e)
              : pick_ln_grad<T, 1>(a, parts, st, &e))) {
    // the column pass first: dx may be written in dy's place
    if (a.part) {
      const int cols = 32 * (vec ? V : 1), tiles = (a.n + cols - 1) / cols;
      parts = static_cast<int>(std::min<int64_t>(parts, std::max(1, 8 * num_sms() / tiles)));
      const int64_t per = (a.rows + parts - 1) / parts;
      parts = static_cast<int>((a.rows + per - 1) / per);
      const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(parts));
      e = vec ? launch_rows(ln_columns_long_kernel<T, V>, grid, kLongWarps * 32, 0, st, a, per)
              : launch_rows(ln_columns_long_kernel<T, 1>, grid, kLongWarps * 32, 0, st, a, per);
    }
    if (e == cudaSuccess) {
      int ctas = 0;
      // up to 2048 words: the ring without the sums; longer or unaligned rows are read twice
      if (vec && a.n / V <= 2048 && a.rows >= 2 * static_cast<int64_t>(num_sms()))
        e = a.dres ? run_ln_grad_ring<T, V, 16, 4, true, false>(a, &ctas, status, st)
                   : run_ln_grad_ring<T, V, 16, 4, false, false>(a, &ctas, status, st);
      else
        e = launch_rows(ln_backward_long_kernel<T>, dim3(static_cast<unsigned>(a.rows)), 512, 0, st, a);
    }
  }
  if (e != cudaSuccess || !a.part) return e;
  return launch_column_sums(a.part, parts, 2 * static_cast<int64_t>(a.n), a.n, dw, db, st);
}

cudaError_t launch_layernorm_grad(const LayerNormGradProblem& p, unsigned* status, cudaStream_t st) {
  LnGradArgs a{};
  a.dy = p.dy;
  a.x = p.x;
  a.dres = p.dres;
  a.rows = p.rows;
  a.n = static_cast<int>(p.cols);
  a.w = p.weight;
  a.mean = p.mean;
  a.rstd = p.rstd;
  a.dx = p.dx;
  a.dx_bf16 = p.dx_bf16;
  a.part = p.dweight || p.dbias ? p.ws : nullptr;
  return p.bf16 ? ln_grad<__nv_bfloat16>(a, p.dweight, p.dbias, status, st)
                : ln_grad<float>(a, p.dweight, p.dbias, status, st);
}

}  // namespace fp4
