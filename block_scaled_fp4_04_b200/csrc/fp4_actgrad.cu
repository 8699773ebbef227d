// fp4_actgrad.cu -- backward pass of the activation between two matrix products.
//
//   plain  dZ = dH act'(Z)                                       [rows, cols]
//   gated  dZ = [dH U act'(G) | dH act(G)], H = act(G) U          [rows, 2 cols]
//
// The gated result is one matrix, the operand of a single product with the stacked weights:
// dX = [dG dU] . [Wg; Wu].  Besides (or instead of) FP32 / BF16 it can be written as NVFP4 or
// MXFP4 codes with scales in the tensor cores' layout, and its column sums give the bias
// gradients.  Memory-bound: one pass, every element read once; a special-function exponential
// and reciprocal per element stay below the memory time.
#include "fp4_act.cuh"
#include "fp4_rows.cuh"

namespace fp4 {

struct ActGradArgs {
  const void *dh, *g, *u;
  int64_t rows;
  int n;  // columns of dh
  int act;
  void* dz;
  int dz_bf16;
  int64_t ldz;       // columns of dz: n, or 2 n
  int64_t rows_per;  // rows of one slab (grid.y slabs)
  float* part;       // [slabs][ldz] partial column sums, or null
  RowCodes q;
  unsigned* amax;
  unsigned* status;
};

constexpr int kAgWarps = 8;

// Words of a row per lane: several where a word is a single element or a pair, so that a row's
// address is worked out once for as many bytes.
template <int V>
__host__ __device__ constexpr int ag_words() { return V == 1 ? 4 : V == 2 ? 2 : 1; }

// A CTA takes 32 J V columns (J words a lane, 32 V columns apart) and a slab of rows; warp w the
// slab's rows w, w + 8, ...
template <typename T, int V, bool GATED, int FMT>
__global__ void __launch_bounds__(kAgWarps * 32) act_grad_kernel(const ActGradArgs p) {
  constexpr int kHalves = GATED ? 2 : 1;
  constexpr int U = 2;  // rows in flight per warp
  constexpr int J = ag_words<V>();
  __shared__ float s_sum[kAgWarps][kHalves][32 * V * J];
  rows_wait_prior();
  rows_allow_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col0 = (blockIdx.x * 32 * J + lane) * V;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * p.rows_per;
  const int64_t r1 = min(p.rows, r0 + p.rows_per);
  float acc[kHalves][J][V];
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[h][j][i] = 0.0f;
  float gs = 1.0f;
  if constexpr (FMT == kCodesNv) gs = *p.q.g;
  uint32_t m = 0;
  bool bad = false;
  with_act(p.act, [&](auto tag) __attribute__((always_inline)) {
    constexpr int A = decltype(tag)::value;
    for (int64_t r = r0 + warp; r < r1; r += kAgWarps * U) {
      RowVec<T, V> rd[U][J], rg[U][J], ru[U][J];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t rr = r + k * kAgWarps;
        const int64_t at = rr * p.n + col0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          rd[k][j].zero();
          rg[k][j].zero();
          ru[k][j].zero();
          if (col0 + j * 32 * V < p.n && rr < r1) {
            rd[k][j].load(static_cast<const T*>(p.dh) + at + j * 32 * V);
            rg[k][j].load(static_cast<const T*>(p.g) + at + j * 32 * V);
            if constexpr (GATED) ru[k][j].load(static_cast<const T*>(p.u) + at + j * 32 * V);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int64_t rr = r + k * kAgWarps;
        if (rr >= r1) break;  // warp-uniform
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int col = col0 + j * 32 * V;
          const bool col_ok = col < p.n;
          float d[V], g[V], u[V], z[kHalves][V];
          rd[k][j].unpack(d);
          rg[k][j].unpack(g);
          ru[k][j].unpack(u);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float value;
            const float slope = act_slope<A>(g[i], value);
            if constexpr (GATED) {
              z[0][i] = d[i] * u[i] * slope;
              z[1][i] = d[i] * value;
            } else {
              z[0][i] = d[i] * slope;
            }
          }
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            const int64_t zc = static_cast<int64_t>(h) * p.n + col;
            if (col_ok) {
              if (p.dz) store_row_vec<V>(p.dz, p.dz_bf16, rr * p.ldz + zc, z[h]);
#pragma unroll
              for (int i = 0; i < V; ++i) acc[h][j][i] += z[h][i];
              if (p.amax) {
#pragma unroll
                for (int i = 0; i < V; ++i) m = max(m, abs_bits_of(z[h][i]));
              }
            }
            if constexpr (FMT != kCodesNone) bad |= encode_row_vec<FMT, V>(p.q, gs, rr, zc, col_ok, z[h]);
          }
        }
      }
    }
  });
  if (p.amax) {
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0 && m) atomicMax(p.amax, m);
  }
  if (FMT != kCodesNone && bad) atomicOr(p.status, kStatusNonFinite);
  if (!p.part) return;
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) s_sum[warp][h][(j * V + i) * 32 + lane] = acc[h][j][i];
  __syncthreads();
  for (int t = threadIdx.x; t < kHalves * 32 * V * J; t += kAgWarps * 32) {
    const int h = t / (32 * V * J), k = t % (32 * V * J);  // column k of the CTA's: element k % V of a lane's word
    const int c = blockIdx.x * 32 * V * J + k;
    if (c >= p.n) continue;
    const int j = k / (32 * V), l = k % (32 * V) / V, i = k % V;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kAgWarps; ++w) v += s_sum[w][h][(j * V + i) * 32 + l];
    p.part[static_cast<int64_t>(blockIdx.y) * p.ldz + static_cast<int64_t>(h) * p.n + c] = v;
  }
}

constexpr int kAgMaxSlabs = 64;   // partial sums per column
constexpr int kAgSlabRows = 64;   // rows of a slab where no column sums are wanted

size_t act_grad_workspace_bytes(int64_t rows, int64_t cols, int gated) {
  const int64_t slabs = std::min<int64_t>(kAgMaxSlabs, (rows + kAgWarps - 1) / kAgWarps);
  return static_cast<size_t>(slabs) * cols * (gated ? 2 : 1) * sizeof(float);
}

template <typename T, int V, int FMT>
static cudaError_t run_ag(ActGradArgs a, cudaStream_t st) {
  // column sums: few enough slabs that their partial sums stay small beside the tensor
  int64_t per = kAgSlabRows;
  if (a.part) per = std::max<int64_t>((a.rows + kAgMaxSlabs - 1) / kAgMaxSlabs, kAgWarps);
  // the slabs of a launch are grid.y, at most 65535
  per = std::max(per, (a.rows + 65534) / 65535);
  a.rows_per = per;
  constexpr int kCols = 32 * V * ag_words<V>();
  const dim3 grid(static_cast<unsigned>((a.n + kCols - 1) / kCols), static_cast<unsigned>((a.rows + per - 1) / per));
  return a.u ? launch_rows(act_grad_kernel<T, V, true, FMT>, grid, kAgWarps * 32, 0, st, a)
             : launch_rows(act_grad_kernel<T, V, false, FMT>, grid, kAgWarps * 32, 0, st, a);
}

template <typename T>
static cudaError_t pick_ag(const ActGradArgs& a, int fmt, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  auto al = [](const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  const bool vec = a.n % V == 0 && al(a.dh) && al(a.g) && al(a.u) && al(a.dz);
  if (fmt == kCodesNv) return vec ? run_ag<T, V, kCodesNv>(a, st) : cudaErrorInvalidValue;
  if (fmt == kCodesMx) return vec ? run_ag<T, V, kCodesMx>(a, st) : cudaErrorInvalidValue;
  if (vec) return run_ag<T, V, kCodesNone>(a, st);
  return a.n % 2 == 0 ? run_ag<T, 2, kCodesNone>(a, st) : run_ag<T, 1, kCodesNone>(a, st);
}

cudaError_t launch_act_grad(const ActGradProblem& p, unsigned* status, cudaStream_t st) {
  ActGradArgs a{};
  a.dh = p.dh;
  a.g = p.g;
  a.u = p.u;
  a.rows = p.rows;
  a.n = static_cast<int>(p.cols);
  a.act = p.act;
  a.dz = p.dz;
  a.dz_bf16 = p.dz_bf16;
  a.ldz = p.cols * (p.u ? 2 : 1);
  a.part = p.dbias ? p.ws : nullptr;
  a.q = RowCodes{p.q.codes, p.q.scales, p.q.g, a.ldz, (a.ldz / (p.q.fmt == kCodesMx ? 32 : 16) + 3) / 4};
  a.amax = reinterpret_cast<unsigned*>(p.amax_out);
  a.status = status;
  const cudaError_t e = p.bf16 ? pick_ag<__nv_bfloat16>(a, p.q.fmt, st) : pick_ag<float>(a, p.q.fmt, st);
  if (e != cudaSuccess || !a.part) return e;
  int64_t per = std::max<int64_t>((p.rows + kAgMaxSlabs - 1) / kAgMaxSlabs, kAgWarps);
  return launch_column_sums(a.part, static_cast<int>((p.rows + per - 1) / per), a.ldz, a.ldz, p.dbias, nullptr, st);
}

}  // namespace fp4
