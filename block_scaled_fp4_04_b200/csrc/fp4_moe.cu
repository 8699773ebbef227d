// fp4_moe.cu -- tokens to their experts and back: a stable sort of the router's (token, choice)
// slots by expert, the copy of token rows into the experts' order (as they are, as FP4 codes in
// the grouped scale layout, or as 8-bit rows with a scale each), the weighted sum on the way back,
// and its gradients.  Also the 8-bit quantizer of plain rows, which is the same kernel.
//
// A slot s = t topk + j is token t's j-th choice; row_of[s] is its row in the experts' order, or
// -1 where it has no expert.  All of these but the sort go by token, not by sorted row: a token's
// row is read once, and encoded once, for all its experts.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cstdint>

#include "fp4_codes.cuh"
#include "fp4_moe.h"
#include "fp4_rows.cuh"

namespace fp4 {

// ------------------------------------------------------------------------------------- sort
// A counting sort that keeps the slots' order within an expert.  Each warp counts a contiguous
// segment of slots per expert in its own shared counters; prefix sums over warps and experts turn
// the counts into first rows; then each warp passes over its segment again and hands out rows in
// order, 32 slots at a time: equal experts within the 32 find one another by votes on the bits of
// their numbers (16384 slots in one block: 16.0 us; with the match instruction 18.7), and a slot's
// place among them is the number of lower lanes.  No atomic decides an order, so the result is the
// same every time.  What bounds it: launches, barriers and the latency of a few dependent steps.
//
// Up to kSortOneBlock slots one block does it all, up to kSortCluster a cluster of eight whose blocks
// read one another's counts: one launch.  Beyond, blocks of kSortChunk slots or more first write
// their counts to the workspace, and each block of a second launch sums those before it.  (Calls back
// to back: 1000 slots 7.2 us by one block, 5.6 by a cluster; 16384 slots 16.0, 8.4 by a cluster, 11.7
// by two launches; 131072 slots 19.3 by a cluster, 13.3 by two launches.)
struct SortArgs {
  const void* ids;
  int64_t slots, chunk;
  int E;
  int blocks;
  uint32_t* hist;  // [blocks, E], null for one block or one cluster
  int32_t *offsets, *row_of, *scale_row_of;
};

constexpr int kSortThreads = 1024;
constexpr int64_t kSortOneBlock = 512, kSortCluster = 32768, kSortChunk = 4096;
constexpr int kSortClusterBlocks = 8, kSortMaxBlocks = 128, kSortKeys = 16;
// Shared memory of a block: a column of counters for each warp, three more, and two launches' partial sums.
constexpr size_t sort_smem(int threads, int E, bool parts) {
  return (static_cast<size_t>(threads / 32) * (E + 1) + 3 * E + (parts ? 2 * threads : 0)) * 4;
}

template <typename ID>
__device__ __forceinline__ int sort_key(const SortArgs& a, int64_t s, int64_t hi) {
  if (s >= hi) return a.E;
  const ID id = static_cast<const ID*>(a.ids)[s];
  return id >= 0 && id < static_cast<ID>(a.E) ? static_cast<int>(id) : a.E;
}

template <typename ID>
__global__ void __launch_bounds__(kSortThreads) moe_hist_kernel(const SortArgs a) {
  extern __shared__ uint32_t s_cnt[];
  rows_wait_prior();
  rows_allow_dependents();
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) s_cnt[e] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * a.chunk, hi = min(a.slots, lo + a.chunk);
  for (int64_t s = lo + threadIdx.x; s < hi; s += blockDim.x) atomicAdd(&s_cnt[sort_key<ID>(a, s, hi)], 1u);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.hist[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_cnt[e];
}

template <typename ID>
__global__ void __launch_bounds__(kSortThreads, 1) moe_sort_kernel(const SortArgs a) {
  extern __shared__ uint32_t s_mem[];
  const int E = a.E, E1 = E + 1;  // the last counter takes the slots without an expert
  const int warps = blockDim.x / 32, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  uint32_t* s_cnt = s_mem;              // [warps, E1]
  uint32_t* s_all = s_cnt + warps * E1;  // [E] rows of an expert, then its first row
  uint32_t* s_before = s_all + E;       // [E] of them in earlier blocks
  uint32_t* s_sfirst = s_before + E;    // [E] its first row in the grouped scale layout
  uint32_t* s_part = s_sfirst + E;      // [2, blockDim.x] (several blocks only)
  rows_wait_prior();
  rows_allow_dependents();
  for (int i = threadIdx.x; i < warps * E1; i += blockDim.x) s_cnt[i] = 0;
  const int64_t lo = blockIdx.x * a.chunk, hi = min(a.slots, lo + a.chunk);
  const int64_t seg = ((hi - lo + warps - 1) / warps + 31) / 32 * 32;
  const int64_t from = min(hi, lo + warp * seg), to = min(hi, from + seg);
  uint32_t* mine = s_cnt + warp * E1;
  // a segment's numbers stay in registers between the two passes, all asked for at once, where it
  // is that short
  int key[kSortKeys];
  const bool kept = seg <= 32 * kSortKeys;
  if (kept) {
#pragma unroll
    for (int i = 0; i < kSortKeys; ++i) key[i] = sort_key<ID>(a, from + 32 * i + lane, to);
  }
  __syncthreads();
  if (kept) {
#pragma unroll
    for (int i = 0; i < kSortKeys; ++i)
      if (from + 32 * i + lane < to) atomicAdd(&mine[key[i]], 1u);
  } else {
    for (int64_t s = from + lane; s < to; s += 32) atomicAdd(&mine[sort_key<ID>(a, s, to)], 1u);
  }
  const bool cluster = !a.hist && gridDim.x > 1;
  if (a.hist) {
    // columns of the histograms: neighbouring threads take neighbouring experts, and the blocks
    // are shared out over as many groups of threads as there are
    int wide = 32;
    while (wide < E) wide *= 2;  // at most 1024
    const int parts = blockDim.x / wide, e = threadIdx.x % wide, part = threadIdx.x / wide;
    uint32_t before = 0, all = 0;
    if (e < E) {
#pragma unroll 4
      for (int b = part; b < a.blocks; b += parts) {
        const uint32_t c = __ldcg(a.hist + static_cast<int64_t>(b) * E + e);
        all += c;
        if (b < static_cast<int>(blockIdx.x)) before += c;
      }
    }
    s_part[threadIdx.x] = all;
    s_part[blockDim.x + threadIdx.x] = before;
    __syncthreads();
    if (part == 0 && e < E) {
      for (int q = 1; q < parts; ++q) {
        all += s_part[q * wide + e];
        before += s_part[blockDim.x + q * wide + e];
      }
      s_all[e] = all;
      s_before[e] = before;
    }
  }
  __syncthreads();
  // counts of an expert become the places of each warp's first row among the block's
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    uint32_t sum = 0;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) {
      const uint32_t c = s_cnt[w * E1 + e];
      s_cnt[w * E1 + e] = sum;
      sum += c;
    }
    if (!a.hist) {
      s_all[e] = sum;
      s_before[e] = 0;
    }
  }
  if (cluster) {
    cluster_sync_all();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      uint32_t all = 0, before = 0;
#pragma unroll
      for (uint32_t r = 0; r < kSortClusterBlocks; ++r) {
        uint32_t c;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c) : "r"(cluster_addr(smem_u32(s_all + e), r)));
        all += c;
        if (r < blockIdx.x) before += c;
      }
      s_sfirst[e] = all;
      s_before[e] = before;
    }
    cluster_sync_all();  // the counts have been read: they may change, and this block may end
    for (int e = threadIdx.x; e < E; e += blockDim.x) s_all[e] = s_sfirst[e];
  }
  __syncthreads();
  if (warp == 0) {  // first rows: prefix sums over the experts
    uint32_t rows = 0, blocks = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + lane;
      const uint32_t n = e < E ? s_all[e] : 0u, nb = (n + 127) / 128;
      uint32_t in = n, inb = nb;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t t = __shfl_up_sync(0xFFFFFFFFu, in, d), tb = __shfl_up_sync(0xFFFFFFFFu, inb, d);
        if (lane >= d) {
          in += t;
          inb += tb;
        }
      }
      if (e < E) {
        const uint32_t first = rows + in - n;
        s_all[e] = first + s_before[e];
        s_sfirst[e] = (blocks + inb - nb) * 128 + s_before[e];
        if (blockIdx.x == 0) a.offsets[e] = static_cast<int32_t>(first);
      }
      rows += __shfl_sync(0xFFFFFFFFu, in, 31);
      blocks += __shfl_sync(0xFFFFFFFFu, inb, 31);
    }
    if (lane == 0 && blockIdx.x == 0) a.offsets[E] = static_cast<int32_t>(rows);
  }
  __syncthreads();
  const int bits = 32 - __clz(E);  // of the numbers up to E
  auto place = [&](int64_t s, int k) {
    unsigned same = 0xFFFFFFFFu;  // lanes with this expert: a vote on each bit of its number
    for (int b = 0; b < bits; ++b) {
      const bool one = k >> b & 1;
      const unsigned ones = __ballot_sync(0xFFFFFFFFu, one);
      same &= one ? ones : ~ones;
    }
    const uint32_t at = mine[k], lower = __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (lower == 0) mine[k] = at + __popc(same);
    __syncwarp();
    if (s < to) {
      a.row_of[s] = k < E ? static_cast<int32_t>(s_all[k] + at + lower) : -1;
      if (a.scale_row_of) a.scale_row_of[s] = k < E ? static_cast<int32_t>(s_sfirst[k] + at + lower) : -1;
    }
  };
  if (kept) {
#pragma unroll
    for (int i = 0; i < kSortKeys; ++i)
      if (from + 32 * i < to) place(from + 32 * i + lane, key[i]);  // (the same for the whole warp)
  } else {
    for (int64_t s0 = from; s0 < to; s0 += 32) place(s0 + lane, sort_key<ID>(a, s0 + lane, to));
  }
}

static int sort_blocks(int64_t slots, int64_t* chunk) {
  if (slots <= kSortOneBlock) {
    *chunk = slots;
    return 1;
  }
  if (slots <= kSortCluster) {
    *chunk = (slots + kSortClusterBlocks - 1) / kSortClusterBlocks;
    return kSortClusterBlocks;
  }
  *chunk = std::max(kSortChunk, (slots + kSortMaxBlocks - 1) / kSortMaxBlocks);
  return static_cast<int>((slots + *chunk - 1) / *chunk);
}

size_t moe_sort_workspace_bytes(int64_t slots, int E) {
  int64_t chunk;
  const int blocks = sort_blocks(slots, &chunk);
  return slots <= kSortCluster ? 0 : static_cast<size_t>(blocks) * E * sizeof(uint32_t);
}

template <typename ID>
static cudaError_t sort_typed(const SortArgs& a, cudaStream_t st) {
  auto kern = moe_sort_kernel<ID>;
  // one block: as many warps as segments of 32 slots, but at least one expert's column a thread
  const int64_t want = std::max<int64_t>((std::min(a.chunk, a.slots) + 31) / 32 * 32, (std::min(a.E, 256) + 31) / 32 * 32);
  const int threads = a.hist ? kSortThreads : static_cast<int>(std::min<int64_t>(kSortThreads, want));
  const size_t smem = sort_smem(threads, a.E, a.hist != nullptr);
  cudaError_t e = cudaSuccess;
  // The limit is one for all calls of a kernel on a device, from all host threads: the largest sort's, and
  // never less again (with each call's own size a call could find another's, and be refused).
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (smem > 48 * 1024 && (dev < 0 || dev >= 64 || !attr_done[dev])) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sort_smem(kSortThreads, kMaxGroups, true)));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_done[dev] = true;
  }
  if (a.hist) {
    e = launch_rows(moe_hist_kernel<ID>, dim3(a.blocks), kSortThreads, static_cast<size_t>(a.E + 1) * 4, st, a);
    if (e != cudaSuccess) return e;
  }
  return launch_rows_cluster(kern, dim3(a.blocks), threads, smem, st, a.hist ? 1 : a.blocks, a);
}

cudaError_t launch_moe_sort(const void* ids, int id_bytes, int64_t slots, int E, int32_t* offsets, int32_t* row_of,
                            int32_t* scale_row_of, void* ws, cudaStream_t st) {
  SortArgs a{};
  a.ids = ids;
  a.slots = slots;
  a.E = E;
  a.blocks = sort_blocks(slots, &a.chunk);
  a.hist = slots > kSortCluster ? static_cast<uint32_t*>(ws) : nullptr;
  a.offsets = offsets;
  a.row_of = row_of;
  a.scale_row_of = scale_row_of;
  return id_bytes == 8 ? sort_typed<int64_t>(a, st) : sort_typed<int32_t>(a, st);
}

// --------------------------------------------------------------------------------- dispatch
// How rows are moved.  Words of 16 bytes of the input (V = 8 BF16 or 4 FP32) where all rows start at
// 16 bytes (a matrix of the other type then moves 8 or 32 bytes at once, which its rows' starts
// allow).  Other widths: the words of the matrix that is written (for the gradient, also of the one
// that it shares rows with) still stand at 16 bytes, from some element of the row on, and the values
// for them come from the two words of the other matrix that hold them (RowVec::load_any); the
// elements before and behind go one by one.  Narrow rows go one by one altogether.  (2000 tokens, 6
// choices, 2049 BF16 columns, floor 8.8 / 8.8 / 16.3 us: dispatch 12.5 us, sum 24, gradient 26.7; one by one
// 20, 32 and 53.)
enum { kByElement = 0, kByWord = 1, kByShift = 2 };

static int row_way(int64_t cols, int bf16) {
  const int v = bf16 ? 8 : 4;
  return cols % v == 0 ? kByWord : cols >= 64 ? kByShift : kByElement;
}

template <typename T, int WAY>
__host__ __device__ constexpr int word_size() { return WAY == kByElement ? 1 : 16 / static_cast<int>(sizeof(T)); }

// A row's words by its offset in the matrix: word i holds elements [first + V i, first + V (i + 1)).
// kByShift leaves out a word more than it has to on either side, so that the words of another row
// around the same elements, and around those behind the last word, lie within that row.
template <int V, int WAY>
struct RowSpan {
  int first, words, cols;
  __device__ __forceinline__ RowSpan(int64_t at, int64_t columns) : cols(static_cast<int>(columns)) {
    if constexpr (WAY == kByShift) {
      first = (static_cast<int>(-at) & (V - 1)) + V;
      words = max(0, (cols - first) / V - 1);
    } else {
      first = 0;
      words = cols / V;
    }
  }
  __device__ __forceinline__ int singles() const { return cols - words * V; }  // kByShift: at most 4 V - 2
  __device__ __forceinline__ int single(int i) const { return i < first ? i : i + words * V; }
};

// A row over several blocks of `per` words.
static dim3 row_grid(int64_t tokens, int64_t words, int64_t per) {
  return dim3(static_cast<unsigned>(tokens), static_cast<unsigned>((words + per - 1) / per));
}

template <int WAY>
struct WayTag {
  static constexpr int value = WAY;
};
template <typename F>
static cudaError_t with_rows(int bf16, int way, F&& f) {
  if (bf16) {
    if (way == kByWord) return f(__nv_bfloat16{}, WayTag<kByWord>{});
    if (way == kByShift) return f(__nv_bfloat16{}, WayTag<kByShift>{});
    return f(__nv_bfloat16{}, WayTag<kByElement>{});
  }
  if (way == kByWord) return f(float{}, WayTag<kByWord>{});
  if (way == kByShift) return f(float{}, WayTag<kByShift>{});
  return f(float{}, WayTag<kByElement>{});
}

// Threads that take `per` words each of a row's `words`.
static int row_threads(int64_t words, int per, int most) {
  return static_cast<int>(std::min<int64_t>(most, std::max<int64_t>(32, ((words + per - 1) / per + 31) / 32 * 32)));
}

// y[row_of[t, j]] = x[t]: a block copies kCopyWords words a thread of one token's row to its topk
// places.  Bound by the copy rate: 16384 x 8 x 4096 BF16 (a tenth of the slots without an expert)
// 174 us, 168 at the rate; 4096 x 4 x 2880 21 us, 18 at the rate.
constexpr int kCopyWords = 4, kCopyThreads = 256;

template <typename T, int WAY>
__global__ void __launch_bounds__(kCopyThreads) moe_dispatch_kernel(const DispatchProblem p) {
  constexpr int V = word_size<T, WAY>(), W = kCopyWords;
  rows_wait_prior();
  rows_allow_dependents();
  const int64_t t = blockIdx.x, from = t * p.cols;
  const T* x = static_cast<const T*>(p.x);
  const int32_t* rows = p.row_of + t * p.topk;
  const bool same = p.y_bf16 == (sizeof(T) == 2);  // one type: the same bits, those of a NaN too
  const int w0 = blockIdx.y * blockDim.x * W + threadIdx.x;
  RowVec<T, V> in[W];
  if constexpr (WAY != kByShift) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (w0 + i * blockDim.x < p.cols / V) in[i].load(x + from + (w0 + i * blockDim.x) * V);
  }
  for (int j = 0; j < p.topk; ++j) {
    const int32_t row = __ldg(rows + j);
    if (row < 0) continue;
    const int64_t to = row * p.cols;
    const RowSpan<V, WAY> span(to, p.cols);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const int w = w0 + i * blockDim.x, e = span.first + w * V;
      if (w >= span.words) continue;
      if constexpr (WAY == kByShift) in[i].load_any(x, from + e);
      if (same) {
        in[i].store(static_cast<T*>(p.y) + to + e);
      } else {
        float v[V];
        in[i].unpack(v);
        store_row_vec<V>(p.y, p.y_bf16, to + e, v);
      }
    }
    if (WAY == kByShift && blockIdx.y == 0)
      for (int i = threadIdx.x; i < span.singles(); i += blockDim.x) {
        const int e = span.single(i);
        RowVec<T, 1> one;
        one.load(x + from + e);
        if (same) {
          one.store(static_cast<T*>(p.y) + to + e);
        } else {
          float v[1];
          one.unpack(v);
          store_row_vec<1>(p.y, p.y_bf16, to + e, v);
        }
      }
  }
}

cudaError_t launch_moe_dispatch(const DispatchProblem& p, cudaStream_t st) {
  const int way = row_way(p.cols, p.bf16);
  const int64_t words = p.cols / (way == kByElement ? 1 : p.bf16 ? 8 : 4);
  const int threads = row_threads(words, kCopyWords, kCopyThreads);
  const dim3 grid = row_grid(p.tokens, words, static_cast<int64_t>(threads) * kCopyWords);
  return with_rows(p.bf16, way, [&](auto t, auto n) {
    return launch_rows(moe_dispatch_kernel<decltype(t), decltype(n)::value>, grid, threads, 0, st, p);
  });
}

// ------------------------------------------------------------------- dispatch to FP4 codes
// A token's row is encoded once, a block a thread; its codes go to row row_of[t, j], its scales to
// row scale_row_of[t, j] of the grouped layout.  Blocks behind the tokens' write the layout's pads:
// num_experts blocks the rows behind each expert's last, then one block per 128-row block of the
// buffer, which clears it if it lies behind the last expert's.  8192 x 4 x 2880 BF16 to MXFP4: 20 us, 15
// at the copy rate (49 with the block's maximum over lanes and scales stored byte by byte); to NVFP4, whose blocks
// are half as long, 28 us of 15.
constexpr int kCodeThreads = 256;

__device__ __forceinline__ void clear_scale_rows(uint8_t* scales, int64_t atoms, int64_t block, int first_row) {
  for (int64_t i = threadIdx.x; i < atoms * 128; i += blockDim.x) {
    const int w = static_cast<int>(i % 128);  // word w of an atom: 4 scales of row (w % 4) 32 + w / 4
    if ((w & 3) * 32 + (w >> 2) >= first_row)
      reinterpret_cast<uint32_t*>(scales)[(block * atoms + i / 128) * 128 + w] = 0;
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kCodeThreads) moe_dispatch_codes_kernel(const DispatchCodesProblem p, unsigned* status) {
  constexpr int BLOCK = FMT == kCodesMx ? 32 : 16;
  rows_wait_prior();
  rows_allow_dependents();
  const int64_t blocks_k = p.cols / BLOCK, atoms = (blocks_k + 3) / 4;
  const int64_t t = blockIdx.x;
  if (t >= p.tokens) {  // pads
    const int64_t i = t - p.tokens;
    const int upto = i < p.num_experts ? static_cast<int>(i) : p.num_experts;  // experts to count
    __shared__ int s_sum[kCodeThreads / 32];
    int sum = 0;
    for (int e = threadIdx.x; e < upto; e += blockDim.x) sum += (p.offsets[e + 1] - p.offsets[e] + 127) / 128;
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (threadIdx.x % 32 == 0) s_sum[threadIdx.x / 32] = sum;
    __syncthreads();
    int64_t first = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) first += s_sum[w];
    if (i < p.num_experts) {
      const int n = p.offsets[i + 1] - p.offsets[i];
      if (n % 128) clear_scale_rows(p.q.scales, atoms, first + n / 128, n % 128);
    } else if (i - p.num_experts >= first) {
      clear_scale_rows(p.q.scales, atoms, i - p.num_experts, 0);
    }
    return;
  }
  const float g = FMT == kCodesNv ? __ldg(p.q.g) : 1.0f;
  constexpr int V = 16 / sizeof(T), CH = BLOCK / V;  // 16-byte words of a block
  const T* x = static_cast<const T*>(p.x) + t * p.cols;
  bool bad = false;
  for (int64_t k0 = 0; k0 < atoms * 4; k0 += blockDim.x) {  // whole warps: neighbours share a scale word
    const int64_t k = k0 + threadIdx.x;
    const bool ok = k < blocks_k;
    RowVec<T, V> in[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      in[c].zero();
      if (ok) in[c].load(x + k * BLOCK + c * V);
    }
    float v[BLOCK];
#pragma unroll
    for (int c = 0; c < CH; ++c) in[c].unpack(*reinterpret_cast<float(*)[V]>(v + c * V));
    uint32_t packed[BLOCK / 8], sb;
    encode_block<FMT, BLOCK>(g, v, packed, sb, bad);
    // the scales of four blocks, the row's pad columns (0) among them, are one word of an atom
    uint32_t word = (ok ? sb : 0u) << (8 * (k & 3));
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
    for (int j = 0; j < p.topk; ++j) {
      const int64_t s = t * p.topk + j;
      const int32_t row = __ldg(p.row_of + s);
      if (row < 0) continue;
      if (ok) {
        uint8_t* dst = p.q.codes + row * (p.cols / 2) + k * (BLOCK / 2);
        if constexpr (BLOCK == 32) *reinterpret_cast<uint4*>(dst) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
        else *reinterpret_cast<uint2*>(dst) = make_uint2(packed[0], packed[1]);
      }
      if ((k & 3) == 0 && k < atoms * 4)
        *reinterpret_cast<uint32_t*>(p.q.scales + scale_at(__ldg(p.scale_row_of + s), k, atoms)) = word;
    }
  }
  if (bad) atomicOr(status, kStatusNonFinite);
}

cudaError_t launch_moe_dispatch_codes(const DispatchCodesProblem& p, unsigned* status, cudaStream_t st) {
  const int64_t pads = p.num_experts + (p.tokens * p.topk + 127) / 128 + p.num_experts;
  const dim3 grid(static_cast<unsigned>(p.tokens + pads));
  const int threads = row_threads((p.cols / (p.q.fmt == kCodesMx ? 32 : 16) + 3) / 4 * 4, 1, kCodeThreads);
  using BF = __nv_bfloat16;
  if (p.q.fmt == kCodesMx)
    return p.bf16 ? launch_rows(moe_dispatch_codes_kernel<BF, kCodesMx>, grid, threads, 0, st, p, status)
                  : launch_rows(moe_dispatch_codes_kernel<float, kCodesMx>, grid, threads, 0, st, p, status);
  return p.bf16 ? launch_rows(moe_dispatch_codes_kernel<BF, kCodesNv>, grid, threads, 0, st, p, status)
                : launch_rows(moe_dispatch_codes_kernel<float, kCodesNv>, grid, threads, 0, st, p, status);
}

// -------------------------------------------------------------------------------- 8-bit rows
// q = rn(x (1 / s)), s = max|x| / 127 of the row, at least 2^-126 (its reciprocal is finite, so
// that a zero stays zero), 1 for a zero row.  A block per row: its words stay in registers between
// the maximum and the encoding (kI8Words a thread; longer rows are read again).  Bound by the copy
// rate: 16384 x 8 x 4096 BF16 97 us, 94 at the rate; by the barrier between the two for fewer rows,
// 8192 x 4 x 2880 28 us of 22.
constexpr int kI8Words = 4, kI8Threads = 1024;

template <int V>
__device__ __forceinline__ void store_i8(int8_t* dst, const float (&v)[V], float inv) {
  uint32_t w[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    int q[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) q[h] = __float2int_rn(__fmul_rn(v[4 * i + h], inv));
    uint32_t hi;
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, 0;" : "=r"(hi) : "r"(q[3]), "r"(q[2]));
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w[i]) : "r"(q[1]), "r"(q[0]), "r"(hi));
  }
  if constexpr (V == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(dst) = w[0];
}

template <typename T, int V>
__global__ void __launch_bounds__(kI8Threads) quantize_i8_kernel(const I8RowsProblem p, unsigned* status) {
  __shared__ uint32_t s_max[kI8Threads / 32];
  rows_wait_prior();
  rows_allow_dependents();
  const int64_t t = blockIdx.x, words = p.cols / V;
  if (p.valid && t >= __ldg(p.valid)) return;
  const T* x = static_cast<const T*>(p.x) + t * p.cols;
  RowVec<T, V> in[kI8Words];
  uint32_t m = 0;
  auto largest = [&](const RowVec<T, V>& r) {
    float v[V];
    r.unpack(v);
#pragma unroll
    for (int i = 0; i < V; ++i) m = max(m, abs_bits_of(v[i]));
  };
#pragma unroll
  for (int i = 0; i < kI8Words; ++i) {
    in[i].zero();
    const int64_t w = threadIdx.x + i * static_cast<int64_t>(blockDim.x);
    if (w < words) in[i].load(x + w * V);
  }
#pragma unroll
  for (int i = 0; i < kI8Words; ++i) largest(in[i]);
  for (int64_t w = threadIdx.x + kI8Words * static_cast<int64_t>(blockDim.x); w < words; w += blockDim.x) {
    RowVec<T, V> r;
    r.load(x + w * V);
    largest(r);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (blockDim.x > 32) {
    if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = m;
    __syncthreads();
    m = threadIdx.x % 32 < blockDim.x / 32 ? s_max[threadIdx.x % 32] : 0u;
    m = __reduce_max_sync(0xFFFFFFFFu, m);
  }
  if (threadIdx.x == 0 && m >= 0x7F800000u) atomicOr(status, kStatusNonFinite);
  const float s = m ? fmaxf(__fdiv_rn(__uint_as_float(m), 127.0f), 0x1p-126f) : 1.0f;
  const float inv = __frcp_rn(s);
  for (int j = 0; j < p.topk; ++j) {
    const int64_t row = p.row_of ? __ldg(p.row_of + t * p.topk + j) : t;
    if (row < 0) continue;
    if (threadIdx.x == 0) p.scales[row] = s;
    int8_t* q = p.codes + row * p.cols;
#pragma unroll
    for (int i = 0; i < kI8Words; ++i) {
      const int64_t w = threadIdx.x + i * static_cast<int64_t>(blockDim.x);
      float v[V];
      in[i].unpack(v);
      if (w < words) store_i8<V>(q + w * V, v, inv);
    }
    for (int64_t w = threadIdx.x + kI8Words * static_cast<int64_t>(blockDim.x); w < words; w += blockDim.x) {
      RowVec<T, V> r;
      r.load(x + w * V);
      float v[V];
      r.unpack(v);
      store_i8<V>(q + w * V, v, inv);
    }
  }
}

cudaError_t launch_quantize_i8(const I8RowsProblem& p, unsigned* status, cudaStream_t st) {
  const int64_t words = p.cols / (p.bf16 ? 8 : 4);
  // few rows: one word a thread, for the shortest way through a row
  const int threads = row_threads(words, p.rows <= num_sms() ? 1 : kI8Words, kI8Threads);
  const dim3 grid(static_cast<unsigned>(p.rows));
  return p.bf16 ? launch_rows(quantize_i8_kernel<__nv_bfloat16, 8>, grid, threads, 0, st, p, status)
                : launch_rows(quantize_i8_kernel<float, 4>, grid, threads, 0, st, p, status);
}

// ----------------------------------------------------------------------------------- combine
// out[t] = sum_j w[t, j] y[row_of[t, j]] + res[t], the sum in FP32 in the order of j, rounded once.
// R rows' words (2 for up to two choices, else 4) are asked for before the first is needed, 8 in all
// a thread, by four blocks an SM with four rows.  (Three blocks are 1 to 6% slower for FP32 rows by word:
// 4096 x 4 x 2880 41.7 us, with four 39.5.  BF16 ones spill 40 bytes in four blocks' 64 registers, and three
// are up to 7% faster there, 21.8 us for 23.4, but 1% slower for 2000 x 6 x 2048.)  Bound by the copy rate for
// long batches (16384 x 8 x 4096 BF16 164 us, 168 at the rate) and by a block's two dependent loads, row
// numbers and rows, for short ones (4096 x 4 x 2880 23 us of 18).
// By shift a warp asks for 32 words of each row for 31 of the sum, instead of both words by each lane
// (4095 x 2 x 8191 FP32: 107 us so, 82 with 8 words and three blocks, 74 with 4 words and five; with four
// rows the other way round, 4766 x 3 x 3855 FP32 50 and 58 us).  Blocks that stay for many tokens and ask
// for the next one's row numbers ahead were slower: 16384 x 8 x 4096 BF16 177 us.
constexpr int kSumThreads = 256;
template <int WAY, int R>
__host__ __device__ constexpr int sum_words() { return WAY == kByShift && R == 2 ? 2 : 8 / R; }

template <typename T, int WAY, int R>
__global__ void __launch_bounds__(kSumThreads, R == 4 ? 4 : WAY == kByShift ? 5 : 3) moe_combine_kernel(const CombineProblem p) {
  constexpr int V = word_size<T, WAY>(), W = sum_words<WAY, R>(), LANES = WAY == kByShift ? 31 : 32;
  rows_wait_prior();
  rows_allow_dependents();
  const int64_t t = blockIdx.x, to = t * p.cols;
  const T* y = static_cast<const T*>(p.y);
  const RowSpan<V, WAY> span(to, p.cols);
  const int round = blockDim.x / 32 * LANES, lane = threadIdx.x % 32;
  const int w0 = blockIdx.y * round * W + threadIdx.x / 32 * LANES + lane;
  const int limit = span.words + (WAY == kByShift);  // the word behind the last is asked for too
  // by shift: one of the single elements for each of the first block's first threads
  const bool extra = WAY == kByShift && blockIdx.y == 0 && static_cast<int>(threadIdx.x) < span.singles();
  const int single = extra ? span.single(threadIdx.x) : 0;
  float sum[W][V] = {}, sum1[1] = {0.0f};
  for (int j0 = 0; j0 < p.topk; j0 += R) {
    RowVec<T, V> in[R][W];
    RowVec<T, 1> in1[R];
    float weight[R];
    bool on[R];
    int off[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t s = t * p.topk + j0 + j;
      const int32_t row = j0 + j < p.topk ? __ldg(p.row_of + s) : -1;
      on[j] = row >= 0;
      off[j] = WAY == kByShift ? static_cast<int>(row * p.cols + span.first) & (V - 1) : 0;
      in1[j].zero();
      if (extra && on[j]) in1[j].load(y + row * p.cols + single);
      weight[j] = on[j] && p.weights ? __ldg(p.weights + s) : 1.0f;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int w = w0 + i * round;
        if (!on[j] || w >= limit) continue;
        if constexpr (WAY == kByShift) in[j][i].hold(y, row * p.cols + span.first + w * V);
        else in[j][i].load(y + row * p.cols + w * V);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (!on[j]) continue;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (WAY == kByShift) in[j][i].shift(off[j]);
        float v[V];
        in[j][i].unpack(v);
#pragma unroll
        for (int k = 0; k < V; ++k) sum[i][k] = fmaf(weight[j], v[k], sum[i][k]);
      }
      if constexpr (WAY == kByShift) {
        float v[1];
        in1[j].unpack(v);
        sum1[0] = fmaf(weight[j], v[0], sum1[0]);
      }
    }
  }
  if (extra) {
    float r[1];
    if (p.res) {
      load_row_any<1>(p.res, p.res_bf16, to + single, r);
      sum1[0] += r[0];
    }
    store_row_vec<1>(p.out, p.out_bf16, to + single, sum1);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int w = w0 + i * round;
    if (w >= span.words || lane >= LANES) continue;
    const int64_t at = to + span.first + w * V;
    if (p.res) {
      float r[V];
      load_row_any<V>(p.res, p.res_bf16, at, r);
#pragma unroll
      for (int k = 0; k < V; ++k) sum[i][k] += r[k];
    }
    store_row_vec<V>(p.out, p.out_bf16, at, sum[i]);
  }
}

template <int R>
static cudaError_t combine_rows(const CombineProblem& p, cudaStream_t st) {
  const int way = row_way(p.cols, p.bf16);
  const int64_t words = p.cols / (way == kByElement ? 1 : p.bf16 ? 8 : 4);
  const int each = way == kByShift ? sum_words<kByShift, R>() : sum_words<kByWord, R>();
  const int threads = row_threads(words, each, kSumThreads);
  const dim3 grid = row_grid(p.tokens, words, static_cast<int64_t>(way == kByShift ? threads / 32 * 31 : threads) * each);
  return with_rows(p.bf16, way, [&](auto t, auto n) {
    return launch_rows(moe_combine_kernel<decltype(t), decltype(n)::value, R>, grid, threads, 0, st, p);
  });
}

cudaError_t launch_moe_combine(const CombineProblem& p, cudaStream_t st) {
  return p.topk <= 2 ? combine_rows<2>(p, st) : combine_rows<4>(p, st);
}

// ------------------------------------------------------------------------- its backward pass
// dy[row_of[t, j]] = w[t, j] dout[t], dw[t, j] = <dout[t], y[row_of[t, j]]>: a block per token, so
// that dout is read once and each dot product is summed in one place, in a fixed order.
// Rows are taken R at a time (as many as there are choices, up to 8), and all their words of a column
// are asked for before the first is needed; with R fixed at 8 and word after word it took 210 us
// where it takes 68 (8192 tokens, 4 choices, 2880 BF16 columns; 65 at the copy rate, its bound).
constexpr int kGradThreads = 256;

template <typename T, int WAY, int R>
__global__ void __launch_bounds__(kGradThreads, R == 8 ? 3 : 4) moe_combine_grad_kernel(const CombineGradProblem p) {
  constexpr int V = word_size<T, WAY>();
  __shared__ float s_dot[kGradThreads / 32][R];
  rows_wait_prior();
  rows_allow_dependents();
  const int64_t t = blockIdx.x;
  const T* dout = static_cast<const T*>(p.dout);
  const T* y = static_cast<const T*>(p.y);
  const bool dots = p.dweights != nullptr;
  for (int j0 = 0; j0 < p.topk; j0 += R) {
    int32_t row[R];
    float weight[R], dot[R];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int64_t s = t * p.topk + j0 + j;
      row[j] = j0 + j < p.topk ? __ldg(p.row_of + s) : -1;
      weight[j] = row[j] >= 0 && p.weights ? __ldg(p.weights + s) : 1.0f;
      dot[j] = 0.0f;
    }
    if constexpr (WAY == kByShift) {
      // Words at each row's own offset, so that every row takes dout's two words around them anew; all
      // loads of a round are asked for before the first is needed.  They pass L1 by: through it 8192 x 4 x
      // 2881 BF16 took 103 us for 93.5, 4766 x 3 x 3855 FP32 104 for 99, 2000 x 6 x 2049 BF16 27.2 for 26.6; only
      // 4095 x 2 x 8191 FP32 (138.8 for 139.8) and 300 x 4 x 2050 BF16 (6.2 for 6.7) were faster.
      const int64_t from = t * p.cols;
      int64_t at[R];
      int first[R], words[R];
      int most = 0;
#pragma unroll
      for (int j = 0; j < R; ++j) {
        at[j] = row[j] * p.cols;
        const RowSpan<V, WAY> span(at[j], p.cols);
        first[j] = span.first;
        words[j] = row[j] >= 0 ? span.words : 0;
        most = max(most, words[j]);
      }
      for (int w = threadIdx.x; w < most; w += blockDim.x) {
        RowVec<T, V> a[R], b[R], yr[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
          a[j].zero();
          b[j].zero();
          yr[j].zero();
          if (w >= words[j]) continue;
          const int e = first[j] + w * V;
          a[j].hold(dout, from + e);
          b[j].hold(dout, from + e + V);
          if (dots) yr[j].load(y + at[j] + e);
        }
#pragma unroll
        for (int j = 0; j < R; ++j) {
          a[j].join(b[j], from + first[j]);
          float d[V], v[V];
          a[j].unpack(d);
          yr[j].unpack(v);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            dot[j] = fmaf(d[k], v[k], dot[j]);
            v[k] = weight[j] * d[k];
          }
          if (p.dy && w < words[j]) store_row_vec<V>(p.dy, p.dy_bf16, at[j] + first[j] + w * V, v);
        }
      }
#pragma unroll
      for (int j = 0; j < R; ++j) {
        if (row[j] < 0) continue;
        const RowSpan<V, WAY> span(at[j], p.cols);
        for (int i = threadIdx.x; i < span.singles(); i += blockDim.x) {
          const int e = span.single(i);
          RowVec<T, 1> in, yr;
          in.load(dout + from + e);
          yr.zero();
          if (dots) yr.load(y + at[j] + e);
          float d[1], v[1];
          in.unpack(d);
          yr.unpack(v);
          dot[j] = fmaf(d[0], v[0], dot[j]);
          v[0] = weight[j] * d[0];
          if (p.dy) store_row_vec<1>(p.dy, p.dy_bf16, at[j] + e, v);
        }
      }
    } else {
      for (int w = threadIdx.x; w < static_cast<int>(p.cols) / V; w += blockDim.x) {
        RowVec<T, V> in, yr[R];
        in.load(dout + t * p.cols + w * V);
#pragma unroll
        for (int j = 0; j < R; ++j) {
          yr[j].zero();
          if (dots && row[j] >= 0) yr[j].load(y + row[j] * p.cols + w * V);
        }
        float d[V];
        in.unpack(d);
#pragma unroll
        for (int j = 0; j < R; ++j) {
          float v[V];
          yr[j].unpack(v);
#pragma unroll
          for (int k = 0; k < V; ++k) dot[j] = fmaf(d[k], v[k], dot[j]);
          if (!p.dy || row[j] < 0) continue;
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] = weight[j] * d[k];
          store_row_vec<V>(p.dy, p.dy_bf16, row[j] * p.cols + w * V, v);
        }
      }
    }
    if (dots) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float v = warp_sum(dot[j]);
        if (threadIdx.x % 32 == 0) s_dot[threadIdx.x / 32][j] = v;
      }
      __syncthreads();
      if (threadIdx.x < R && j0 + static_cast<int>(threadIdx.x) < p.topk) {
        // (a slot without an expert: 0, not 0 times what dout may hold)
        float v = 0.0f;
        for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) v += s_dot[w][threadIdx.x];
        const int64_t s = t * p.topk + j0 + threadIdx.x;
        p.dweights[s] = __ldg(p.row_of + s) >= 0 ? v : 0.0f;
      }
      __syncthreads();
    }
  }
}

template <int R>
static cudaError_t combine_grad_rows(const CombineGradProblem& p, int way, cudaStream_t st) {
  const int threads = row_threads(p.cols / (way == kByElement ? 1 : p.bf16 ? 8 : 4), 2, kGradThreads);
  const dim3 grid(static_cast<unsigned>(p.tokens));
  return with_rows(p.bf16, way, [&](auto t, auto n) {
    // by shift a row takes three times the registers: eight at a time would spill
    constexpr int kWay = decltype(n)::value, kRows = kWay == kByShift && R == 8 ? 4 : R;
    return launch_rows(moe_combine_grad_kernel<decltype(t), kWay, kRows>, grid, threads, 0, st, p);
  });
}

cudaError_t launch_moe_combine_grad(const CombineGradProblem& p, cudaStream_t st) {
  const int way = row_way(p.cols, p.bf16);
  if (p.topk <= 2) return combine_grad_rows<2>(p, way, st);
  return p.topk <= 4 ? combine_grad_rows<4>(p, way, st) : combine_grad_rows<8>(p, way, st);
}

}  // namespace fp4
