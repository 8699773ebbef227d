// fp4_gated.cu -- the gated product H = act(A Wg^T + bg) * (A Wu^T + bu) in one launch, dense
// and grouped by experts.
//
// A tile computes 128 output columns of both products: its 256 MMA columns are 128 gate rows
// and 128 up rows of the weights (two operands, two tensor maps), so that the accumulator of
// one thread's row holds gate and up sums of the same outputs and the product never leaves
// the SM.  On CTA pairs the leader loads the tile's gate rows and the other CTA its up rows.
#include "fp4_gemm_host.h"

namespace fp4 {

// A tile is 128 (a CTA pair: 256) rows by 128 output columns.
static Plan gated_plan(int64_t M, int64_t F, int64_t K, int groups, int mx) {
  Plan pl{};
  pl.num_kb = static_cast<int>((K + 255) / 256);
  pl.BN = 256;
  pl.ACC = 1;
  pl.Mk = M;
  pl.Nk = F;
  pl.tiles_n = static_cast<int>((F + 127) / 128);
  if (groups) {
    pl.mode = kModeGrouped;
    // CTA pairs for many rows per expert, as the plain grouped product's; with MXFP4's half as
    // many scale copies single CTAs are faster throughout (us, pairs / singles: 32 experts x 2048
    // rows x 2880 x 2880 732 / 695, 8 x 4096 x 4096 x 4096 589 / 549, 4 x 2048 x 8192 x 8192 568 / 507)
    pl.pair = !mx && M >= 1280 * static_cast<int64_t>(groups);
    return pl;
  }
  pl.tiles_m = static_cast<int>((M + 127) / 128);
  const int64_t tiles = static_cast<int64_t>(pl.tiles_m) * pl.tiles_n;
  const int sms = num_sms();
  // Fewer tiles than SMs: a tile's K steps, about 0.5 us each, can be split over CTAs.  What that
  // costs (partial sums of 16 bytes a thread meet in L2, then are read back) grows with the rows
  // and tiles; in us, from: F = 256, K = 8192: 33 rows 14.9 split / 20.1 whole, 128 rows 26.9 /
  // 21.5; F = 2880, K = 28672: 128 rows 50 / 76, 512 rows 83 / 76; F = 2880, K = 2880: 33 rows
  // 23.6 / 11.5, 512 rows 45.6 / 13.2.
  const double saved = 0.5 * static_cast<double>(pl.num_kb - (tiles * pl.num_kb + sms - 1) / sms);
  const double cost = 8.0 + 0.09 * static_cast<double>(std::min<int64_t>(M, 128)) + 0.05 * static_cast<double>(tiles);
  if (tiles < sms && saved > cost) {
    pl.mode = kModeStreamK;
    pl.units = tiles * pl.num_kb;
    pl.ws_bytes = (static_cast<size_t>(2 * M * ((F + 3) / 4 * 4)) * 4 + 255) / 256 * 256 + (static_cast<size_t>(tiles) * 4 + 255) / 256 * 256;
    return pl;
  }
  pl.mode = kModeTile;
  pl.units = tiles;
  // (NVFP4 4096 x 8192 x 8192: pairs 251 us, singles 293; MXFP4 245 both)
  if (M >= 256 && tiles >= sms) {
    pl.pair = true;
    pl.tiles_m = static_cast<int>((M + 255) / 256);
    pl.units = static_cast<int64_t>(pl.tiles_m) * pl.tiles_n;
  }
  return pl;
}

// Up to 16 rows the decode kernel streams the weights faster than whole tiles with 112 rows
// empty; from 17 rows on its 32-wide MMAs and partial sums cost more than they save (us,
// quantized operands, decode / tiles: F = 28672, K = 8192: 1 row 48.5 / 69.5, 16 rows 52.7 / 69.8, 32
// rows 63.6 / 58.5; F = K = 2880: 16 rows 12.4 / 11.9, 32 rows 20.1 / 11.8).
bool gated_decode_eligible(int64_t M, int64_t F, int64_t K) { return M <= 16 && decode_eligible(M, F, K); }

size_t gated_workspace_bytes(int64_t M, int64_t F, int64_t K, int mx, bool rows_in_place) {
  if (!mx && !rows_in_place && gated_decode_eligible(M, F, K)) return decode_gated_workspace_bytes(M, F);
  return gated_plan(M, F, K, 0, mx).ws_bytes;
}

template <bool MX>
static cudaError_t dispatch_gated(const Plan& pl, const GemmMaps& tm, const GemmArgs& a, cudaStream_t st) {
  if (pl.mode != kModeStreamK && a.sectors && a.Nk % 16 == 0)
    return pl.pair ? run<256, MX, 1, true, false, kEpiGatedWhole>(tm, a, pl.units, st)
                   : run<256, MX, 1, false, false, kEpiGatedWhole>(tm, a, pl.units, st);
  return pl.pair ? run<256, MX, 1, true, false, kEpiGated>(tm, a, pl.units, st)
                 : run<256, MX, 1, false, false, kEpiGated>(tm, a, pl.units, st);
}

int launch_gated(const GatedProblem& g, unsigned* status, cudaStream_t st, const char** why, cudaError_t* err) {
  const int grouped = g.num_groups > 0;
  if (!grouped && !g.mx && !g.q_codes && !g.amax_out && gated_decode_eligible(g.M, g.F, g.K)) {
    DecodeProblem q{};
    q.W = g.Wg;
    q.sW = g.sWg;
    q.gW = g.gWg;
    q.Xq = g.A;
    q.Xs = g.sA;
    q.gX = g.gA;
    q.M = g.M;
    q.N = g.F;
    q.K = g.K;
    q.D = g.H;
    q.out_bf16 = g.out_bf16;
    q.ws = g.ws;
    q.ws_bytes = g.ws_bytes;
    q.weights_ready = g.weights_ready;
    q.bias = g.bias_g;
    q.act = g.act;
    DecodeExtra x{};
    x.W2 = g.Wu;
    x.sW2 = g.sWu;
    x.gW2 = g.gWu;
    x.bias2 = g.bias_u;
    x.pre = g.G;
    x.pre2 = g.U;
    return launch_decode_extra(q, x, status, st, why, err);
  }
  const Plan pl = gated_plan(g.M, g.F, g.K, g.num_groups, g.mx);
  if (g.ws_bytes < pl.ws_bytes || (pl.ws_bytes && !g.ws)) {
    *why = "workspace too small (see fp4_gemm_gated_workspace_size)";
    return 1;
  }
  const int64_t atoms_k = (g.K / (g.mx ? 32 : 16) + 3) / 4;
  const int64_t f_blocks = (g.F + 127) / 128;
  const int64_t experts = grouped ? g.num_groups : 1;
  const uint64_t rows_w = static_cast<uint64_t>(experts * g.F), kb = static_cast<uint64_t>(g.K / 2);
  GemmMaps tm;
  if (!make_tensor_map_u8(&tm.a, g.A, kb, static_cast<uint64_t>(g.M), 128) ||
      !make_tensor_map_u8(&tm.b, g.Wg, kb, rows_w, 128) || !make_tensor_map_u8(&tm.b2, g.Wu, kb, rows_w, 128)) {
    *why = "cuTensorMapEncodeTiled failed (alignment or driver)";
    return 1;
  }
  tm.sfa = tm.sfb = tm.sfb2 = tm.a;
  if (pl.pair) {
    const uint32_t box_rows = (g.mx ? 2u : 4u) * 512u / 256u;  // one stage's atoms of a 128-row block
    const int64_t sfa_blocks = (g.M + 127) / 128 + (grouped ? g.num_groups : 0);
    const uint64_t w_bytes = static_cast<uint64_t>(experts * f_blocks * atoms_k) * 512;
    if (!make_sf_map(&tm.sfa, g.sA, static_cast<uint64_t>(sfa_blocks * atoms_k) * 512, box_rows) ||
        !make_sf_map(&tm.sfb, g.sWg, w_bytes, box_rows) || !make_sf_map(&tm.sfb2, g.sWu, w_bytes, box_rows)) {
      *why = "cuTensorMapEncodeTiled failed for the scale factors (alignment or driver)";
      return 1;
    }
  }
  GemmArgs a{};
  a.sfa = g.sA;
  a.sfb = g.sWg;
  a.sfb2 = g.sWu;
  a.sfa_rb_bytes = a.sfb_rb_bytes = atoms_k * 512;
  a.sf_atoms_k = static_cast<int>(atoms_k);
  a.sfb_rbs = static_cast<int>(f_blocks);
  a.ga = g.gA;
  a.gb = g.gWg;
  a.gb2 = g.gWu;
  a.Mk = static_cast<int>(g.M);
  a.Nk = static_cast<int>(g.F);
  a.K = static_cast<int>(g.K);
  a.num_kb = pl.num_kb;
  a.out = g.H;
  a.out_bf16 = g.out_bf16;
  a.indep = g.weights_ready ? 2 : 0;
  a.ldo = g.F;
  const int esz = g.out_bf16 ? 2 : 4;
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  a.vec_store = (g.F * esz) % 16 == 0 && al(g.H) && al(g.G) && al(g.U);
  auto al32 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; };
  a.sectors = (g.F * esz) % 32 == 0 && al32(g.H) && al32(g.G) && al32(g.U);
  a.mode = pl.mode;
  a.tiles_m = pl.tiles_m;
  a.tiles_n = pl.tiles_n;
  a.group_m = 16;
  a.total_units = pl.units;
  a.status = status;
  a.bias = g.bias_g;
  a.bias2 = g.bias_u;
  a.bias_any = g.bias_g || g.bias_u;
  a.act = g.act;
  a.pre = g.G;
  a.pre2 = g.U;
  a.q_codes = g.q_codes;
  a.q_scales = g.q_scales;
  a.q_g = g.q_g;
  a.q_atoms = (g.F / 16 + 3) / 4;
  a.amax_out = reinterpret_cast<unsigned*>(g.amax_out);
  if (pl.mode == kModeStreamK) {
    a.ws = static_cast<float*>(g.ws);
    a.ws_ld = static_cast<int>((g.F + 3) / 4 * 4);
    a.tile_cnt = reinterpret_cast<int*>(static_cast<uint8_t*>(g.ws) + (static_cast<size_t>(2 * g.M * a.ws_ld) * 4 + 255) / 256 * 256);
  }
  if (grouped) {
    a.num_groups = g.num_groups;
    a.offsets = g.offsets;
    a.b_rows_per_group = static_cast<int>(g.F);
    a.sfb_group_bytes = f_blocks * atoms_k * 512;
    a.bias_group = g.F;
  }
  const cudaError_t e = g.mx ? dispatch_gated<true>(pl, tm, a, st) : dispatch_gated<false>(pl, tm, a, st);
  if (e != cudaSuccess) {
    *err = e;
    return 2;
  }
  return 0;
}

}  // namespace fp4
