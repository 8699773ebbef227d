// fp4_ops.h -- declarations of the operators around the FP4 GEMM (layer norm, the
// activation's backward pass, the gated GEMM) shared by their translation units and the API.
#pragma once

#include "fp4_internal.h"

namespace fp4 {

// Codes of an activation function (fp4_act in fp4.h has the same values).
enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };

// What follows the product:
//   kEpiPlain  scale, bias, ReLU, store (and the NVFP4 copy): the accumulator's values go to
//              memory as they are read
//   kEpiFull   any activation, a residual, the pre-activation's copy
//   kEpiGated  two products at once: a tile's first half of columns are gate columns
//              (operand B), the second half the up columns (operand B2) of the same outputs,
//              H = act(G) U
// In the general kernel the last two first empty the accumulator into registers and hand it
// back, so that their longer arithmetic and their loads overlap the next tile's MMAs.
//   kEpiFullWhole, kEpiGatedWhole  the same where all columns come in whole sixteens, rows start
//              at 32-byte sectors and K is not split (the general kernels carry the other cases'
//              code: 32 x 512 x 2880 x 2880 gated experts 223 us against 194)
enum { kEpiPlain = 0, kEpiFull = 1, kEpiGated = 2, kEpiFullWhole = 3, kEpiGatedWhole = 4 };

// Where a row kernel writes a block-scaled copy of its result (fmt: kCodesNone / Nv / Mx).
struct CodesOut {
  int fmt;
  uint8_t *codes, *scales;
  const float* g;
};

struct LayerNormProblem {
  const void* x;
  int bf16;
  int64_t rows, cols;
  const float *weight, *bias;
  float eps;
  void* y;
  int y_bf16;
  float *mean, *rstd;
  CodesOut q;
  float* amax_out;  // zeroed by the entry point
};
cudaError_t launch_layernorm(const LayerNormProblem& p, unsigned* status, cudaStream_t st);

struct LayerNormGradProblem {
  const void *dy, *x;
  int bf16;
  int64_t rows, cols;
  const float *weight, *mean, *rstd;
  const void* dres;
  void* dx;
  int dx_bf16;
  float *dweight, *dbias;
  float* ws;
};
size_t layernorm_grad_workspace_bytes(int64_t rows, int64_t cols);
cudaError_t launch_layernorm_grad(const LayerNormGradProblem& p, unsigned* status, cudaStream_t st);

struct ActGradProblem {
  const void *dh, *g, *u;  // u null: a plain activation
  int bf16;
  int64_t rows, cols;
  int act;
  void* dz;
  int dz_bf16;
  float* dbias;
  CodesOut q;
  float* amax_out;
  float* ws;
};
size_t act_grad_workspace_bytes(int64_t rows, int64_t cols, int gated);
cudaError_t launch_act_grad(const ActGradProblem& p, unsigned* status, cudaStream_t st);

// out0[c] = sum_p part[p][c] for c < n0, out1[c - n0] for the rest of the `width` columns, in
// the order of p; either output may be null.  Clears part.
cudaError_t launch_column_sums(float* part, int parts, int64_t width, int64_t n0, float* out0, float* out1,
                               cudaStream_t st);

// GemmProblem with the long epilogue's operands (full null: the plain epilogue).
struct GemmFull {
  const void* res;  // [M, N] added after the activation, or null
  int res_bf16;
  void* pre;        // the pre-activation [M, N] in the output type, or null
};
struct GemmProblemFull : GemmProblem {
  const GemmFull* full;
};
size_t gemm_full_workspace_bytes(int64_t M, int64_t N, int64_t K, int mx, bool fp4_out);
int launch_gemm_full(const GemmProblemFull& g, unsigned* status, cudaStream_t st, const char** why, cudaError_t* err);

// The decode kernel with the long epilogue, or with a second weight (a gated product: W and
// bias are the gate's, W2 and bias2 the up projection's).
struct DecodeExtra {
  const uint8_t *W2, *sW2;
  const float *gW2, *bias2;
  const void* res;
  int res_bf16;
  void *pre, *pre2;
};
size_t decode_gated_workspace_bytes(int64_t M, int64_t F);
bool gated_decode_eligible(int64_t M, int64_t F, int64_t K);  // whether a gated product takes it
int launch_decode_extra(const DecodeProblem& q, const DecodeExtra& x, unsigned* status, cudaStream_t st,
                        const char** why, cudaError_t* err);

struct GatedProblem {
  int mx;
  const uint8_t *A, *sA;
  const float* gA;
  const uint8_t *Wg, *sWg;
  const float* gWg;
  const uint8_t *Wu, *sWu;
  const float* gWu;
  int64_t M, F, K;
  const float *bias_g, *bias_u;
  int act;
  void *H, *G, *U;
  int out_bf16;
  uint8_t *q_codes, *q_scales;
  const float* q_g;
  float* amax_out;
  void* ws;
  size_t ws_bytes;
  int weights_ready;
  int num_groups;  // 0: one problem
  const int32_t* offsets;
};
size_t gated_workspace_bytes(int64_t M, int64_t F, int64_t K, int mx, bool rows_in_place);
int launch_gated(const GatedProblem& g, unsigned* status, cudaStream_t st, const char** why, cudaError_t* err);

}  // namespace fp4
