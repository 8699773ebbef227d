// fp4_moe.h -- declarations of the operators that bring tokens to their experts and back, and of
// the products in 8-bit integers, shared by their translation units and the API.
#pragma once

#include "fp4_ops.h"

namespace fp4 {

size_t moe_sort_workspace_bytes(int64_t slots, int E);
cudaError_t launch_moe_sort(const void* ids, int id_bytes, int64_t slots, int E, int32_t* offsets, int32_t* row_of,
                            int32_t* scale_row_of, void* ws, cudaStream_t st);

struct DispatchProblem {
  const void* x;
  int bf16;
  int64_t tokens, cols;
  int topk;
  const int32_t* row_of;
  void* y;
  int y_bf16;
};
cudaError_t launch_moe_dispatch(const DispatchProblem& p, cudaStream_t st);

struct DispatchCodesProblem {
  const void* x;
  int bf16;
  int64_t tokens, cols;
  int topk, num_experts;
  const int32_t *row_of, *scale_row_of, *offsets;
  CodesOut q;
};
cudaError_t launch_moe_dispatch_codes(const DispatchCodesProblem& p, unsigned* status, cudaStream_t st);

// 8-bit rows with a scale each, in place (row_of null, topk 1; with `valid` only that many of them)
// or in the experts' order.
struct I8RowsProblem {
  const void* x;
  int bf16;
  int64_t rows, cols;
  int topk;
  const int32_t* row_of;
  const int32_t* valid;
  int8_t* codes;
  float* scales;
};
cudaError_t launch_quantize_i8(const I8RowsProblem& p, unsigned* status, cudaStream_t st);

struct CombineProblem {
  const void* y;
  int bf16;
  const int32_t* row_of;
  const float* weights;  // null: all 1
  int64_t tokens, cols;
  int topk;
  const void* res;
  int res_bf16;
  void* out;
  int out_bf16;
};
cudaError_t launch_moe_combine(const CombineProblem& p, cudaStream_t st);

struct CombineGradProblem {
  const void *dout, *y;
  int bf16;
  const int32_t* row_of;
  const float* weights;
  int64_t tokens, cols;
  int topk;
  void* dy;
  int dy_bf16;
  float* dweights;
};
cudaError_t launch_moe_combine_grad(const CombineGradProblem& p, cudaStream_t st);

// D[m, n] = act(sA[m] sB[n] sum_k A[m, k] B[n, k] + bias[n]) in 8-bit integers; by experts: rows
// [offsets[e], offsets[e + 1]) of A with weights, scales and bias number e.
struct I8Problem {
  const int8_t *A, *B;
  const float *sA, *sB;
  int64_t M, N, K;
  const float* bias;
  int act;
  void* D;
  int out_bf16;
  void* ws;
  size_t ws_bytes;
  int weights_ready;
  int num_groups;  // 0: one problem
  const int32_t* offsets;
};
size_t i8_workspace_bytes(int64_t M, int64_t N, int64_t K, int num_groups);
int launch_gemm_i8(const I8Problem& p, unsigned* status, cudaStream_t st, const char** why, cudaError_t* err);

}  // namespace fp4
