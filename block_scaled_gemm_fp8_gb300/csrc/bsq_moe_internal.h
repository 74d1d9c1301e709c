// bsq_moe_internal.h -- launch descriptions of the operators around a mixture layer's products
// (router, tokens to their experts' rows and back, 4-bit products of few rows), shared between
// the host entry points (bsq_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsq {

constexpr int kMaxSlots = 32;   // slots a token (k): one lane of a warp each

// bsq_route (ids, weights written), or with grad_logits bsq_route_backward (ids read, grad_weights).
struct RouteArgs {
  int dtype;               // bsq_dtype of logits and grad_logits
  const void* logits;      // [T][E]
  int64_t T;
  int E, k, gate;          // gate: bsq_gate
  bool renormalize;
  const float* bias;       // f32[E] or null (forward)
  float factor;
  int32_t* ids;            // [T][k]
  float* weights;          // f32[T][k] (forward)
  const float* grad_weights;
  void* grad_logits;       // [T][E] (backward)
  cudaStream_t stream;
};
int launch_route(const RouteArgs& a, const char** msg);

struct SortArgs {
  const int32_t* ids;      // [n]
  int64_t n;
  int E;
  int32_t* offsets;        // [E]
  int32_t* rows;           // [n]
  int32_t* slots;          // [n] or null
  cudaStream_t stream;
};
int launch_sort_experts(const SortArgs& a, const char** msg);

// bsq_dispatch and bsq_combine_backward (y, grad_weights): a token's columns to its rows;
// bsq_combine: its rows' sum to `out`.
struct TokenArgs {
  const void* x;           // bf16 [T][cols]: tokens, or the gradient of the combined tokens (combine: unused)
  const void* y;           // bf16 [S][cols]: rows to combine, or to multiply x with
  int64_t T, S, cols;
  const int32_t* rows;     // [T][k]
  int k;
  const float* weights;    // f32[T][k] or null for 1
  void* out;               // bf16 [S][cols] or null (combine: [T][cols])
  void* codes;             // u8 [S][cols] or null
  float* scale;            // f32 [S][ceil(cols / 128)] with codes
  float* grad_weights;     // f32[T][k] or null
  int num_sms;
  cudaStream_t stream;
};
int launch_dispatch(const TokenArgs& a, const char** msg);
int launch_combine(const TokenArgs& a, const char** msg);
int launch_combine_backward(const TokenArgs& a, const char** msg);

// A dense product of more rows takes bsq_linear_forward's 256-row tile kernel (14336 x 5120 MXFP4: 64 rows
// 38 us in the few-rows kernel's two passes, 65 there 42; NVFP4 39.5 and 46).
constexpr int kFp4Rows = 64;

struct Fp4Args {
  int fmt;                 // BSQ_MXFP4 or BSQ_NVFP4
  const void* x;           // bf16 [S][K]
  const void* w;           // codes [E][N][K / 2]
  const void* w_scale;     // [E][N][K / 32] or [E][N][K / 16]
  const float* tensor_scale;   // NVFP4: f32[E]
  int64_t S, N, K, E;
  const int32_t* offsets;  // device cumulative ends [E]; null: one group of S rows
  void* y;                 // bf16 [S][N]
  int32_t* err;
  int num_sms;
  cudaStream_t stream;
};
int launch_fp4_smallm(const Fp4Args& a, const char** msg);

}  // namespace bsq
