// bsq_fp8_internal.h -- launch descriptions of the E4M3 operators and AdamW, shared between the
// host entry points (bsq_api.cu) and their kernels.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace bsq {

// A product of E4M3 operands on their own codes (bsq_fp8.cu, bsq_fp8_smallm.cu).
struct Fp8Args {
  bool dgrad;              // false: y[S][N] = X[S][K] W^T; true: gx[S][K] = G[S][N] W
  const void* x;           // E4M3 codes [S][K] (dgrad: [S][N])
  const float* x_scale;    // [S][ceil(columns / 128)]
  const void* w;           // E4M3 codes [E][N][K]
  const float* w_scale;    // [E][ceil(N / 128)][ceil(K / 128)]
  int64_t S, N, K, E;
  const int32_t* offsets;  // device cumulative ends [E]; null: one group of S rows
  void* y;                 // bf16
  int32_t* err;
  int num_sms;
  cudaStream_t stream;
};
int launch_fp8(const Fp8Args& a, const char** msg);
// The forward for a few token rows.
int launch_fp8_smallm(const Fp8Args& a, const char** msg);
// Whether the forward of these sizes takes the few-rows kernel (the offsets are the device's).
bool fp8_takes_smallm(const Fp8Args& a);

struct QuantE4m3Args {
  int dtype;               // bsq_dtype of x
  const void* x;           // [batch][rows][cols]
  int64_t batch, rows, cols;
  int block_rows;          // 1 or 128
  void* codes;
  float* scale;
  cudaStream_t stream;
};
int launch_quantize_e4m3(const QuantE4m3Args& a, const char** msg);

// One AdamW step over `count` tensors (bsq_adamw.cu); the checked arguments of bsq_adamw.
struct AdamwArgs {
  const void* tensors;     // host bsq_adamw_tensor[count]
  int count;
  int grad_dtype, state_bits;
  int64_t step;
  double lr, beta1, beta2, eps;
  const float* grad_scale;
  uint32_t seed;
  cudaStream_t stream;
};
int launch_adamw(const AdamwArgs& a, const char** msg);

}  // namespace bsq
