// Internal interface between the C-ABI layer of the 8-bit operators (w8a8_api.cpp)
// and their kernels.  Arguments that reach the launchers are validated: required
// pointers non-NULL and aligned, extents positive and within their limits,
// K % 16 == 0.  A grid that the hardware cannot take is refused as
// hipErrorInvalidConfiguration.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w8a8.h"

namespace w4a16 {

constexpr int kBlock8 = W8A8_BLOCK;

inline int blocks8(int n) { return (n + kBlock8 - 1) / kBlock8; }

// rows to e4m3 (w8a8_rows.hip)
struct Rows8 {
  const void *X;
  const int32_t *num_rows;  // device word or NULL
  uint8_t *codes;
  float *scales;
  int M, K, dtype;
  bool swiglu;
};
hipError_t launch_rows8(const Rows8 &p, hipStream_t stream);

// residual addition, norm, rows to e4m3 (w8a8_norm.hip); NULL outputs are not made
struct Norm8 {
  const void *X, *residual, *weight;
  void *H, *Y;
  uint8_t *codes;
  float *scales;
  int M, K, dtype;
  bool weight_f32;  // weight in fp32 (else in dtype)
  float eps;
};
hipError_t launch_norm8(const Norm8 &p, hipStream_t stream);

// Y[r] = X[token_index[r]] . W_e^T; without expert_offsets one expert owns all rows,
// without token_index slot r reads row r
struct Gemm8 {
  const uint8_t *X;
  const float *xs;
  const int32_t *token_index, *expert_offsets;
  const uint8_t *W;
  const float *ws;
  void *Y;
  int rows_x, R, E, N, K, dtype;
};
// W8A8_KERNEL_*: the kernel for R rows of one expert, or R slots over E of them
int gemm8_kernel(long R, long E, bool grouped);
hipError_t launch_gemm8(const Gemm8 &p, hipStream_t stream);
hipError_t launch_gemm8_skinny(const Gemm8 &p, hipStream_t stream);
hipError_t launch_gemm8_tile(const Gemm8 &p, hipStream_t stream);

}  // namespace w4a16
