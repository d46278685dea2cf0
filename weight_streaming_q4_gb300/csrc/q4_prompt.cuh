// What the operators of a prompt's layer beside its attention share: their
// arguments and launchers (include/q4.h; sm_103a).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "q4.h"
#include "q4_paged.cuh"

namespace q4 {

// Rows of the caller's: binary16 or fp32, ld values apart (null: none).
struct RowsIn {
  const void* p;
  int64_t ld;
  int f32;
};
struct RowsOut {
  void* p;
  int64_t ld;
  int f32;
};

// ------------------------------------------------------------------ products (q4_gemm.cu)

struct GemmArgs {
  const uint8_t* w[2];      // Q4_0 [n][k / 32]; the second one of a gated product, or null
  const __half* x;
  int64_t x_ld;
  int n, k, rows;
  const float* bias[2];
  int act;
  float scale;
  RowsIn residual;
  __half* y;
  int64_t y_ld;
};
// What the kernels need to know of the device they run on.
struct PromptDevice {
  int sms;
  int clusters[4];          // of 2, 4, 8 and 16 CTAs of the product's kernel that run at once
};
cudaError_t gemm_prepare(PromptDevice* d);
cudaError_t gemm_launch(const GemmArgs& a, const PromptDevice& d, cudaStream_t s);

// ------------------------------------------------------------------ norms (q4_block_norm.cu)

struct NormArgs {
  q4_norms p;
  int rows, n;
  RowsIn block, residual;
  RowsOut t, z;
};
cudaError_t block_norm_prepare();
cudaError_t block_norm_launch(const NormArgs& a, int sms, cudaStream_t s);

// ------------------------------------------------------------------ rotary positions (q4_rope.cu)

struct RopeArgs {
  q4_rotation rot;
  const int* positions;     // null: the batch's
  int64_t positions_ld;
  PagedBatch b;
  int rows, heads, inverse;
  RowsIn x;
  RowsOut y;
};
cudaError_t rope_launch(const RopeArgs& a, int sms, cudaStream_t s);

}  // namespace q4
