// Products of many rows with Q4_0 weights, with an epilogue (sm_103a): a 64 x 64
// tile of outputs per CTA, 4 x 4 of them per thread, fp32 sums.
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_prompt.cuh"

namespace q4 {

namespace {

constexpr int kT = 64;

__device__ __forceinline__ float activate(float t, int act) {
  switch (act) {
    case Q4_ACT_RELU: return fmaxf(t, 0.f);
    case Q4_ACT_SILU: return t / (1.f + expf(-t));
    case Q4_ACT_GELU: return 0.5f * t * (1.f + erff(t * 0.70710678f));
    case Q4_ACT_GELU_TANH: return 0.5f * t * (1.f + tanhf(0.79788456f * (t + 0.044715f * t * t * t)));
    default: return t;
  }
}

template <int MATS>
__global__ void __launch_bounds__(256) gemm_kernel(GemmArgs a) {
  __shared__ float sw[MATS][32][kT + 1], sx[32][kT + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n0 = blockIdx.x * kT, r0 = blockIdx.y * kT, nb = a.k / kQK;
  float acc[MATS][4][4] = {};
  for (int b = 0; b < nb; ++b) {
    for (int i = tid; i < MATS * 16 * kT; i += 256) {
      const int j = i & 15, n = (i >> 4) & (kT - 1), m = i / (16 * kT);
      float lo = 0.f, hi = 0.f;
      if (n0 + n < a.n) {
        const uint8_t* blk = a.w[m] + (static_cast<size_t>(n0 + n) * nb + b) * kBlockBytes;
        const __half d = *reinterpret_cast<const __half*>(blk);
        const int q = blk[2 + j];
        lo = __half2float(__hmul(__int2half_rn((q & 15) - 8), d));
        hi = __half2float(__hmul(__int2half_rn((q >> 4) - 8), d));
      }
      sw[m][j][n] = lo, sw[m][j + 16][n] = hi;
    }
    for (int i = tid; i < 32 * kT; i += 256) {
      const int k = i & 31, r = i >> 5;
      sx[k][r] = r0 + r < a.rows ? __half2float(a.x[static_cast<int64_t>(r0 + r) * a.x_ld + b * kQK + k]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 32; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j)
          for (int m = 0; m < MATS; ++m) acc[m][i][j] = fmaf(sx[k][ty + 16 * i], sw[m][k][tx + 16 * j], acc[m][i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (r >= a.rows || n >= a.n) continue;
      float t = activate(acc[0][i][j] + (a.bias[0] ? a.bias[0][n] : 0.f), a.act) * a.scale;
      if (MATS == 2) t *= acc[MATS - 1][i][j] + (a.bias[1] ? a.bias[1][n] : 0.f);
      if (a.residual.p) {
        const int64_t at = r * a.residual.ld + n;
        t += a.residual.f32 ? static_cast<const float*>(a.residual.p)[at] : __half2float(static_cast<const __half*>(a.residual.p)[at]);
      }
      a.y[r * a.y_ld + n] = __float2half_rn(t);
    }
}

}  // namespace

cudaError_t gemm_prepare() { return cudaSuccess; }

cudaError_t gemm_launch(const GemmArgs& a, int, cudaStream_t s) {
  const dim3 grid((a.n + kT - 1) / kT, (a.rows + kT - 1) / kT);
  if (a.w[1])
    gemm_kernel<2><<<grid, 256, 0, s>>>(a);
  else
    gemm_kernel<1><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace q4
