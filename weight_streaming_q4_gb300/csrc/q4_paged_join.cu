// Joins the parts of items that several CTAs of a paged attention kernel share
// (q4_paged_sched.cuh; sm_103a): out = sum_c O_c 2^(m_c - M) / sum_c l_c 2^(m_c - M)
// over the CTAs c in order, M the largest m_c.  One block per CTA that begins
// such an item and 32 of its rows, a warp per row at a time.  Launched as a
// programmatic dependent of that kernel: its blocks take their place while the
// last CTAs finish and wait for them, so the second launch costs less than one
// after the other.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "q4_paged_sched.cuh"

namespace q4 {

namespace {

constexpr int kPjThreads = 256;
constexpr int kPjRows = 32;

template <int HD>
__global__ void __launch_bounds__(kPjThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, PartSlots parts) {
  constexpr int E = HD / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const JoinRecord rec = *parts.record(cta);
  const int end = min(rec.rows, static_cast<int>(blockIdx.y + 1) * kPjRows);
  if (rec.n <= 0) return;
  for (int r = blockIdx.y * kPjRows + warp; r < end; r += kPjThreads / 32) {
    // part 0 is slot 1 of this CTA, part c > 0 slot 0 of CTA cta + c
    float top = -INFINITY;
    for (int c = lane; c < rec.n; c += 32) top = fmaxf(top, parts.max(cta + c, c == 0)[r]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
    float sum = 0.f, o[E] = {};
#pragma unroll 4
    for (int c = 0; c < rec.n; ++c) {
      const float m = parts.max(cta + c, c == 0)[r], l = parts.sum(cta + c, c == 0)[r];
      const float* src = parts.out(cta + c, c == 0) + static_cast<size_t>(r) * HD + lane * 2;
      const float f = m == -INFINITY ? 0.f : exp2f(m - top);
      sum += l * f;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2*>(src + e * 32);
        o[e] += v.x * f;
        o[e + 1] += v.y * f;
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int row = rec.row0 + r;
    __half* out = a.out + static_cast<int64_t>(rec.t0 + row / a.group) * a.out_ld + (rec.head * a.group + row % a.group) * HD + lane * 2;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<__half2*>(out + e * 32) = __floats2half2_rn(o[e] * inv, o[e + 1] * inv);
  }
}

}  // namespace

cudaError_t paged_join_launch(const PagedAttnArgs& a, const PartSlots& parts, int grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, (parts.rows + kPjRows - 1) / kPjRows);
  cfg.blockDim = dim3(kPjThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  switch (a.kv.hd) {
    case 64: return cudaLaunchKernelEx(&cfg, paged_join_kernel<64>, a, parts);
    case 128: return cudaLaunchKernelEx(&cfg, paged_join_kernel<128>, a, parts);
    case 192: return cudaLaunchKernelEx(&cfg, paged_join_kernel<192>, a, parts);
    default: return cudaLaunchKernelEx(&cfg, paged_join_kernel<256>, a, parts);
  }
}

}  // namespace q4
