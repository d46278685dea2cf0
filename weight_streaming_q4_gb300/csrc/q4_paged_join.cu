// Joins the parts of items that several CTAs of a paged attention kernel share
// (q4_paged_sched.cuh; sm_103a): out = sum_c O_c 2^(m_c - M) / sum_c l_c 2^(m_c - M)
// over the CTAs c in order, M the largest m_c.  One block per CTA that begins
// such an item and 8 of its rows, a warp per row.  Launched as a
// programmatic dependent of that kernel: its blocks take their place while the
// last CTAs finish and wait for them, so the second launch costs less than one
// after the other.  A batch of chunks and single tokens takes 183 us with it and 171
// in a timing copy without.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "q4_paged_sched.cuh"

namespace q4 {

namespace {

constexpr int kPjThreads = 256;
constexpr int kPjRows = kPjThreads / 32;

template <int HD>
__global__ void __launch_bounds__(kPjThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, PartSlots parts) {
  constexpr int E = HD / 32, B = 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int cta = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const JoinRecord rec = *parts.record(cta);
  const int end = min(rec.rows, static_cast<int>(blockIdx.y + 1) * kPjRows);
  if (rec.n <= 0) return;
  const int r = blockIdx.y * kPjRows + warp;
  if (r < end) {
    // Part 0 is slot 1 of this CTA, part c > 0 slot 0 of CTA cta + c.  Four parts' loads at a time are
    // under way together; the sums run in the order of the parts, rescaled when a later one raises the maximum.
    float top = -INFINITY, sum = 0.f, o[E] = {};
    for (int c0 = 0; c0 < rec.n; c0 += B) {
      float m[B], l[B];
      float2 v[B][E / 2];
#pragma unroll
      for (int k = 0; k < B; ++k) {
        const int c = c0 + k;
        m[k] = -INFINITY;
        if (c >= rec.n) continue;
        m[k] = parts.max(cta + c, c == 0)[r];
        l[k] = parts.sum(cta + c, c == 0)[r];
        const float* src = parts.out(cta + c, c == 0) + static_cast<size_t>(r) * HD + lane * 2;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) v[k][e] = *reinterpret_cast<const float2*>(src + e * 64);
      }
      float most = top;
#pragma unroll
      for (int k = 0; k < B; ++k) most = fmaxf(most, m[k]);
      const float back = top == most ? 1.f : exp2f(top - most);
      top = most;
      sum *= back;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= back;
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (c0 + k >= rec.n) continue;
        const float f = m[k] == -INFINITY ? 0.f : exp2f(m[k] - top);       // (times 0: what is not a number stays so)
        sum += l[k] * f;
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          o[2 * e] += v[k][e].x * f;
          o[2 * e + 1] += v[k][e].y * f;
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __half* out = a.out + a.row_at(rec.t0, rec.head, rec.row0 + r, a.out_ld) + lane * 2;
#pragma unroll
    for (int e = 0; e < E / 2; ++e)
      *reinterpret_cast<__half2*>(out + e * 64) = __floats2half2_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
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
