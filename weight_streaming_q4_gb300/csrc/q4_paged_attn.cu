// Attention of new tokens over a paged KV cache (sm_103a): a warp per token
// and query head, every visible position in turn, the softmax in one pass with
// a running maximum and sum (in powers of two; all sums fp32).
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "q4_paged.cuh"

namespace q4 {

namespace {

constexpr int kPaThreads = 128;

// hd / 32 consecutive values per lane.
template <int HD, bool F32, bool Q8>
__global__ void __launch_bounds__(kPaThreads) paged_attn_plain_kernel(PagedAttnArgs a) {
  constexpr int E = HD / 32;
  const int n_q = a.kv.n_kv * a.group;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kPaThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(warp / n_q), h = static_cast<int>(warp % n_q), head = h / a.group;
  if (row >= a.b.n_tokens) return;
  const int s = paged_seq_of(a.b, row);
  if (s < 0) return;
  const SeqSpan sp = paged_span(a.kv, a.b, s);
  const int p = sp.len - sp.n_new + row - sp.t0;
  float q[E], o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int64_t at = row * a.q_ld + h * HD + lane * E + i;
    q[i] = (F32 ? static_cast<const float*>(a.q)[at] : __half2float(static_cast<const __half*>(a.q)[at])) * a.scale;
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int end = min(p + 1, sp.len);
  const int first = a.window ? max(0, p - a.window + 1) : 0;
  for (int t = 0; t < end; ++t) {
    if (t == min(a.sinks, first) && t < first) t = first;
    const int r = paged_row(a.kv, a.b, s, t, head);
    if (r < 0) continue;
    const size_t at = static_cast<size_t>(r) * HD + lane * E;
    float kx[E], vx[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if (Q8) {
        kx[i] = __half2float(__hmul(__int2half_rn(static_cast<const int8_t*>(a.kv.k)[at + i]), a.kv.ks[(at + i) / 32]));
        vx[i] = __half2float(__hmul(__int2half_rn(static_cast<const int8_t*>(a.kv.v)[at + i]), a.kv.vs[(at + i) / 32]));
      } else {
        kx[i] = __half2float(static_cast<const __half*>(a.kv.k)[at + i]);
        vx[i] = __half2float(static_cast<const __half*>(a.kv.v)[at + i]);
      }
    }
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) x = fmaf(q[i], kx[i], x);
#pragma unroll
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
    const float m2 = fmaxf(m, x);
    const float c = m2 == -INFINITY ? 0.f : exp2f(m - m2), w = m2 == -INFINITY ? 0.f : exp2f(x - m2);
    l = l * c + w;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(w, vx[i], o[i] * c);
    m = m2;
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
  for (int i = 0; i < E; ++i) a.out[row * a.out_ld + h * HD + lane * E + i] = __float2half_rn(o[i] * inv);
}

template <int HD>
void launch_hd(const PagedAttnArgs& a, bool f32, bool q8, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(a.b.n_tokens) * a.kv.n_kv * a.group;
  const unsigned n = static_cast<unsigned>((warps * 32 + kPaThreads - 1) / kPaThreads);
  auto kern = f32 ? (q8 ? paged_attn_plain_kernel<HD, true, true> : paged_attn_plain_kernel<HD, true, false>)
                  : (q8 ? paged_attn_plain_kernel<HD, false, true> : paged_attn_plain_kernel<HD, false, false>);
  kern<<<n, kPaThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t paged_attn_launch(const PagedAttnArgs& a, bool q_f32, bool q8, cudaStream_t s) {
  switch (a.kv.hd) {
    case 64: launch_hd<64>(a, q_f32, q8, s); break;
    case 128: launch_hd<128>(a, q_f32, q8, s); break;
    case 192: launch_hd<192>(a, q_f32, q8, s); break;
    default: launch_hd<256>(a, q_f32, q8, s); break;
  }
  return cudaGetLastError();
}

}  // namespace q4
