// Writing new tokens into the pages of a KV cache, and reading positions back
// out of them (sm_103a).
//
// The serving counterpart of the per-layer KV cache PIPO moves with the layer
// ("PIPO: Pipelined Offloading for Efficient Inference on Consumer Devices",
// Method, "Offloading architecture").
//
// Both are one pass over the rows: 8 values per thread and step (16 or 32
// bytes of the row, 16 or 8 of the page), a warp per 32 such chunks of a
// token's key and value.  A Q8 block of 32 values is four neighbouring lanes:
// its maximum is two shuffles.  They are bound by HBM bandwidth for many
// tokens and by the launch and three dependent loads (starts, length, page)
// for few.
//
// Exactness of the quantiser in 32 bits: amax / 127 and x / d are IEEE
// divisions.  A quotient can only round across a tie of the next rounding (a
// binary16 midpoint for d, n + 1/2 for a code) if the true quotient lies within
// half an fp32 step of the tie without being it.  tie * divisor has at most
// 12 + 7 and 8 + 11 significant bits, so it is an fp32 number, and the dividend
// differs from it by a whole fp32 step or not at all: relative to the tie at
// least 2^-23 / m with the dividend's mantissa m < 2, more than the quotient's
// half step.  So d and the codes are those of exact arithmetic.
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_paged.cuh"

namespace q4 {

namespace {

constexpr int kPcThreads = 256;

template <bool F32>
__device__ __forceinline__ void load8(const void* row, int64_t at, float (&x)[8]) {
  if (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(row) + at);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(row) + at));
    const __half2* h = reinterpret_cast<const __half2*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
}

// A warp per 32 chunks of one token: chunk c of the token's 2 * n_kv * hd / 8
// is 8 values of its key (first half) or its value.
template <bool F32, bool Q8>
__global__ void __launch_bounds__(kPcThreads) paged_write_kernel(PagedKv kv, PagedBatch b, const void* k, const void* v,
                                                                int64_t ld, int groups) {
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kPcThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(warp / groups), c = static_cast<int>(warp % groups) * 32 + lane;
  if (row >= b.n_tokens) return;
  const int s = paged_seq_of(b, row);
  if (s < 0) return;
  const SeqSpan sp = paged_span(kv, b, s);
  const int p = sp.len - sp.n_new + row - sp.t0;
  const int half = kv.n_kv * kv.hd / 8;
  const bool live = c < 2 * half && p >= 0;
  const int at = c < half ? c : c - half, e = at * 8;
  const int head = e / kv.hd, i = e - head * kv.hd;
  const int dst = live ? paged_row(kv, b, s, p, head) : -1;
  float x[8] = {};
  if (dst >= 0) load8<F32>(c < half ? k : v, row * ld + e, x);
  if (!Q8) {
    if (dst < 0) return;
    uint4 o;
    __half2* h = reinterpret_cast<__half2*>(&o);
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<uint4*>(static_cast<__half*>(c < half ? kv.k : kv.v) + static_cast<size_t>(dst) * kv.hd + i) = o;
    return;
  }
  // the block's maximum and whether it holds a NaN (fmaxf drops NaN): the four
  // lanes of a block share its fate (a head is a whole number of blocks)
  float m = 0.f;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j])), nan |= x[j] != x[j];
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 1));
  m = fmaxf(m, __shfl_xor_sync(~0u, m, 2));
  const unsigned nans = __ballot_sync(~0u, nan);
  nan = (nans >> (lane & 28)) & 15;
  if (dst < 0) return;
  __half d = __float2half_rn(__fdiv_rn(m, 127.f));
  if (nan || !(__half2float(d) <= 65504.f)) d = __ushort_as_half(0x7fff);
  const float df = __half2float(d);
  uint2 o;
  int8_t* q = reinterpret_cast<int8_t*>(&o);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    q[j] = df > 0.f ? static_cast<int8_t>(fminf(fmaxf(rintf(__fdiv_rn(x[j], df)), -127.f), 127.f)) : int8_t(0);
  const size_t to = static_cast<size_t>(dst) * kv.hd + i;
  *reinterpret_cast<uint2*>(static_cast<int8_t*>(c < half ? kv.k : kv.v) + to) = o;
  if ((lane & 3) == 0) (c < half ? kv.ks : kv.vs)[to / 32] = d;
}

template <bool F32, bool Q8>
__global__ void __launch_bounds__(kPcThreads) paged_read_kernel(PagedKv kv, PagedBatch b, void* k, void* v, int64_t ld,
                                                               int groups) {
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kPcThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(warp / groups), c = static_cast<int>(warp % groups) * 32 + lane;
  if (row >= b.n_tokens) return;
  const int s = paged_seq_of(b, row);
  if (s < 0) return;
  const SeqSpan sp = paged_span(kv, b, s);
  const int p = sp.len - sp.n_new + row - sp.t0;
  const int half = kv.n_kv * kv.hd / 8;
  if (c >= 2 * half) return;
  const int at = c < half ? c : c - half, e = at * 8;
  const int head = e / kv.hd, i = e - head * kv.hd;
  const int src = p >= 0 ? paged_row(kv, b, s, p, head) : -1;
  uint4 u = make_uint4(0, 0, 0, 0);
  __half2* h = reinterpret_cast<__half2*>(&u);
  if (src >= 0) {
    const size_t from = static_cast<size_t>(src) * kv.hd + i;
    if (Q8) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(c < half ? kv.k : kv.v) + from));
      const __half2 d = __half2half2((c < half ? kv.ks : kv.vs)[from / 32]);
      q8_values4(q.x, d, h[0], h[1]);
      q8_values4(q.y, d, h[2], h[3]);
    } else {
      u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(c < half ? kv.k : kv.v) + from));
    }
  }
  void* out = c < half ? k : v;
  if (F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * ld + e);
    const float2 f0 = __half22float2(h[0]), f1 = __half22float2(h[1]), f2 = __half22float2(h[2]), f3 = __half22float2(h[3]);
    o[0] = make_float4(f0.x, f0.y, f1.x, f1.y);
    o[1] = make_float4(f2.x, f2.y, f3.x, f3.y);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__half*>(out) + row * ld + e) = u;
  }
}

// Grid of a warp per 32 chunks of a row.  The blocks fit an int: 2^31 of them
// would be 4 TB of rows.
unsigned blocks_of(const PagedKv& kv, const PagedBatch& b, int* groups) {
  *groups = (2 * kv.n_kv * kv.hd / 8 + 31) / 32;
  const int64_t warps = static_cast<int64_t>(b.n_tokens) * *groups;
  return static_cast<unsigned>((warps * 32 + kPcThreads - 1) / kPcThreads);
}

}  // namespace

cudaError_t paged_write_launch(const PagedKv& kv, const PagedBatch& b, const void* k, const void* v, bool f32,
                               int64_t ld, bool q8, cudaStream_t s) {
  int groups;
  const unsigned n = blocks_of(kv, b, &groups);
  auto kern = f32 ? (q8 ? paged_write_kernel<true, true> : paged_write_kernel<true, false>)
                  : (q8 ? paged_write_kernel<false, true> : paged_write_kernel<false, false>);
  kern<<<n, kPcThreads, 0, s>>>(kv, b, k, v, ld, groups);
  return cudaGetLastError();
}

cudaError_t paged_read_launch(const PagedKv& kv, const PagedBatch& b, void* k, void* v, bool f32, int64_t ld, bool q8,
                              cudaStream_t s) {
  int groups;
  const unsigned n = blocks_of(kv, b, &groups);
  auto kern = f32 ? (q8 ? paged_read_kernel<true, true> : paged_read_kernel<true, false>)
                  : (q8 ? paged_read_kernel<false, true> : paged_read_kernel<false, false>);
  kern<<<n, kPcThreads, 0, s>>>(kv, b, k, v, ld, groups);
  return cudaGetLastError();
}

}  // namespace q4
