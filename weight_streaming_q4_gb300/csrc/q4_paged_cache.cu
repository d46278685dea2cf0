// Writing new tokens into the pages of a KV cache, and reading positions back
// out of them (sm_103a).
//
// The serving counterpart of the per-layer KV cache PIPO moves with the layer
// ("PIPO: Pipelined Offloading for Efficient Inference on Consumer Devices",
// Method, "Offloading architecture").
//
// Both are one pass over the rows: 8 values per thread and step (16 or 32
// bytes of the row, 16 or 8 of the page), a warp per 32 or 128 such chunks of a
// token's key and value.  A Q8 block of 32 values is four neighbouring lanes:
// its maximum is two shuffles.  They are bound by HBM bandwidth for many
// tokens and by the launch and three dependent loads (starts, length, page)
// for few.  Measured: 11 878 tokens of the 8B heads from fp32 to Q8 and back to
// binary16 40 us for both, 4.9 TB/s (the quantiser's issue slots are 68 % busy);
// 16 tokens to binary16 2.1 us; 4096 positions of Q8 read 7.3 us, 3.5 TB/s.
//
// The quantiser is exact: d and the codes are those of exact arithmetic.
// d: amax / 127 is an IEEE division, and a quotient can only round across a tie
// of the next rounding (a binary16 midpoint) if the true quotient lies within half an
// fp32 step of the tie without being it.  tie * 127 has at most 12 + 7 significant
// bits, so it is an fp32 number, and amax differs from it by a whole fp32 step or
// not at all: relative to the tie at least 2^-23 / m with amax's mantissa m < 2,
// more than the quotient's half step.
// Codes: x * (1 / d) is within 2^-23 of the quotient relative to it, at most 127.5
// (a block with a subnormal d: clamped), so its nearest integer n is the
// quotient's or, next to a tie, one beside it.  r = x - n d is exact (n d has 18 bits, and r is
// a multiple of x's last bit no larger than d), so comparing |r| with d / 2 tells,
// ties going to the even n.  (An IEEE division per value took a third of the
// kernel's instructions, this test for each value another third: it is one comparison
// for all but the blocks with a value on a tie or across one.)
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_paged.cuh"

namespace q4 {

namespace {

constexpr int kPcThreads = 128;

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

// The larger of two numbers; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// rint(x / d) within -127..127 of 8 values, as bytes; 0 where d is 0 or NaN.
__device__ __forceinline__ uint2 q8_codes(const float (&x)[8], float d) {
  if (!(d > 0.f)) return make_uint2(0, 0);
  constexpr float kMagic = 12582912.f;       // 1.5 * 2^23: a number added to it is rounded to an integer, in its low bits
  const float inv = __fdiv_rn(1.f, d), half = 0.5f * d;
  uint32_t n[8];
  bool near = d < 6.103515625e-05f;          // (a subnormal scale: the codes may pass 127)
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = __fmaf_rn(x[j], inv, kMagic);
    near |= fabsf(__fmaf_rn(kMagic - t, d, x[j])) >= half;
    n[j] = __float_as_uint(t);
  }
  if (near) {                                // on a tie or across one: rare
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float r = __fmaf_rn(kMagic - __uint_as_float(n[j]), d, x[j]);
      int q = static_cast<int>(n[j]);
      if (fabsf(r) > half || (fabsf(r) == half && (q & 1))) q += r > 0.f ? 1 : -1;
      n[j] = static_cast<uint32_t>(min(max(q, 0x4b400000 - 127), 0x4b400000 + 127));
    }
  }
  return make_uint2(__byte_perm(__byte_perm(n[0], n[1], 0x0040), __byte_perm(n[2], n[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(n[4], n[5], 0x0040), __byte_perm(n[6], n[7], 0x0040), 0x5410));
}

// Where a warp's part of a token lives.  Chunk c of a token's 2 * n_kv * HD / 8
// is 8 values of its key (first half) or its value; a warp takes U * 32 chunks
// in a row, and looks up the token's page once.
template <int HD>
struct TokenAt {
  int page, slot;           // page: -1 when the token is in none
  bool mine;                // the row belongs to a sequence
  __device__ __forceinline__ TokenAt(const PagedKv& kv, const PagedBatch& b, int row) {
    page = -1, slot = 0;
    const int s = paged_seq_of(b, row);
    mine = s >= 0;
    if (!mine) return;
    const SeqSpan sp = paged_span(kv, b, s);
    const int p = sp.len - sp.n_new + row - sp.t0, e = p >> kv.page_log2;
    if (p < 0 || e >= b.width) return;
    page = __ldg(b.table + static_cast<size_t>(s) * b.width + e);
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(kv.n_pages)) page = -1;
    slot = p & ((1 << kv.page_log2) - 1);
  }
  // first of the chunk's values in the page memory; at: its first value within the key or value row
  __device__ __forceinline__ size_t value(const PagedKv& kv, int at) const {
    const int head = at / HD;
    return ((static_cast<size_t>(page) * kv.n_kv + head) << kv.page_log2) * HD + static_cast<size_t>(slot) * HD + (at - head * HD);
  }
};

template <int HD, bool F32, bool Q8, int U>
__global__ void __launch_bounds__(kPcThreads) paged_write_kernel(PagedKv kv, PagedBatch b, const void* k, const void* v,
                                                                int64_t ld, int groups) {
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kPcThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(warp / groups), c0 = static_cast<int>(warp % groups) * 32 * U + lane;
  if (row >= b.n_tokens) return;
  const int half = kv.n_kv * HD / 8;
  // the rows do not wait for the page (a row that is in none is read for nothing)
  float x[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * 32;
    if (c < 2 * half) load8<F32>(c < half ? k : v, row * ld + (c < half ? c : c - half) * 8, x[u]);
  }
  const TokenAt<HD> t(kv, b, row);
  if (t.page < 0) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * 32;
    const bool live = c < 2 * half;
    const size_t to = live ? t.value(kv, (c < half ? c : c - half) * 8) : 0;
    if (!Q8) {
      uint4 o;
      __half2* h = reinterpret_cast<__half2*>(&o);
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(x[u][2 * j], x[u][2 * j + 1]);
      if (live) *reinterpret_cast<uint4*>(static_cast<__half*>(c < half ? kv.k : kv.v) + to) = o;
      continue;
    }
    // the block's maximum, NaN if it holds one: the four lanes of a block share its fate (a head is a whole
    // number of blocks)
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!live) x[u][j] = 0.f;
      m = max_nan(m, fabsf(x[u][j]));
    }
    m = max_nan(m, __shfl_xor_sync(~0u, m, 1));
    m = max_nan(m, __shfl_xor_sync(~0u, m, 2));
    __half d = __float2half_rn(__fdiv_rn(m, 127.f));
    if (!(__half2float(d) <= 65504.f)) d = __ushort_as_half(0x7fff);
    const uint2 o = q8_codes(x[u], __half2float(d));
    if (!live) continue;
    *reinterpret_cast<uint2*>(static_cast<int8_t*>(c < half ? kv.k : kv.v) + to) = o;
    if ((lane & 3) == 0) (c < half ? kv.ks : kv.vs)[to / 32] = d;
  }
}

template <int HD, bool F32, bool Q8, int U>
__global__ void __launch_bounds__(kPcThreads) paged_read_kernel(PagedKv kv, PagedBatch b, void* k, void* v, int64_t ld,
                                                               int groups) {
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kPcThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int row = static_cast<int>(warp / groups), c0 = static_cast<int>(warp % groups) * 32 * U + lane;
  if (row >= b.n_tokens) return;
  const TokenAt<HD> t(kv, b, row);
  if (!t.mine) return;
  const int half = kv.n_kv * HD / 8;
  uint4 f[U];               // binary16 values, or Q8 codes in the first half
  __half d[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * 32;
    f[u] = make_uint4(0, 0, 0, 0);
    d[u] = __ushort_as_half(0);
    if (c >= 2 * half || t.page < 0) continue;
    const size_t from = t.value(kv, (c < half ? c : c - half) * 8);
    if (Q8) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(c < half ? kv.k : kv.v) + from));
      f[u].x = q.x, f[u].y = q.y;
      d[u] = (c < half ? kv.ks : kv.vs)[from / 32];
    } else {
      f[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __half*>(c < half ? kv.k : kv.v) + from));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + u * 32;
    if (c >= 2 * half) continue;
    const int64_t to = row * ld + (c < half ? c : c - half) * 8;
    uint4 y = f[u];
    __half2* h = reinterpret_cast<__half2*>(&y);
    if (Q8) {
      const __half2 d2 = __half2half2(d[u]);
      q8_values4(f[u].x, d2, h[0], h[1]);
      q8_values4(f[u].y, d2, h[2], h[3]);
    }
    void* out = c < half ? k : v;
    if (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + to);
      const float2 f0 = __half22float2(h[0]), f1 = __half22float2(h[1]), f2 = __half22float2(h[2]), f3 = __half22float2(h[3]);
      o[0] = make_float4(f0.x, f0.y, f1.x, f1.y);
      o[1] = make_float4(f2.x, f2.y, f3.x, f3.y);
    } else {
      *reinterpret_cast<uint4*>(static_cast<__half*>(out) + to) = y;
    }
  }
}

// U * 32 chunks of a row per warp.  Where the rows fill the GPU anyway, four
// loads per lane under way and one look-up for them; few rows (a step's tokens)
// are spread over as many warps as they have.
constexpr int kPcMany = 4;
bool many_rows(const PagedKv& kv, const PagedBatch& b) {
  return static_cast<int64_t>(b.n_tokens) * kv.n_kv * kv.hd >= int64_t{1} << 20;
}
unsigned blocks_of(const PagedKv& kv, const PagedBatch& b, int u, int* groups) {
  *groups = (2 * kv.n_kv * kv.hd / 8 + 32 * u - 1) / (32 * u);
  // (the blocks fit an int: 2^31 of them would be 4 TB of rows)
  const int64_t warps = static_cast<int64_t>(b.n_tokens) * *groups;
  return static_cast<unsigned>((warps * 32 + kPcThreads - 1) / kPcThreads);
}

template <int HD, bool F32, bool Q8>
void launch_write(const PagedKv& kv, const PagedBatch& b, const void* k, const void* v, int64_t ld, cudaStream_t s) {
  int groups;
  if (many_rows(kv, b)) {
    const unsigned n = blocks_of(kv, b, kPcMany, &groups);
    paged_write_kernel<HD, F32, Q8, kPcMany><<<n, kPcThreads, 0, s>>>(kv, b, k, v, ld, groups);
  } else {
    const unsigned n = blocks_of(kv, b, 1, &groups);
    paged_write_kernel<HD, F32, Q8, 1><<<n, kPcThreads, 0, s>>>(kv, b, k, v, ld, groups);
  }
}

template <int HD, bool F32, bool Q8>
void launch_read(const PagedKv& kv, const PagedBatch& b, void* k, void* v, int64_t ld, cudaStream_t s) {
  int groups;
  if (many_rows(kv, b)) {
    const unsigned n = blocks_of(kv, b, kPcMany, &groups);
    paged_read_kernel<HD, F32, Q8, kPcMany><<<n, kPcThreads, 0, s>>>(kv, b, k, v, ld, groups);
  } else {
    const unsigned n = blocks_of(kv, b, 1, &groups);
    paged_read_kernel<HD, F32, Q8, 1><<<n, kPcThreads, 0, s>>>(kv, b, k, v, ld, groups);
  }
}

// f<HD, F32, Q8>(...) of the types at hand.
#define Q4_BY_TYPE(f, hd, f32, q8, ...)                                                          \
  do {                                                                                           \
    switch (hd) {                                                                                \
      case 64: f32 ? (q8 ? f<64, true, true>(__VA_ARGS__) : f<64, true, false>(__VA_ARGS__))     \
                   : (q8 ? f<64, false, true>(__VA_ARGS__) : f<64, false, false>(__VA_ARGS__));  \
        break;                                                                                   \
      case 128: f32 ? (q8 ? f<128, true, true>(__VA_ARGS__) : f<128, true, false>(__VA_ARGS__))  \
                    : (q8 ? f<128, false, true>(__VA_ARGS__) : f<128, false, false>(__VA_ARGS__)); \
        break;                                                                                   \
      case 192: f32 ? (q8 ? f<192, true, true>(__VA_ARGS__) : f<192, true, false>(__VA_ARGS__))  \
                    : (q8 ? f<192, false, true>(__VA_ARGS__) : f<192, false, false>(__VA_ARGS__)); \
        break;                                                                                   \
      default: f32 ? (q8 ? f<256, true, true>(__VA_ARGS__) : f<256, true, false>(__VA_ARGS__))   \
                   : (q8 ? f<256, false, true>(__VA_ARGS__) : f<256, false, false>(__VA_ARGS__)); \
    }                                                                                            \
  } while (0)

}  // namespace

cudaError_t paged_write_launch(const PagedKv& kv, const PagedBatch& b, const void* k, const void* v, bool f32,
                               int64_t ld, bool q8, cudaStream_t s) {
  Q4_BY_TYPE(launch_write, kv.hd, f32, q8, kv, b, k, v, ld, s);
  return cudaGetLastError();
}

cudaError_t paged_read_launch(const PagedKv& kv, const PagedBatch& b, void* k, void* v, bool f32, int64_t ld, bool q8,
                              cudaStream_t s) {
  Q4_BY_TYPE(launch_read, kv.hd, f32, q8, kv, b, k, v, ld, s);
  return cudaGetLastError();
}

}  // namespace q4
