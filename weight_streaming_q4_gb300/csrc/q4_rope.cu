// Rotary positions of one or several axes (sm_103a).
//
// Pair i of every head of row r turns by the angle p f_i, p the row's position
// on the pair's axis.  p times the turns of one position in 2^-64 of a circle
// (a 64-bit product that wraps, as whole turns may) is the angle's fraction of
// a turn, exact to 2^-33 of it at any position; sincospi takes it from there.
// A CTA takes some heads of some rows: one cosine and sine per pair and row
// into shared memory, then every head's values by 16-byte pieces, read and
// written once.
//
// Measured in a graph: 4096 rows of 40 heads of 128, three axes, binary16: 19.3 us, 4.4 TB/s; four pieces loaded
// at once per thread measured 19.8 to 23.0, more and smaller CTAs 20.1.  16 rows: 3.1 us, a launch.
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_prompt.cuh"

namespace q4 {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 1024;       // cosines of a CTA: rows times pairs

template <int V>
__device__ __forceinline__ void load_v(const float* p, float* v) {
  if (V == 1) {
    v[0] = p[0];
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 f = *(reinterpret_cast<const float4*>(p) + i);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  }
}
template <int V>
__device__ __forceinline__ void load_v(const __half* p, float* v) {
  if (V == 1) {
    v[0] = __half2float(p[0]);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float* v) {
  if (V == 1) {
    p[0] = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) *(reinterpret_cast<float4*>(p) + i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store_v(__half* p, const float* v) {
  if (V == 1) {
    p[0] = __float2half_rn(v[0]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Pieces of V values (8, or 1 where alignment or sizes want it).  Halves: a
// piece of the first half of the turning values with its partner; adjacent: one
// piece (V 1: both values of a pair).  Then the values that stay.
template <int V, bool HALVES, typename X, typename Y>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a, int cta_rows, int cta_heads) {
  __shared__ __align__(16) float s_cos[kRopeTable];
  __shared__ __align__(16) float s_sin[kRopeTable];
  __shared__ bool s_row[kRopeTable];     // the row belongs to a sequence
  const int pairs = a.rot.rot_dim / 2, hd = a.rot.head_dim;
  const int row0 = blockIdx.x * cta_rows, rows = min(cta_rows, a.rows - row0);
  const int head0 = blockIdx.y * cta_heads, heads = min(cta_heads, a.heads - head0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < rows; r += kRopeThreads / 32) {
    int place = 0;
    bool in = true;
    if (!a.positions) {
      const int s = paged_seq_of(a.b, row0 + r);
      in = s >= 0;
      if (in) place = __ldg(a.b.lens + s) - __ldg(a.b.starts + s + 1) + row0 + r;
    }
    if (lane == 0) s_row[r] = in;
    for (int i = lane; in && i < pairs; i += 32) {
      if (a.positions) place = __ldg(a.positions + a.rot.axis[i] * a.positions_ld + row0 + r);
      const uint64_t part = static_cast<uint64_t>(static_cast<int64_t>(place)) * a.rot.turn[i];
      float c, s;
      sincospif(static_cast<float>(static_cast<int64_t>(part)) * 0x1p-63f, &s, &c);
      s_cos[r * pairs + i] = c;
      s_sin[r * pairs + i] = a.inverse ? -s : s;
    }
  }
  __syncthreads();
  constexpr int P = HALVES ? V : (V == 1 ? 2 : V);          // values of a turning piece, on one side
  const int turning = (HALVES ? pairs : a.rot.rot_dim) / P;
  const int each = turning + (hd - a.rot.rot_dim) / V;      // pieces of a head
  const int all = rows * heads * each;
  for (int i = threadIdx.x; i < all; i += kRopeThreads) {
    const int piece = i % each, rh = i / each, r = rh / heads, h = rh - r * heads;
    if (!s_row[r]) continue;
    const X* x = static_cast<const X*>(a.x.p) + (row0 + r) * a.x.ld + static_cast<int64_t>(head0 + h) * hd;
    Y* y = static_cast<Y*>(a.y.p) + (row0 + r) * a.y.ld + static_cast<int64_t>(head0 + h) * hd;
    float u[P], v[P];
    if (piece >= turning) {
      const int at = a.rot.rot_dim + (piece - turning) * V;
      load_v<V>(x + at, u);
      store_v<V>(y + at, u);
    } else if (HALVES) {
      const int at = piece * V;
      float c[P], s[P];
      load_v<V>(x + at, u);
      load_v<V>(x + pairs + at, v);
      load_v<V>(s_cos + r * pairs + at, c);
      load_v<V>(s_sin + r * pairs + at, s);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = u[e] * c[e] - v[e] * s[e];
        v[e] = u[e] * s[e] + v[e] * c[e];
        u[e] = t;
      }
      store_v<V>(y + at, u);
      store_v<V>(y + pairs + at, v);
    } else {
      const int at = piece * P;
      if (V == 1) {
        load_v<V>(x + at, u), load_v<V>(x + at + 1, u + 1);
      } else {
        load_v<V>(x + at, u);
      }
#pragma unroll
      for (int e = 0; e < P; e += 2) {
        const float c = s_cos[r * pairs + (at + e) / 2], s = s_sin[r * pairs + (at + e) / 2];
        v[e] = u[e] * c - u[e + 1] * s;
        v[e + 1] = u[e] * s + u[e + 1] * c;
      }
      if (V == 1) {
        store_v<V>(y + at, v), store_v<V>(y + at + 1, v + 1);
      } else {
        store_v<V>(y + at, v);
      }
    }
  }
}

template <int V, bool HALVES>
void launch_types(const RopeArgs& a, dim3 grid, int cta_rows, int cta_heads, cudaStream_t s) {
  if (a.x.f32 && a.y.f32)
    rope_kernel<V, HALVES, float, float><<<grid, kRopeThreads, 0, s>>>(a, cta_rows, cta_heads);
  else if (a.x.f32)
    rope_kernel<V, HALVES, float, __half><<<grid, kRopeThreads, 0, s>>>(a, cta_rows, cta_heads);
  else if (a.y.f32)
    rope_kernel<V, HALVES, __half, float><<<grid, kRopeThreads, 0, s>>>(a, cta_rows, cta_heads);
  else
    rope_kernel<V, HALVES, __half, __half><<<grid, kRopeThreads, 0, s>>>(a, cta_rows, cta_heads);
}

bool rows16(const void* p, int64_t ld, int f32) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (f32 ? 4 : 2) % 16 == 0;
}

}  // namespace

cudaError_t rope_launch(const RopeArgs& a, int sms, cudaStream_t s) {
  const bool halves = a.rot.style == Q4_ROPE_HALVES;
  const int pairs = a.rot.rot_dim / 2;
  const bool wide = a.rot.head_dim % 8 == 0 && (halves ? pairs : a.rot.rot_dim) % 8 == 0 &&
                    rows16(a.x.p, a.x.ld, a.x.f32) && rows16(a.y.p, a.y.ld, a.y.f32);
  // About 8 pieces a thread; with few rows the heads are shared out too, up to two CTAs per SM.
  // (one head of 8 values is half of two pieces)
  const int each = wide ? 16 : 2;
  const int64_t pieces = (static_cast<int64_t>(a.heads) * a.rot.head_dim + each - 1) / each;
  int cta_rows = static_cast<int>(8 * kRopeThreads / pieces);
  cta_rows = cta_rows < 1 ? 1 : cta_rows > kRopeTable / pairs ? kRopeTable / pairs : cta_rows;
  while (cta_rows > 1 && (a.rows + cta_rows - 1) / cta_rows < 2 * sms) cta_rows /= 2;
  const int row_ctas = (a.rows + cta_rows - 1) / cta_rows;
  int parts = 2 * sms / row_ctas;
  const int64_t most = (pieces * cta_rows + kRopeThreads - 1) / kRopeThreads;      // (a piece a thread)
  if (parts > most) parts = static_cast<int>(most);
  if (parts < (a.heads + 4095) / 4096) parts = (a.heads + 4095) / 4096;
  if (parts > a.heads) parts = a.heads;
  if (parts < 1) parts = 1;
  const int cta_heads = (a.heads + parts - 1) / parts;
  const dim3 grid(row_ctas, (a.heads + cta_heads - 1) / cta_heads);
  if (wide)
    halves ? launch_types<8, true>(a, grid, cta_rows, cta_heads, s) : launch_types<8, false>(a, grid, cta_rows, cta_heads, s);
  else
    halves ? launch_types<1, true>(a, grid, cta_rows, cta_heads, s) : launch_types<1, false>(a, grid, cta_rows, cta_heads, s);
  return cudaGetLastError();
}

}  // namespace q4
