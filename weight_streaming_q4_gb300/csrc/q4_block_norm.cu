// The norms after and before a block with its gate, its scale and the residual,
// in one pass (sm_103a).
//
//   u = block or norm(block) * post_weight + post_bias;  t = residual + scale * gate * u;  z = norm(t) * weight + bias
//
// One CTA per row, whose values stay in registers from the first load to the
// last store: block and residual are read once, t and z written once, and
// nothing else comes from memory (the vectors are read by every row, out of
// L1 and L2).
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_prompt.cuh"

namespace q4 {

namespace {

// E values of a row per thread, V side by side: chunk j of V values starts at (j * threads + thread) * V.
template <int V>
__device__ __forceinline__ void load_row(const RowsIn& r, int64_t at, float* v) {
  if (V == 1) {
    v[0] = r.f32 ? static_cast<const float*>(r.p)[at] : __half2float(static_cast<const __half*>(r.p)[at]);
  } else if (r.f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(r.p) + at);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 f = __ldcs(p + i);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __half*>(r.p) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
  }
}

template <int V>
__device__ __forceinline__ void store_row(const RowsOut& r, int64_t at, const float* v) {
  if (V == 1) {
    if (r.f32)
      static_cast<float*>(r.p)[at] = v[0];
    else
      static_cast<__half*>(r.p)[at] = __float2half_rn(v[0]);
  } else if (r.f32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(r.p) + at);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) p[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__half*>(r.p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int V>
__device__ __forceinline__ void load_vec(const float* p, int at, float* v) {
  if (V == 1) {
    v[0] = __ldg(p + at);
  } else {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + at) + i);
      v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
    }
  }
}

// Sum over the CTA, the same order in every thread.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  __syncthreads();                      // (the sums before this one have been read)
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <int V, int E, int T>
__global__ void __launch_bounds__(T) block_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[32];
  const int64_t row = blockIdx.x;
  const int step = blockDim.x * V, at0 = threadIdx.x * V;
  const float inv_n = 1.f / static_cast<float>(a.n);
  const q4_norms& p = a.p;
  float v[E];

  // v: centred (Q4_NORM_LAYER) and the factor 1 / sqrt(mean of squares + eps) of it
  auto stats = [&]() {
    float s = 0.f;
    if (p.kind == Q4_NORM_LAYER) {
#pragma unroll
      for (int i = 0; i < E; ++i) s += v[i];
      const float mean = cta_sum(s, red) * inv_n;
#pragma unroll
      for (int j = 0; j < E / V; ++j)
        if (at0 + j * step < a.n)
#pragma unroll
          for (int i = 0; i < V; ++i) v[j * V + i] -= mean;
      s = 0.f;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(v[i], v[i], s);
    return 1.f / sqrtf(fmaf(cta_sum(s, red), inv_n, p.eps));
  };

  float r[E];
#pragma unroll
  for (int j = 0; j < E / V; ++j) {
    const int at = at0 + j * step;
#pragma unroll
    for (int i = 0; i < V; ++i) v[j * V + i] = r[j * V + i] = 0.f;
    if (at < a.n) {
      if (a.block.p) load_row<V>(a.block, row * a.block.ld + at, v + j * V);
      if (a.residual.p) load_row<V>(a.residual, row * a.residual.ld + at, r + j * V);
    }
  }
  const bool post = a.block.p && p.post;
  const float f = post ? stats() : 1.f;
  const float* gate = !p.gate ? nullptr : p.gate + (p.gate_rows ? row / p.gate_rows * p.gate_ld : 0);
#pragma unroll
  for (int j = 0; j < E / V; ++j) {
    const int at = at0 + j * step;
    if (at >= a.n) continue;
    float w[V];
    if (post) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[j * V + i] *= f;
      if (p.post_weight) {
        load_vec<V>(p.post_weight, at, w);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j * V + i] *= w[i];
      }
      if (p.post_bias) {
        load_vec<V>(p.post_bias, at, w);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j * V + i] += w[i];
      }
    }
    if (gate) {
      load_vec<V>(gate, at, w);
#pragma unroll
      for (int i = 0; i < V; ++i) v[j * V + i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[j * V + i] = a.block.p ? fmaf(v[j * V + i], p.scale, r[j * V + i]) : r[j * V + i];
    if (a.t.p) store_row<V>(a.t, row * a.t.ld + at, v + j * V);
  }
  if (!a.z.p) return;
  const float g = stats();
#pragma unroll
  for (int j = 0; j < E / V; ++j) {
    const int at = at0 + j * step;
    if (at >= a.n) continue;
    float w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[j * V + i] *= g;
    if (p.weight) {
      load_vec<V>(p.weight, at, w);
#pragma unroll
      for (int i = 0; i < V; ++i) v[j * V + i] *= w[i];
    }
    if (p.bias) {
      load_vec<V>(p.bias, at, w);
#pragma unroll
      for (int i = 0; i < V; ++i) v[j * V + i] += w[i];
    }
    store_row<V>(a.z, row * a.z.ld + at, v + j * V);
  }
}

bool rows16(const void* p, int64_t ld, int f32) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (f32 ? 4 : 2) % 16 == 0);
}
bool vec16(const float* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t block_norm_launch(const NormArgs& a, cudaStream_t s) {
  const q4_norms& p = a.p;
  const bool wide = a.n % 8 == 0 && rows16(a.block.p, a.block.ld, a.block.f32) &&
                    rows16(a.residual.p, a.residual.ld, a.residual.f32) && rows16(a.t.p, a.t.ld, a.t.f32) &&
                    rows16(a.z.p, a.z.ld, a.z.f32) && vec16(p.post_weight) && vec16(p.post_bias) && vec16(p.gate) &&
                    (!p.gate || !p.gate_rows || p.gate_ld % 4 == 0) && vec16(p.weight) && vec16(p.bias);
  // 16 values per thread up to 8192 of a row, else 32 (1024 threads take 32768)
  const int e = a.n <= 8192 ? 16 : 32;
  const int threads = ((a.n + e - 1) / e + 31) / 32 * 32;
  void (*const kernel)(NormArgs) = e == 16          ? (wide ? block_norm_kernel<8, 16, 512> : block_norm_kernel<1, 16, 512>)
                                   : threads <= 512 ? (wide ? block_norm_kernel<8, 32, 512> : block_norm_kernel<1, 32, 512>)
                                                    : (wide ? block_norm_kernel<8, 32, 1024> : block_norm_kernel<1, 32, 1024>);
  kernel<<<a.rows, threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace q4
