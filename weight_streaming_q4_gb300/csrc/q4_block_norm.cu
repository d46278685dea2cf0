// The norms after and before a block with its gate, its scale and the residual,
// in one pass (sm_103a).
//
//   u = block or norm(block) * post_weight + post_bias;  t = residual + scale * gate * u;  z = norm(t) * weight + bias
//
// A CTA per row, whose values stay in registers: block and residual are read once,
// t and z written once.  Rows of whole 16-byte pieces go through persistent CTAs
// that fetch the next rows while they work on one.
//
// Measured in a graph, other buffers every time: 2048 rows of 8192, binary16 block onto an fp32 residual, t and z: 34 us,
// 5.9 TB/s (a copy of as many bytes 31); with a post norm, its bias and gates 44 us on the same card, since
// one row's statistics, gate and second statistics follow one another on an SM.  16 rows of 4096: 2.9 us, a launch.
// Rows that are not whole pieces, 2048 of 8191 with all of it: 78 us (eight scalar loads for a wide one).
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_prompt.cuh"

namespace q4 {

namespace {

// V values side by side.
template <int V>
__device__ __forceinline__ void load_row(const RowsIn& r, int64_t at, float* v) {
  if (r.f32) {
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
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p + at) + i);
    v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
  }
}

__device__ __forceinline__ void cp16_once(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Sum over the CTA, the same order in every thread.  red: not the place of the sum before it (whose readers are known to be
// done only behind this one's barrier).
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// Rows of any alignment and length: persistent CTAs, a value per access (a warp takes 32 side by side).  Every load of a
// batch is issued before any of them is used, and with AHEAD the next row is on its way, as the bits it has in memory,
// while a row is worked on.
template <int E, int T, bool AHEAD>
__global__ void __launch_bounds__(T, 1) block_norm_any_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][32];
  int turn = 0;
  const float inv_n = 1.f / static_cast<float>(a.n);
  const q4_norms& p = a.p;
  // (a warp's values side by side, so that a thread's lie at fixed distances from its first one)
  constexpr int step = 32;
  const int at0 = static_cast<int>(threadIdx.x >> 5) * 32 * E + static_cast<int>(threadIdx.x & 31);
  const bool has_block = a.block.p != nullptr, post = has_block && p.post;
  // (without a block the residual takes its place)
  const RowsIn first{has_block ? a.block.p : a.residual.p, has_block ? a.block.ld : a.residual.ld, has_block ? a.block.f32 : a.residual.f32};
  const RowsIn second{has_block ? a.residual.p : nullptr, a.residual.ld, a.residual.f32};

  // COUNT values of a row from chunk j0 on, as their bits
  auto get = [&](const RowsIn& r, int64_t row, int j0, auto& raw) {
    constexpr int COUNT = sizeof(raw) / sizeof(raw[0]);
    const int left = row < a.rows && r.p ? a.n : 0;
    if (r.f32) {
      const uint32_t* src = static_cast<const uint32_t*>(r.p) + row * r.ld + at0;
#pragma unroll
      for (int j = 0; j < COUNT; ++j) raw[j] = at0 + (j0 + j) * step < left ? src[(j0 + j) * step] : 0;
    } else {
      const uint16_t* src = static_cast<const uint16_t*>(r.p) + row * r.ld + at0;
#pragma unroll
      for (int j = 0; j < COUNT; ++j) raw[j] = at0 + (j0 + j) * step < left ? src[(j0 + j) * step] : 0;
    }
  };
  auto value = [](const RowsIn& r, uint32_t raw) {
    return r.f32 ? __uint_as_float(raw) : __half2float(__ushort_as_half(static_cast<unsigned short>(raw)));
  };
  auto vector = [&](const float* src, int j0, float other, auto& w) {
    constexpr int COUNT = sizeof(w) / sizeof(w[0]);
    const int left = src ? a.n : 0;
#pragma unroll
    for (int j = 0; j < COUNT; ++j) w[j] = at0 + (j0 + j) * step < left ? __ldg(src + at0 + (j0 + j) * step) : other;
  };

  uint32_t next1[E], next2[AHEAD ? E : 1];
  if (AHEAD) get(first, blockIdx.x, 0, next1), get(second, blockIdx.x, 0, next2);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float v[E], r[AHEAD ? E : 1];
    if (!AHEAD) get(first, row, 0, next1);
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = value(first, next1[j]);
    if (AHEAD) {
#pragma unroll
      for (int j = 0; j < E; ++j) r[j % (AHEAD ? E : 1)] = value(second, next2[j % (AHEAD ? E : 1)]);
      get(first, row + gridDim.x, 0, next1), get(second, row + gridDim.x, 0, next2);
    }
    // v: centred (Q4_NORM_LAYER) and the factor 1 / sqrt(mean of squares + eps) of it
    auto stats = [&]() {
      float s = 0.f;
      if (p.kind == Q4_NORM_LAYER) {
#pragma unroll
        for (int j = 0; j < E; ++j) s += v[j];
        const float mean = cta_sum(s, red[turn ^= 1]) * inv_n;
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (at0 + j * step < a.n) v[j] -= mean;
        s = 0.f;
      }
#pragma unroll
      for (int j = 0; j < E; ++j) s = fmaf(v[j], v[j], s);
      return rsqrtf(fmaf(cta_sum(s, red[turn ^= 1]), inv_n, p.eps));
    };
    if (has_block) {
      const float f = post ? stats() : 1.f;
      const float* gate = !p.gate ? nullptr : p.gate + (p.gate_rows ? row / p.gate_rows * p.gate_ld : 0);
#pragma unroll
      for (int j0 = 0; j0 < E; j0 += 4) {
        float w[4], b[4], g[4];
        uint32_t raw[4] = {};
        if (post) vector(p.post_weight, j0, 1.f, w), vector(p.post_bias, j0, 0.f, b);
        vector(gate, j0, 1.f, g);
        if (!AHEAD) get(second, row, j0, raw);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x = v[j0 + j];
          if (post) x = fmaf(x * f, w[j], b[j]);
          x = fmaf(x * g[j], p.scale, AHEAD ? r[(j0 + j) % (AHEAD ? E : 1)] : value(second, raw[j]));
          v[j0 + j] = at0 + (j0 + j) * step < a.n ? x : 0.f;
        }
      }
    }
    if (a.t.p) {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (at0 + j * step < a.n) store_row<1>(a.t, row * a.t.ld + at0 + j * step, v + j);
    }
    if (!a.z.p) continue;
    const float f = stats();
#pragma unroll
    for (int j0 = 0; j0 < E; j0 += 4) {
      float w[4], b[4];
      vector(p.weight, j0, 1.f, w), vector(p.bias, j0, 0.f, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = fmaf(v[j0 + j] * f, w[j], b[j]);
        if (at0 + (j0 + j) * step < a.n) store_row<1>(a.z, row * a.z.ld + at0 + (j0 + j) * step, &x);
      }
    }
  }
}

// Rows of whole 16-byte pieces: persistent CTAs.  A thread's values of the CTA's next rows (block, residual, gate) are on
// their way to its own place in shared memory by cp.async while a row is worked on, so that no thread reads what
// another one fetched; the vectors stay in registers (8 values a thread: rows of up to 8192), since loads of them behind
// each reduction cost twice what the row does.
template <int C>
__global__ void __launch_bounds__(1024) block_norm_ring_kernel(const __grid_constant__ NormArgs a, int depth, int staged_r, int staged_g) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float red[2][32];
  int turn = 0;
  constexpr int E = 8 * C;
  const q4_norms& p = a.p;
  const int step = blockDim.x * 8, at0 = threadIdx.x * 8;
  // (a residual that does not fit beside the block is read where it is added; so is a gate that the rows share, out of L1)
  const int wide_b = a.block.p ? (a.block.f32 ? 32 : 16) : 0, wide_r = staged_r ? (a.residual.f32 ? 32 : 16) : 0;
  const int wide_g = staged_g ? 32 : 0;
  const int pieces = blockDim.x * C, off_r = pieces * wide_b, off_g = off_r + pieces * wide_r, stage = off_g + pieces * wide_g;
  const float inv_n = 1.f / static_cast<float>(a.n);
  const uint32_t base = smem_u32(ring);
  int64_t next = blockIdx.x;                   // the row to fetch
  int next_slot = 0;
  const int gate_rows = p.gate_rows > 0 ? p.gate_rows : 0x7fffffff;
  auto fetch = [&]() {
    if (next < a.rows) {
      const float* gate = wide_g ? p.gate + static_cast<int>(next) / gate_rows * p.gate_ld : nullptr;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int at = at0 + j * step, place = j * blockDim.x + threadIdx.x;
        if (at >= a.n) break;
        const uint32_t to = base + next_slot * stage;
        auto pull = [&](uint32_t dst, const char* src, int wide) {
          if (wide) cp16_once(dst, src);
          if (wide == 32) cp16_once(dst + 16, src + 16);
        };
        pull(to + place * wide_b, static_cast<const char*>(a.block.p) + (next * a.block.ld + at) * (wide_b >> 3), wide_b);
        pull(to + off_r + place * wide_r, static_cast<const char*>(a.residual.p) + (next * a.residual.ld + at) * (wide_r >> 3), wide_r);
        pull(to + off_g + place * wide_g, reinterpret_cast<const char*>(gate + at), wide_g);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    next += gridDim.x;
    if (++next_slot == depth) next_slot = 0;
  };
  auto staged = [&](const char* src, int wide, float* v) {
    if (wide == 32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = *reinterpret_cast<const float4*>(src + 16 * i);
        v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
      }
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(src);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
      }
    }
  };
  for (int s = 0; s < depth - 1; ++s) fetch();
  // the vectors: [0], [1] those of the post norm, [2], [3] the others
  constexpr bool KEEP = C == 1;
  const float* const vec[4] = {p.post_weight, p.post_bias, p.weight, p.bias};
  float kept[4][KEEP ? 8 : 1];
  auto vector = [&](int which, int at, float* w) {
    if (vec[which]) {
      load_vec<8>(vec[which], at, w);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = which & 1 ? 0.f : 1.f;
    }
  };
  if (KEEP)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at0 < a.n) vector(k, at0, kept[k]);
  // x = x f w + b
  auto affine = [&](int which, int at, float f, float* x) {
    float w[8], b[8];
    if (!KEEP) vector(which, at, w), vector(which + 1, at, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i] * f, KEEP ? kept[which][i % (KEEP ? 8 : 1)] : w[i], KEEP ? kept[which + 1][i % (KEEP ? 8 : 1)] : b[i]);
  };

  int slot = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    fetch();
    switch (depth) {
      case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
      case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
      case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
      default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
    const char* const src = ring + slot * stage;
    if (++slot == depth) slot = 0;
    float v[E];
    auto stats = [&]() {
      float s = 0.f;
      if (p.kind == Q4_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < E; ++i) s += v[i];
        const float mean = cta_sum(s, red[turn ^= 1]) * inv_n;
#pragma unroll
        for (int j = 0; j < C; ++j)
          if (at0 + j * step < a.n)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j * 8 + i] -= mean;
        s = 0.f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) s = fmaf(v[i], v[i], s);
      return rsqrtf(fmaf(cta_sum(s, red[turn ^= 1]), inv_n, p.eps));
    };
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int place = j * blockDim.x + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j * 8 + i] = 0.f;
      if (at0 + j * step < a.n) staged(wide_b ? src + place * wide_b : src + off_r + place * wide_r, wide_b ? wide_b : wide_r, v + j * 8);
    }
    if (wide_b) {
      const float f = p.post ? stats() : 1.f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        const int at = at0 + j * step, place = j * blockDim.x + threadIdx.x;
        if (at >= a.n) continue;
        float w[8];
        float* x = v + j * 8;
        if (p.post) affine(0, at, f, x);
        if (p.gate) {
          if (wide_g)
            staged(src + off_g + place * wide_g, wide_g, w);
          else
            load_vec<8>(p.gate + static_cast<int>(row) / gate_rows * p.gate_ld + at, 0, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0.f;
        if (wide_r)
          staged(src + off_r + place * wide_r, wide_r, w);
        else if (a.residual.p)
          load_row<8>(a.residual, row * a.residual.ld + at, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], p.scale, w[i]);
      }
    }
    if (a.t.p) {
#pragma unroll
      for (int j = 0; j < C; ++j)
        if (at0 + j * step < a.n) store_row<8>(a.t, row * a.t.ld + at0 + j * step, v + j * 8);
    }
    if (!a.z.p) continue;
    const float f = stats();
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int at = at0 + j * step;
      if (at >= a.n) continue;
      affine(2, at, f, v + j * 8);
      store_row<8>(a.z, row * a.z.ld + at, v + j * 8);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

bool rows16(const void* p, int64_t ld, int f32) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (f32 ? 4 : 2) % 16 == 0);
}
bool vec16(const float* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

constexpr int kBnMost = 226 * 1024;       // dynamic shared memory at most
constexpr int kBnRing = 100 * 1024;       // shared memory of an SM that the rings take, if a row is not longer

}  // namespace

cudaError_t block_norm_prepare() {
  cudaError_t e = cudaSuccess;
  for (void (*const kernel)(NormArgs, int, int, int) : {block_norm_ring_kernel<1>, block_norm_ring_kernel<2>, block_norm_ring_kernel<4>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBnMost);
  return e;
}

cudaError_t block_norm_launch(const NormArgs& a, int sms, cudaStream_t s) {
  const q4_norms& p = a.p;
  const bool wide = a.n % 8 == 0 && rows16(a.block.p, a.block.ld, a.block.f32) &&
                    rows16(a.residual.p, a.residual.ld, a.residual.f32) && rows16(a.t.p, a.t.ld, a.t.f32) &&
                    rows16(a.z.p, a.z.ld, a.z.f32) && vec16(p.post_weight) && vec16(p.post_bias) && vec16(p.gate) &&
                    (!p.gate || !p.gate_rows || p.gate_ld % 4 == 0) && vec16(p.weight) && vec16(p.bias);
  const int c = a.n <= 8192 ? 1 : a.n <= 16384 ? 2 : 4;
  const int threads_w = ((a.n + 8 * c - 1) / (8 * c) + 31) / 32 * 32;
  // bytes of a row in the ring: the block (or the residual alone), the residual, and a gate that differs from row to row
  int ctas = 1024 / threads_w;
  if (ctas > 8) ctas = 8;
  const int64_t most = static_cast<int64_t>(sms) * ctas, grid = a.rows < most ? a.rows : most;
  const int values = threads_w * c * 2, first = a.block.p ? (a.block.f32 ? 2 : 1) : 0, second = a.residual.p ? (a.residual.f32 ? 2 : 1) : 0;
  int row = values * 8 * first;
  const bool stage_r = second && (!first || 2 * (row + values * 8 * second) <= kBnMost);
  if (stage_r) row += values * 8 * second;
  const bool stage_g = first && p.gate && p.gate_rows > 0 && p.gate_rows < grid && 2 * (row + values * 16) <= kBnMost;
  if (stage_g) row += values * 16;
  if (wide) {
    int depth = kBnRing / ctas / row;
    depth = depth > 4 ? 4 : depth >= 2 ? depth : 2 * row <= kBnMost ? 2 : 1;
    void (*const kernel)(NormArgs, int, int, int) = c == 1 ? block_norm_ring_kernel<1> : c == 2 ? block_norm_ring_kernel<2> : block_norm_ring_kernel<4>;
    kernel<<<static_cast<unsigned>(grid), threads_w, depth * row, s>>>(a, depth, stage_r, stage_g);
    return cudaGetLastError();
  }
  // A value at a time, up to 32 a thread (1024 threads take 32768).  From 4096 on two rows in registers leave room for 512
  // threads: 1852 rows of 5935 in 59 us so, 64 with 1024 threads and a row; 13 rows, of which no CTA has a second, 6.1 and
  // 5.2.  2048 rows of 16383: 16 values a thread 151 us, 32 201.
  const bool ahead = a.n <= 4096 || (a.n <= 8192 && a.rows > sms);
  const int e = a.n <= 4096 || (a.n <= 8192 && !ahead) ? 8 : a.n <= 16384 ? 16 : 32;
  const int threads = ((a.n + e - 1) / e + 31) / 32 * 32;
  const int64_t room = static_cast<int64_t>(sms) * (threads < 512 ? 512 / threads : 1);
  void (*const kernel)(NormArgs) = ahead ? (e == 8 ? block_norm_any_kernel<8, 512, true> : block_norm_any_kernel<16, 512, true>)
                                   : e == 8  ? block_norm_any_kernel<8, 1024, false>
                                   : e == 16 ? block_norm_any_kernel<16, 1024, false>
                                             : block_norm_any_kernel<32, 1024, false>;
  kernel<<<static_cast<unsigned>(a.rows < room ? a.rows : room), threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace q4
