// What the products of many and of few rows share: a weight's way from its
// block to binary16, copies, activations (sm_103a).
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_prompt.cuh"

namespace q4 {

// 16 bytes to shared memory, those behind the first `bytes` as zeros.
__device__ __forceinline__ void cp16_part(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Elements of a block from its d (twice) and one word of codes (elements 4j .. 4j + 3 in the low nibbles, 16 more in the
// high ones): o[0], o[1] and o[8], o[9].  Two code bytes c as the low bytes of 0x6400 are the binary16 values
// t = 1024 + c; with the low nibbles replaced by 8, h = 1032 + 16 (c >> 4).  t - h and h / 16 - 72.5 are the nibbles less
// 8, exactly, and the product with d rounds once.  (Two permutations and two logical operations a word: they share the
// integer pipe, which paces the conversion together with the eight binary16 ones; masking each nibble apart took six.)
__device__ __forceinline__ void q4_values8(uint32_t codes, __half2 d, uint32_t* o) {
  const __half2 sixteenth = bits_h2(0x2c002c00u), m72 = bits_h2(0xd488d488u);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t t = prmt(codes, 0x64646464u, i ? 0x4342 : 0x4140), h = (t & 0xfff0fff0u) | 0x00080008u;
    o[i] = h2_bits(__hmul2(__hsub2(bits_h2(t), bits_h2(h)), d));
    o[8 + i] = h2_bits(__hmul2(__hfma2(bits_h2(h), sixteenth, m72), d));
  }
}

// The blocks of two (9 words): o[c] holds values 2c and 2c + 1 of one.
__device__ __forceinline__ void q4_first_block(const uint32_t* w, uint32_t* o) {
  const __half2 d = bits_h2(prmt(w[0], w[0], 0x1010));
#pragma unroll
  for (int j = 0; j < 4; ++j) q4_values8(__funnelshift_r(w[j], w[j + 1], 16), d, o + 2 * j);
}
__device__ __forceinline__ void q4_second_block(const uint32_t* w, uint32_t* o) {
  const __half2 d = bits_h2(prmt(w[4], w[4], 0x3232));
#pragma unroll
  for (int j = 0; j < 4; ++j) q4_values8(w[5 + j], d, o + 2 * j);
}

// t / (1 + e^z): SiLU with z = -t, and GELU's tanh form, since (1 + tanh y) / 2 = 1 / (1 + e^(-2 y)).  An exponent that
// overflows leaves 0 for every finite t.
__device__ __forceinline__ float over_1_and_exp(float t, float z) { return __fdividef(t, 1.f + __expf(z)); }

// t times the normal distribution's share below t.  The share below -|t| is r 2^(P(r) - t^2 log2(e) / 2) with r = 1 / (1 + 0.4 |t|) and
// a polynomial P that was fitted for the least relative error at all |t| <= 14 (8.6e-8): small values keep their digits, where 1 + erf
// cancels (4 % of the value at -5, all of it at -6, and a large second product brings that up).  Off by (t^2 + 9) 2^-23 of the value
// at most.  (erfcf does as well, but its registers spilled: 4000 rows of 4099 x 4128 took 185 us, with 1 + erf 138, with this 120.)
__device__ __forceinline__ float gelu(float t) {
  float r, e;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(fabsf(t), 0.4f, 1.f)));
  float p = 0.273944438f;
  p = fmaf(p, r, -1.40286124f);
  p = fmaf(p, r, 2.8012476f);
  p = fmaf(p, r, -2.51524973f);
  p = fmaf(p, r, 0.774264574f);
  p = fmaf(p, r, -0.258475393f);
  p = fmaf(p, r, 0.536042273f);
  p = fmaf(p, r, 1.4386102f);
  p = fmaf(p, r, -2.64752269f);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(t * -0.72134752f, t, p)));
  const float below = r * e;
  return t * (t < 0.f ? below : 1.f - below);
}

// The activation of N values; the choice is the same for all.
template <int N>
__device__ __forceinline__ void activate(float* t, int act) {
  switch (act) {
    case Q4_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = t[i] > 0.f || t[i] != t[i] ? t[i] : 0.f;
      break;
    case Q4_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = over_1_and_exp(t[i], -t[i]);
      break;
    case Q4_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = gelu(t[i]);
      break;
    case Q4_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = over_1_and_exp(t[i], -1.5957691f * (t[i] + 0.044715f * t[i] * t[i] * t[i]));
      break;
    default: break;
  }
}

// The kernel of few rows (q4_gemm_few.cu).  At 8 rows it takes 6.2 us for 4096 x 4096 where that of many takes 14.4, and
// 27 us for the gated 14336 x 4096 where that takes 27; a second set of 8 columns took 44 us at 16 rows, for x is staged
// again for every tile.  (The rule goes by rows alone, although the sides' times depend on the number of tiles too: from 9 rows
// on small matrices pay for it.)
constexpr int kFewRows = 8;
cudaError_t gemm_few_prepare();
cudaError_t gemm_few_launch(const GemmArgs& a, const PromptDevice& d, cudaStream_t s);

}  // namespace q4
