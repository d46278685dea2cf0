// The paged KV cache's building blocks shared by its kernels (sm_103a): the
// arguments, where a position lives, and what a Q8 code stands for.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_device.cuh"

namespace q4 {

// One layer's pages (include/q4.h, q4_paged_kv).
struct PagedKv {
  void* k;                  // binary16 values or Q8 codes [n_pages][n_kv][page][hd]
  void* v;
  __half* ks;               // Q8 scales [n_pages][n_kv][page][hd / 32]
  __half* vs;
  int n_pages, page_log2, n_kv, hd;
};

// The new tokens of the batch (q4_paged_batch).
struct PagedBatch {
  const int* starts;
  const int* lens;
  const int* table;
  int n_seqs, n_tokens, width;
};

// Row of the page memory ([hd] values each) that holds slot 0 of a head of a
// page; -1 for a hole.  Below 2^31 by the argument checks.
__device__ __forceinline__ int paged_row0(const PagedKv& kv, int page, int head) {
  return static_cast<unsigned>(page) < static_cast<unsigned>(kv.n_pages) ? (page * kv.n_kv + head) << kv.page_log2 : -1;
}

// The page-memory row of position p (>= 0) of sequence s for a head; -1 when
// it lies past the table or in a hole.
__device__ __forceinline__ int paged_row(const PagedKv& kv, const PagedBatch& b, int s, int p, int head) {
  const int e = p >> kv.page_log2;
  if (e >= b.width) return -1;
  const int r0 = paged_row0(kv, __ldg(b.table + static_cast<size_t>(s) * b.width + e), head);
  return r0 < 0 ? -1 : r0 + (p & ((1 << kv.page_log2) - 1));
}

// The sequence's new token rows [t0, t1) and its length, forced into range
// whatever the arrays hold: no kernel steps outside the caller's buffers.
struct SeqSpan {
  int t0, n_new, len;
};
__device__ __forceinline__ SeqSpan paged_span(const PagedKv& kv, const PagedBatch& b, int s) {
  SeqSpan r;
  r.t0 = min(max(__ldg(b.starts + s), 0), b.n_tokens);
  r.n_new = max(min(__ldg(b.starts + s + 1), b.n_tokens) - r.t0, 0);
  r.len = min(max(__ldg(b.lens + s), 0), b.width << kv.page_log2);
  return r;
}

// The sequence a token row belongs to, found by a whole warp: one 32-way
// probe of the starts per 5 bits of n_seqs (a binary search would be a chain
// of dependent loads per row).  -1 when it belongs to none.
__device__ __forceinline__ int paged_seq_of(const PagedBatch& b, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = b.n_seqs + 1;      // the last start <= row is within [lo, lo + n)
  for (;;) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    const unsigned below = __ballot_sync(~0u, i < n && __ldg(b.starts + lo + min(i, n - 1)) <= row);
    const int c = __popc(below);
    if (c == 0) return -1;
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
    if (step == 1) break;
  }
  return lo < b.n_seqs ? lo : -1;
}

// f16(code * d) of two signed 8-bit codes.  A code c as the low byte of
// 0x6400 | (c + 128) is the binary16 value 1024 + 128 + c; minus 1152 it is c
// exactly, and one binary16 multiplication by d rounds once.  pair(w, sel):
// w holds four codes + 128, sel picks two of them.
__device__ __forceinline__ __half2 q8_pair(uint32_t biased, uint32_t sel) {
  uint32_t m;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(m) : "r"(biased), "r"(0x64646464u), "r"(sel));
  return __hsub2(*reinterpret_cast<__half2*>(&m), __half2half2(__ushort_as_half(0x6480)));
}
__device__ __forceinline__ void q8_values4(uint32_t codes, __half2 d, __half2& lo, __half2& hi) {
  const uint32_t b = codes ^ 0x80808080u;
  lo = __hmul2(q8_pair(b, 0x4140), d);
  hi = __hmul2(q8_pair(b, 0x4342), d);
}

// fp32 queries enter the products as two binary16 parts, of the query times a power of two that brings its largest
// element to 2^14 .. 2^15: 22 bits of every element, or 2^-39 of the largest one (the first part rounds to 11 bits, the
// second to 11 more or to binary16's smallest step).  Without it a query of elements near 2^-12 would keep 12 bits.  A
// row's scores are scaled back with the softmax's constant.
struct QueryScale {
  float up, down;
  // most: the bits of the row's largest |element|.  A row with an infinity or a NaN stays as it is.
  __device__ __forceinline__ explicit QueryScale(uint32_t most) {
    const int top = static_cast<int>(most >> 23);
    const int e = top == 255 ? 0 : min(141 - top, 100);       // (both factors stay normal numbers, and with it the scale)
    up = __int_as_float((127 + e) << 23);
    down = __int_as_float((127 - e) << 23);
  }
};
__device__ __forceinline__ uint32_t abs_bits(float2 f) {
  return max(__float_as_uint(f.x) & 0x7fffffffu, __float_as_uint(f.y) & 0x7fffffffu);
}
// The two parts of a pair.
__device__ __forceinline__ void query_parts(float2 f, float up, __half2* hi, __half2* lo) {
  f.x *= up, f.y *= up;
  *hi = __floats2half2_rn(f.x, f.y);
  const float2 b = __half22float2(*hi);
  *lo = __floats2half2_rn(f.x - b.x, f.y - b.y);
}

// Launchers (q4_paged_cache.cu).
cudaError_t paged_write_launch(const PagedKv& kv, const PagedBatch& b, const void* k, const void* v, bool f32,
                               int64_t ld, bool q8, cudaStream_t s);
cudaError_t paged_read_launch(const PagedKv& kv, const PagedBatch& b, void* k, void* v, bool f32, int64_t ld, bool q8,
                              cudaStream_t s);

struct PagedAttnArgs {
  PagedKv kv;
  PagedBatch b;
  const void* q;
  int64_t q_ld;
  __half* out;
  int64_t out_ld;
  int group;          // query heads per value head
  uint32_t div_mul;   // row / group as row * div_mul >> div_shift (rows below 2^31, paged_attn_divisor)
  int div_shift;
  int window, sinks;
  float scale;        // log2(e) / sqrt(hd): softmax in powers of two

  __device__ __forceinline__ int token_of(int row) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(row)) * div_mul >> div_shift);
  }
  // Offset of a row of an item in buffers whose token rows are ld values apart: row r of a value head is
  // query head r % group of new token r / group.
  __device__ __forceinline__ int64_t row_at(int t0, int head, int row, int64_t ld) const {
    const int t = token_of(row);
    return static_cast<int64_t>(t0 + t) * ld + (head * group + row - t * group) * kv.hd;
  }
};
// With l = ceil(log2 group), ceil(2^(31 + l) / group) is below 2^32 and exceeds the quotient by less than 1, so row
// times it exceeds row / group * 2^(31 + l) by less than 2^31 <= 2^(31 + l) / group: the whole part is exact.
inline void paged_attn_divisor(PagedAttnArgs* a) {
  int l = 0;
  while ((1 << l) < a->group) ++l;
  a->div_shift = 31 + l;
  a->div_mul = static_cast<uint32_t>(((uint64_t{1} << a->div_shift) + a->group - 1) / a->group);
}

}  // namespace q4
