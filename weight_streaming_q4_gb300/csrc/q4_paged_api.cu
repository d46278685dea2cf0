// C ABI of the paged KV cache (include/q4.h): argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "q4.h"
#include "q4_device.cuh"
#include "q4_paged_sched.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool heads_ok(int n_kv, int hd) { return n_kv >= 1 && n_kv <= 1024 && hd >= 64 && hd <= 256 && hd % 64 == 0; }

bool group_ok(int n_q, int n_kv) { return n_q >= n_kv && n_q % n_kv == 0 && n_q / n_kv <= 64; }

// Checks and converts the cache and the batch.  *empty: nothing to do.
int check_batch(const q4_paged_kv* kv, const q4_paged_batch* b, q4::PagedKv* k, q4::PagedBatch* pb, bool* empty) {
  if (!kv || !b || !kv->k_pages || !kv->v_pages) return Q4_ERR_ARG;
  if (kv->type != Q4_KV_F16 && kv->type != Q4_KV_Q8) return Q4_ERR_ARG;
  if (!heads_ok(kv->n_kv_heads, kv->head_dim) || kv->n_pages < 1) return Q4_ERR_ARG;
  int log2 = 4;
  while (log2 < 8 && (1 << log2) != kv->page_size) ++log2;
  if ((1 << log2) != kv->page_size) return Q4_ERR_ARG;
  if ((static_cast<int64_t>(kv->n_pages) * kv->n_kv_heads << log2) > INT32_MAX) return Q4_ERR_ARG;
  if (kv->type == Q4_KV_Q8 && (!kv->k_scales || !kv->v_scales)) return Q4_ERR_ARG;
  if (b->n_seqs < 0 || b->n_seqs > 65535 || b->n_tokens < 0 || b->table_width < 1 || b->max_new < 0) return Q4_ERR_ARG;
  // (the key tiles of a row tile's heads are counted in 32 bits)
  const int64_t positions = static_cast<int64_t>(b->table_width) << log2;
  if (positions > (1 << 30) || positions * kv->n_kv_heads > INT32_MAX) return Q4_ERR_ARG;
  if (!aligned(kv->k_pages, 16) || !aligned(kv->v_pages, 16)) return Q4_ERR_ALIGN;
  if (kv->type == Q4_KV_Q8 && (!aligned(kv->k_scales, 16) || !aligned(kv->v_scales, 16))) return Q4_ERR_ALIGN;
  *empty = b->n_seqs == 0 || b->n_tokens == 0;
  if (!*empty) {
    if (!b->token_starts || !b->kv_lens || !b->page_table) return Q4_ERR_ARG;
    if (!aligned(b->token_starts, 4) || !aligned(b->kv_lens, 4) || !aligned(b->page_table, 4)) return Q4_ERR_ALIGN;
  }
  *k = {kv->k_pages, kv->v_pages, reinterpret_cast<__half*>(kv->k_scales), reinterpret_cast<__half*>(kv->v_scales),
        kv->n_pages, log2, kv->n_kv_heads, kv->head_dim};
  *pb = {b->token_starts, b->kv_lens, b->page_table, b->n_seqs, b->n_tokens, b->table_width};
  return Q4_OK;
}

// Positions that the page table has entries for (at most 2^30).
int positions_of(const q4::PagedAttnArgs& a) { return a.b.width << a.kv.page_log2; }

// A buffer of rows of `row` values of a type, ld apart.
int check_rows(const void* p, int type, int64_t ld, int64_t row) {
  if (!p || (type != Q4_TYPE_F32 && type != Q4_TYPE_F16) || ld < row || ld > (int64_t{1} << 31)) return Q4_ERR_ARG;
  if (!aligned(p, 16) || ld * (type == Q4_TYPE_F32 ? 4 : 2) % 16) return Q4_ERR_ALIGN;
  return Q4_OK;
}

#define Q4_CUDA(call)                                           \
  do {                                                          \
    cudaError_t e_ = (call);                                    \
    if (e_ != cudaSuccess) return q4::record_cuda_error(e_);    \
  } while (0)

// CTAs of the attention kernels on the current device (one per SM), which are
// made ready on its first call.
int attn_grid(int* grid) {
  static std::mutex mutex;
  static int sms[64];
  int dev = 0;
  Q4_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return Q4_ERR_ARG;
  std::lock_guard<std::mutex> lock(mutex);
  if (sms[dev] == 0) {
    int n = 0;
    Q4_CUDA(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    Q4_CUDA(q4::paged_tile_prepare());
    Q4_CUDA(q4::paged_rows_prepare());
    sms[dev] = n < q4::kPagedMaxCtas ? n : q4::kPagedMaxCtas;
  }
  *grid = sms[dev];
  return Q4_OK;
}

}  // namespace

extern "C" int q4_paged_write(const q4_paged_kv* kv, const q4_paged_batch* batch, const void* k, const void* v, int type,
                              int64_t ld, void* stream) {
  q4::PagedKv pk;
  q4::PagedBatch pb;
  bool empty = false;
  int st = check_batch(kv, batch, &pk, &pb, &empty);
  if (st != Q4_OK || empty) return st;
  const int64_t row = static_cast<int64_t>(pk.n_kv) * pk.hd;
  if ((st = check_rows(k, type, ld, row)) != Q4_OK || (st = check_rows(v, type, ld, row)) != Q4_OK) return st;
  Q4_CUDA(q4::paged_write_launch(pk, pb, k, v, type == Q4_TYPE_F32, ld, kv->type == Q4_KV_Q8,
                                 static_cast<cudaStream_t>(stream)));
  return Q4_OK;
}

extern "C" int q4_paged_read(const q4_paged_kv* kv, const q4_paged_batch* batch, void* k, void* v, int type, int64_t ld,
                             void* stream) {
  q4::PagedKv pk;
  q4::PagedBatch pb;
  bool empty = false;
  int st = check_batch(kv, batch, &pk, &pb, &empty);
  if (st != Q4_OK || empty) return st;
  const int64_t row = static_cast<int64_t>(pk.n_kv) * pk.hd;
  if ((st = check_rows(k, type, ld, row)) != Q4_OK || (st = check_rows(v, type, ld, row)) != Q4_OK) return st;
  Q4_CUDA(q4::paged_read_launch(pk, pb, k, v, type == Q4_TYPE_F32, ld, kv->type == Q4_KV_Q8,
                                static_cast<cudaStream_t>(stream)));
  return Q4_OK;
}

extern "C" size_t q4_attn_paged_workspace_bytes(int n_q_heads, int n_kv_heads, int head_dim) {
  if (!heads_ok(n_kv_heads, head_dim) || !group_ok(n_q_heads, n_kv_heads)) return 0;
  // two slots per CTA of up to 256 rows (head_dim above 128: 128): outputs, maximum and sum in fp32
  const size_t rows = head_dim <= 128 ? 256 : 128;
  return q4::kPagedRecordBytes + 2 * q4::kPagedMaxCtas * rows * (head_dim + 2) * sizeof(float);
}

extern "C" int q4_attn_paged(const q4_paged_kv* kv, const q4_paged_batch* batch, const void* q, int q_type, int64_t q_ld,
                             int n_q_heads, int window, int sinks, uint16_t* out, int64_t out_ld, void* workspace,
                             size_t workspace_bytes, void* stream) {
  q4::PagedAttnArgs a;
  bool empty = false;
  int st = check_batch(kv, batch, &a.kv, &a.b, &empty);
  if (st != Q4_OK) return st;
  if (!group_ok(n_q_heads, a.kv.n_kv) || window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return Q4_ERR_ARG;
  // (the kernels count a sequence's query rows of a head, and a window back from a negative position, in an int)
  if (static_cast<int64_t>(a.b.n_tokens) * (n_q_heads / a.kv.n_kv) > (1 << 30)) return Q4_ERR_ARG;
  if (empty) return Q4_OK;
  const int64_t row = static_cast<int64_t>(n_q_heads) * a.kv.hd;
  if ((st = check_rows(q, q_type, q_ld, row)) != Q4_OK) return st;
  if ((st = check_rows(out, Q4_TYPE_F16, out_ld, row)) != Q4_OK) return st;
  if (!workspace) return Q4_ERR_ARG;
  if (!aligned(workspace, 16)) return Q4_ERR_ALIGN;
  if (workspace_bytes < q4_attn_paged_workspace_bytes(n_q_heads, a.kv.n_kv, a.kv.hd)) return Q4_ERR_OOM;
  a.q = q;
  a.q_ld = q_ld;
  a.out = reinterpret_cast<__half*>(out);
  a.out_ld = out_ld;
  a.group = n_q_heads / a.kv.n_kv;
  q4::paged_attn_divisor(&a);
  // (a window over the whole table is none; the kernels' sums of positions and windows stay within an int)
  const int capacity = positions_of(a);
  a.window = window < capacity ? window : 0;
  a.sinks = a.window ? (sinks < capacity ? sinks : capacity) : 0;
  a.scale = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(a.kv.hd)));
  int grid = 0;
  if ((st = attn_grid(&grid)) != Q4_OK) return st;
  const bool f32 = q_type == Q4_TYPE_F32, q8 = kv->type == Q4_KV_Q8;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(batch->max_new) * a.group;
  // Up to 32 query rows of a head: a tcgen05 tile's 128 rows would be mostly empty.  8B heads, 8 sequences of 1000 to
  // 4096 positions, rows kernel against tile kernel: 20 rows 32.1 us and 44.5 (Q8), 32.5 and 38.2 (binary16), 32 rows
  // 37.9 and 46.4, 38.9 and 43.3; 64 rows, two items a head for the rows kernel, 59.9 and 48.1, 63.0 and 45.1.
  // 64 sequences of the 70B heads over Q8: 8 rows 127 and 310, 16 176 and 323, 32 285 and 373.
  if (rows <= 32)
    Q4_CUDA(q4::paged_rows_launch(a, f32, q8, static_cast<int>(rows), workspace, grid, s));
  else
    Q4_CUDA(q4::paged_tile_launch(a, f32, q8, workspace, grid, s));
  return Q4_OK;
}
