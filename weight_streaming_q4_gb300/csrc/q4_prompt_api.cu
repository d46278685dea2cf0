// C ABI of the operators of a prompt's layer beside its attention
// (include/q4.h): argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <mutex>

#include "q4.h"
#include "q4_device.cuh"
#include "q4_prompt.cuh"

namespace {

constexpr int kMostRows = 1 << 24, kMostOutputs = 1 << 30;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool type_ok(int type) { return type == Q4_TYPE_F32 || type == Q4_TYPE_F16; }

// Rows of `row` values of a type, ld apart, aligned to their type.
int check_rows(const void* p, int type, int64_t ld, int64_t row) {
  if (!type_ok(type) || ld < row || ld > (int64_t{1} << 31)) return Q4_ERR_ARG;
  return aligned(p, type == Q4_TYPE_F32 ? 4 : 2) ? Q4_OK : Q4_ERR_ALIGN;
}

// An output that starts where an input does has to have its rows there too.
bool rows_clash(const q4::RowsOut& out, const q4::RowsIn& in, int rows) {
  return out.p && out.p == in.p && (out.f32 != in.f32 || (rows > 1 && out.ld != in.ld));
}

#define Q4_CUDA(call)                                           \
  do {                                                          \
    cudaError_t e_ = (call);                                    \
    if (e_ != cudaSuccess) return q4::record_cuda_error(e_);    \
  } while (0)

// The current device, whose kernels are made ready on its first call.
int device_of(const q4::PromptDevice** out) {
  static std::mutex mutex;
  static q4::PromptDevice known[64];
  int dev = 0;
  Q4_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return Q4_ERR_ARG;
  std::lock_guard<std::mutex> lock(mutex);
  if (known[dev].sms == 0) {
    q4::PromptDevice d = {};
    Q4_CUDA(q4::gemm_prepare(&d));
    Q4_CUDA(q4::block_norm_prepare());
    Q4_CUDA(cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev));
    known[dev] = d;
  }
  *out = &known[dev];
  return Q4_OK;
}

int run_gemm(const void* w0, const void* w1, const uint16_t* x, int64_t x_ld, int n, int k, int rows, const float* bias0,
             const float* bias1, int act, float scale, q4::RowsIn residual, uint16_t* y, int64_t y_ld, void* stream) {
  if (!w0 || n < 1 || n > kMostOutputs || k < q4::kQK || k % q4::kQK || rows < 0 || rows > kMostRows) return Q4_ERR_ARG;
  if (act < Q4_ACT_NONE || act > Q4_ACT_GELU_TANH) return Q4_ERR_ARG;
  // (no address of the kernels needs this: matrices of 4 GB and more with such rows are untested)
  if (k % 256 && static_cast<int64_t>(n) * (k / q4::kQK) > ((int64_t{1} << 32) - 1) / q4::kBlockBytes) return Q4_ERR_ARG;
  if (!aligned(w0, 16) || (w1 && !aligned(w1, 16)) || !aligned(bias0, 4) || !aligned(bias1, 4)) return Q4_ERR_ALIGN;
  if (rows == 0) return Q4_OK;
  if (!x || !y || x_ld < k || x_ld > (int64_t{1} << 31) || y_ld < n || y_ld > (int64_t{1} << 31)) return Q4_ERR_ARG;
  if (!aligned(x, 16) || x_ld % 8 || !aligned(y, 2)) return Q4_ERR_ALIGN;
  const void* const out = y;
  if (out == x || out == w0 || out == w1 || rows_clash({y, y_ld, 0}, residual, rows)) return Q4_ERR_ARG;
  q4::GemmArgs a;
  a.w[0] = static_cast<const uint8_t*>(w0), a.w[1] = static_cast<const uint8_t*>(w1);
  a.x = reinterpret_cast<const __half*>(x), a.x_ld = x_ld;
  a.n = n, a.k = k, a.rows = rows;
  a.bias[0] = bias0, a.bias[1] = bias1;
  a.act = act, a.scale = scale, a.residual = residual;
  a.y = reinterpret_cast<__half*>(y), a.y_ld = y_ld;
  const q4::PromptDevice* d = nullptr;
  const int st = device_of(&d);
  if (st != Q4_OK) return st;
  // (a chained q4_gemv behind this product starts after it)
  q4::oneshot_chain_break(static_cast<cudaStream_t>(stream));
  Q4_CUDA(q4::gemm_launch(a, *d, static_cast<cudaStream_t>(stream)));
  return Q4_OK;
}

// 1 / (2 pi), the turns of a radian, in 2^-128.
constexpr uint64_t kTurnHigh = 0x28be60db9391054a, kTurnLow = 0x7f09d5f47d4d3770;
constexpr double kMostFreq = 1152921504606846976.;      // 2^60: the constant's last bit is 2^-5 of a unit of turns_of there

// The turns of freq radians in 2^-64, whole ones left out, rounded: freq is m 2^(e - 53) with a whole number m, and the product
// of m and the constant's 126 bits is whole too.  (A division in 64-bit floating point is off by 2^-53 of the turns, whole ones
// among them, which 2^31 positions make 2^-22.)
uint64_t turns_of(double freq) {
  int e;
  const uint64_t m = static_cast<uint64_t>(ldexp(frexp(fabs(freq), &e), 53));
  const unsigned __int128 low = static_cast<unsigned __int128>(m) * kTurnLow;
  const unsigned __int128 high = static_cast<unsigned __int128>(m) * kTurnHigh + static_cast<uint64_t>(low >> 64);
  // in 2^(e - 53 - 128), 181 bits at most
  const uint64_t word[4] = {static_cast<uint64_t>(low), static_cast<uint64_t>(high), static_cast<uint64_t>(high >> 64), 0};
  const int shift = 53 + 128 - 64 - e;      // (56 or more, as freq is 2^60 at most)
  if (shift >= 192) return 0;
  const int w = shift / 64, b = shift % 64;
  uint64_t turns = word[w] >> b | (b ? word[w + 1] << (64 - b) : 0);
  turns += word[(shift - 1) / 64] >> (shift - 1) % 64 & 1;
  return freq < 0 ? 0 - turns : turns;
}

}  // namespace

extern "C" int q4_gemm(const void* w, const uint16_t* x, int64_t x_ld, int n, int k, int rows, const q4_epilogue* ep,
                       uint16_t* y, int64_t y_ld, void* stream) {
  const q4_epilogue plain = {nullptr, Q4_ACT_NONE, 1.f, nullptr, Q4_TYPE_F16, 0};
  const q4_epilogue& e = ep ? *ep : plain;
  if (e.residual) {
    const int st = check_rows(e.residual, e.residual_type, e.residual_ld, n);
    if (st != Q4_OK) return st;
  }
  return run_gemm(w, nullptr, x, x_ld, n, k, rows, e.bias, nullptr, e.act, e.scale,
                  {e.residual, e.residual_ld, e.residual_type == Q4_TYPE_F32}, y, y_ld, stream);
}

extern "C" int q4_gemm_gated(const void* w_gate, const void* w_up, const uint16_t* x, int64_t x_ld, int n, int k, int rows,
                             const q4_gated_epilogue* ep, uint16_t* y, int64_t y_ld, void* stream) {
  if (!w_up) return Q4_ERR_ARG;
  return run_gemm(w_gate, w_up, x, x_ld, n, k, rows, ep ? ep->bias_gate : nullptr, ep ? ep->bias_up : nullptr,
                  ep ? ep->act : Q4_ACT_SILU, 1.f, {nullptr, 0, 0}, y, y_ld, stream);
}

extern "C" int q4_block_norm(const q4_norms* norms, int rows, int n, const void* block, int block_type, int64_t block_ld,
                             const void* residual, int residual_type, int64_t residual_ld, void* t, int t_type,
                             int64_t t_ld, void* z, int z_type, int64_t z_ld, void* stream) {
  if (!norms || (norms->kind != Q4_NORM_RMS && norms->kind != Q4_NORM_LAYER) || !(norms->eps >= 0.f)) return Q4_ERR_ARG;
  if (n < 1 || n > 32768 || rows < 0 || rows > kMostRows || norms->gate_rows < 0) return Q4_ERR_ARG;
  if (norms->gate && norms->gate_rows && norms->gate_ld < n) return Q4_ERR_ARG;
  for (const float* v : {norms->post_weight, norms->post_bias, norms->gate, norms->weight, norms->bias})
    if (!aligned(v, 4)) return Q4_ERR_ALIGN;
  if (rows == 0) return Q4_OK;
  if ((!block && !residual) || (!t && !z)) return Q4_ERR_ARG;
  int st = Q4_OK;
  if (block && (st = check_rows(block, block_type, block_ld, n)) != Q4_OK) return st;
  if (residual && (st = check_rows(residual, residual_type, residual_ld, n)) != Q4_OK) return st;
  if (t && (st = check_rows(t, t_type, t_ld, n)) != Q4_OK) return st;
  if (z && (st = check_rows(z, z_type, z_ld, n)) != Q4_OK) return st;
  q4::NormArgs a;
  a.p = *norms;
  a.rows = rows, a.n = n;
  a.block = {block, block_ld, block_type == Q4_TYPE_F32};
  a.residual = {residual, residual_ld, residual_type == Q4_TYPE_F32};
  a.t = {t, t_ld, t_type == Q4_TYPE_F32};
  a.z = {z, z_ld, z_type == Q4_TYPE_F32};
  if (t == z) return Q4_ERR_ARG;
  for (const q4::RowsIn& in : {a.block, a.residual})
    if (rows_clash(a.t, in, rows) || rows_clash(a.z, in, rows)) return Q4_ERR_ARG;
  const q4::PromptDevice* d = nullptr;
  if ((st = device_of(&d)) != Q4_OK) return st;
  Q4_CUDA(q4::block_norm_launch(a, d->sms, static_cast<cudaStream_t>(stream)));
  return Q4_OK;
}

extern "C" int q4_rotation_init(q4_rotation* rot, int head_dim, int rot_dim, const double* freqs, const int* axes, int style) {
  if (!rot || !freqs || head_dim < 2 || head_dim > 1024 || rot_dim < 2 || rot_dim > 2 * Q4_ROPE_PAIRS || rot_dim % 2 ||
      rot_dim > head_dim || (style != Q4_ROPE_HALVES && style != Q4_ROPE_ADJACENT))
    return Q4_ERR_ARG;
  q4_rotation r;
  memset(&r, 0, sizeof(r));
  r.head_dim = head_dim, r.rot_dim = rot_dim, r.style = style, r.n_axes = 1;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!(fabs(freqs[i]) <= kMostFreq) || (axes && (axes[i] < 0 || axes[i] >= Q4_ROPE_AXES))) return Q4_ERR_ARG;
    r.turn[i] = turns_of(freqs[i]);
    r.axis[i] = static_cast<uint8_t>(axes ? axes[i] : 0);
    if (r.axis[i] >= r.n_axes) r.n_axes = r.axis[i] + 1;
  }
  *rot = r;
  return Q4_OK;
}

extern "C" int q4_rope(const q4_rotation* rot, const q4_places* places, int inverse, int n_heads, const void* x, int x_type,
                       int64_t x_ld, void* y, int y_type, int64_t y_ld, void* stream) {
  if (!rot || !places || rot->head_dim < 2 || rot->head_dim > 1024 || rot->rot_dim < 2 || rot->rot_dim > 2 * Q4_ROPE_PAIRS ||
      rot->rot_dim % 2 || rot->rot_dim > rot->head_dim || (rot->style != Q4_ROPE_HALVES && rot->style != Q4_ROPE_ADJACENT))
    return Q4_ERR_ARG;
  if (n_heads < 1 || n_heads > 65536 || places->n_tokens < 0 || places->n_tokens > kMostRows) return Q4_ERR_ARG;
  if (places->n_tokens == 0) return Q4_OK;
  if (places->positions) {
    if (places->n_axes < rot->n_axes || places->ld < places->n_tokens) return Q4_ERR_ARG;
    for (int i = 0; i < rot->rot_dim / 2; ++i)
      if (rot->axis[i] >= places->n_axes) return Q4_ERR_ARG;
    if (!aligned(places->positions, 4)) return Q4_ERR_ALIGN;
  } else {
    if (places->n_seqs < 0 || places->n_seqs > 65535) return Q4_ERR_ARG;
    if (places->n_seqs == 0) return Q4_OK;
    if (!places->token_starts || !places->kv_lens) return Q4_ERR_ARG;
    if (!aligned(places->token_starts, 4) || !aligned(places->kv_lens, 4)) return Q4_ERR_ALIGN;
  }
  if (!x || !y) return Q4_ERR_ARG;
  const int64_t row = static_cast<int64_t>(n_heads) * rot->head_dim;
  int st = check_rows(x, x_type, x_ld, row);
  if (st != Q4_OK || (st = check_rows(y, y_type, y_ld, row)) != Q4_OK) return st;
  if (x == y && (x_type != y_type || x_ld != y_ld)) return Q4_ERR_ARG;
  q4::RopeArgs a;
  a.rot = *rot;
  a.positions = places->positions, a.positions_ld = places->ld;
  a.b = {places->token_starts, places->kv_lens, nullptr, places->n_seqs, places->n_tokens, 0};
  a.rows = places->n_tokens, a.heads = n_heads, a.inverse = inverse != 0;
  a.x = {x, x_ld, x_type == Q4_TYPE_F32};
  a.y = {y, y_ld, y_type == Q4_TYPE_F32};
  const q4::PromptDevice* d = nullptr;
  if ((st = device_of(&d)) != Q4_OK) return st;
  Q4_CUDA(q4::rope_launch(a, d->sms, static_cast<cudaStream_t>(stream)));
  return Q4_OK;
}
