// Products of many rows with Q4_0 weights, with an epilogue (sm_103a):
//   y[r][i] = f16(residual + scale * act(sum_k W[i][k] x[r][k] + bias[i])),  or  f16(act(g) * u) of two matrices.
//
// The weights are the first operand of the tensor cores, 256 rows of W per
// pair of CTAs (128 in each), and bn <= 256 rows of x the second (128 of two
// matrices' shared x).  A pair walks tiles of 256 x bn outputs in steps of 64
// columns of k:
//   copies      W blocks as they lie in memory, 256 columns at a time, and the CTA's
//               half of x's rows (128-byte swizzle), by TMA into two rings
//   conversion  a thread per row of W: nibbles to f16((q - 8) * d) in registers,
//               stored into a ring of operands in tensor memory
//   products    one thread of the leading CTA: tcgen05.mma over both CTAs, operand A
//               in tensor memory, B in shared memory, fp32 sums in tensor memory
//   epilogue    a thread per row of W: bias, activation, residual, one rounding
// Weights never exist in binary16 outside tensor memory, so that a step moves
// 36 bytes of shared memory per row of W where an unpacked operand would move
// 128, and with a pair each CTA fetches half of x only.
//
// With few tiles, a cluster of 2, 4 or 8 CTAs shares one tile: each pair takes
// a part of k and the parts are added, in a fixed order, over distributed
// shared memory.
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_prompt.cuh"
#include "q4_tensor.cuh"

namespace q4 {

namespace {

constexpr uint32_t kGmWaitLimit = 1u << 21;
__device__ int g_status_gm;

constexpr int kGmThreads = 512;
constexpr int kGmConvert = 4, kGmEpilogue = 12;     // first warps of these roles
constexpr int kGmMaxX = 16, kGmMaxW = 8;            // stages of the rings at most
constexpr int kGmMaxSplit = 4;                      // pairs of a cluster at most
constexpr int kGmSmem = 232448 - 1024;              // dynamic shared memory at most

template <int MATS, bool RAGGED>
struct Gm {
  // bytes between staged rows of W: 256 columns, and where rows do not start 16-byte aligned the pieces around them
  // (a multiple of 16 whose 16-byte loads by 8 threads side by side fall in different banks)
  static constexpr int PITCH = RAGGED ? 176 : 144;
  static constexpr int W_STAGE = MATS * 128 * PITCH;
  static constexpr int NA = 8 / MATS;               // operand ring in tensor memory: steps of 64 columns
  static constexpr int A_COL = 256, A_STEP = 32 * MATS;
  static constexpr int D_STEP = 128;                // columns between the two matrices' sums
};

struct GmMaps {
  CUtensorMap w[2], x;
};

struct GmPlan {
  int bn;             // rows of x of a tile, a multiple of 32 (what a pair's product takes)
  int split;          // pairs that share a tile
  int nx, nw;         // stages of the rings
  int tok_tiles, row_tiles, group;      // tiles; tiles of x that follow one another before the next rows of W
};

struct GmCtl {
  uint64_t w_full[kGmMaxW], w_empty[kGmMaxW], x_full[kGmMaxX], x_empty[kGmMaxX], a_full[8], a_empty[8];
  uint64_t d_full, d_empty;
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(GmCtl) <= 1024, "control data fits its place");

// A wait that gives up at once when one has run out before: the roles walk on and the kernel ends (its results do not
// count: the status word says so).
__device__ __forceinline__ void gm_wait(GmCtl* c, uint64_t* bar, uint32_t parity) {
  if (mbar_test_wait(bar, parity)) return;
  const uint32_t limit = *reinterpret_cast<volatile int*>(&c->dead) ? 0 : kGmWaitLimit;
  if (!mbar_wait_bounded(bar, parity, limit)) {
    *reinterpret_cast<volatile int*>(&c->dead) = 1;
    atomicOr(&g_status_gm, ST_FULL_TIMEOUT);
  }
}
__device__ __forceinline__ void gm_wait_warp(GmCtl* c, uint64_t* bar, uint32_t parity) {
  gm_wait(c, bar, parity);
  __syncwarp();
}
// Before the CTA ends: what is still in flight (nothing is, unless a wait has run out), whatever ran out before.
__device__ __forceinline__ void gm_drain(uint64_t* bar, uint32_t parity) {
  if (!mbar_wait_bounded(bar, parity, kGmWaitLimit)) atomicOr(&g_status_gm, ST_DRAIN_TIMEOUT);
  __syncwarp();
}

// A place in a ring of n stages and the parity of its current turn.
struct Ring {
  int slot = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void step(int n) {
    if (++slot == n) slot = 0, turn ^= 1;
  }
  // the turn's parity of the one before: what frees the slot (the first turn finds it free)
  __device__ __forceinline__ uint32_t before() const { return turn ^ 1; }
};

// The tiles of one pair: tile t is `tok` of x and `row` of W.
struct GmTile {
  int row, tok;
};
__device__ __forceinline__ GmTile gm_tile(const GmPlan& p, int64_t t) {
  const int64_t in_group = static_cast<int64_t>(p.group) * p.row_tiles;
  const int g = static_cast<int>(t / in_group);
  const int64_t rest = t - g * in_group;
  const int width = min(p.group, p.tok_tiles - g * p.group);
  GmTile r;
  r.row = static_cast<int>(rest / width);
  r.tok = g * p.group + static_cast<int>(rest - static_cast<int64_t>(r.row) * width);
  return r;
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Elements of a block from its d (twice) and one word of codes (elements 4j .. 4j + 3 in the low nibbles, 16 more in the
// high ones): o[0], o[1] and o[8], o[9].  A nibble q as the low bits of 0x6400 is the binary16 value 1024 + q, a high
// one 1024 + 16 q: one exact operation each leaves q - 8, and the product with d rounds once.
__device__ __forceinline__ void q4_values8(uint32_t codes, __half2 d, uint32_t* o) {
  const __half2 bias = bits_h2(0x64086408u), sixteenth = bits_h2(0x2c002c00u), m72 = bits_h2(0xd480d480u);
  const uint32_t lo = codes & 0x0f0f0f0fu, hi = codes & 0xf0f0f0f0u;
  o[0] = h2_bits(__hmul2(__hsub2(bits_h2(prmt(lo, 0x64646464u, 0x4140)), bias), d));
  o[1] = h2_bits(__hmul2(__hsub2(bits_h2(prmt(lo, 0x64646464u, 0x4342)), bias), d));
  o[8] = h2_bits(__hmul2(__hfma2(bits_h2(prmt(hi, 0x64646464u, 0x4140)), sixteenth, m72), d));
  o[9] = h2_bits(__hmul2(__hfma2(bits_h2(prmt(hi, 0x64646464u, 0x4342)), sixteenth, m72), d));
}

// Two blocks (9 words) into a row's 64 values: o[c] holds values 2c and 2c + 1.
__device__ __forceinline__ void q4_values64(const uint32_t* w, uint32_t* o) {
  const __half2 d0 = bits_h2(prmt(w[0], w[0], 0x1010)), d1 = bits_h2(prmt(w[4], w[4], 0x3232));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    q4_values8(__funnelshift_r(w[j], w[j + 1], 16), d0, o + 2 * j);
    q4_values8(w[5 + j], d1, o + 16 + 2 * j);
  }
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
      for (int i = 0; i < N; ++i) t[i] = t[i] / (1.f + __expf(-t[i]));
      break;
    case Q4_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = 0.5f * t[i] * (1.f + erff(t[i] * 0.70710678f));
      break;
    case Q4_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = 0.5f * t[i] * (1.f + tanhf(0.79788456f * (t[i] + 0.044715f * t[i] * t[i] * t[i])));
      break;
    default: break;
  }
}

// N columns of sums of this thread's row i of W, of x's rows row0 .. : epilogue and store.
template <int MATS, int N>
__device__ __forceinline__ void finish(const GemmArgs& a, int i, int row0, int rows, float* g, float* u, float bg, float bu) {
#pragma unroll
  for (int c = 0; c < N; ++c) g[c] += bg;
  activate<N>(g, a.act);
#pragma unroll
  for (int c = 0; c < N; ++c) g[c] = MATS == 2 ? g[c] * (u[c] + bu) : g[c] * a.scale;
  if (i >= a.n) return;
  if (MATS == 1 && a.residual.p) {
    const int64_t at = row0 * a.residual.ld + i;
    if (a.residual.f32) {
      const float* r = static_cast<const float*>(a.residual.p) + at;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < rows) g[c] += r[c * a.residual.ld];
    } else {
      const __half* r = static_cast<const __half*>(a.residual.p) + at;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < rows) g[c] += __half2float(r[c * a.residual.ld]);
    }
  }
  __half* y = a.y + row0 * a.y_ld + i;
#pragma unroll
  for (int c = 0; c < N; ++c)
    if (c < rows) y[c * a.y_ld] = __float2half_rn(g[c]);
}

template <int MATS, bool RAGGED>
__global__ void __launch_bounds__(kGmThreads, 1)
    gemm_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ GmMaps maps, const __grid_constant__ GmPlan p) {
  using G = Gm<MATS, RAGGED>;
  extern __shared__ char smem_raw[];
  GmCtl* c = reinterpret_cast<GmCtl*>(smem_raw);
  // (the swizzle's period; the same offset in every CTA of the cluster)
  const uint32_t base = (smem_u32(smem_raw) + sizeof(GmCtl) + 1023) & ~1023u;
  char* s_x = smem_raw + (base - smem_u32(smem_raw));
  const int x_stage = p.bn * 64;                       // half of the rows, 128 bytes each
  char* s_w = s_x + p.nx * x_stage;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
  const uint32_t rank = cluster_rank(), half = rank & 1, leader = rank & ~1u;
  const uint32_t pair_mask = 3u << leader;
  const int part = static_cast<int>(rank >> 1);        // of k
  const int nb = a.k / kQK, units = (nb + 7) / 8;      // blocks, and groups of 256 columns, of a row
  const int u0 = units * part / p.split, u1 = units * (part + 1) / p.split;
  const int steps = (min(nb, u1 * 8) - u0 * 8 + 1) / 2;        // of 64 columns, of a tile
  const int64_t tiles = static_cast<int64_t>(p.tok_tiles) * p.row_tiles;
  const int64_t first = blockIdx.x / (2 * p.split), stride = gridDim.x / (2 * p.split);

  if (tid == 0) {
    for (int i = 0; i < kGmMaxW; ++i) mbar_init(&c->w_full[i], 1), mbar_init(&c->w_empty[i], 4 * MATS);
    for (int i = 0; i < kGmMaxX; ++i) mbar_init(&c->x_full[i], 1), mbar_init(&c->x_empty[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&c->a_full[i], 8 * MATS), mbar_init(&c->a_empty[i], 1);
    mbar_init(&c->d_full, 1), mbar_init(&c->d_empty, 8);
    c->dead = 0;
    fence_mbar_init();
  }
  if (warp == 3) tm2_alloc(&c->tmem, 512);
  tm_before();
  __syncthreads();
  cluster_sync();
  tm_after();
  const uint32_t tmem = __shfl_sync(~0u, c->tmem, 0);

  if (warp == 0) {
    // ---------------------------------------------------------------- copies of W
    Ring r;
    int64_t n = 0;
    for (int64_t t = first; t < tiles; t += stride) {
      const int w0 = gm_tile(p, t).row * 256 + half * 128;
      for (int u = u0; u < u1; ++u, ++n) {
        if (n >= p.nw) gm_wait_warp(c, &c->w_empty[r.slot], r.before());
        char* to = s_w + r.slot * G::W_STAGE;
        if (!RAGGED) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&c->w_full[r.slot], G::W_STAGE);
            for (int m = 0; m < MATS; ++m) tma_load_2d(to + m * 128 * G::PITCH, &maps.w[m], u * 144, w0, &c->w_full[r.slot]);
          }
        } else {
          // a row's blocks with the bytes around them up to 16-byte boundaries, but not past the matrix's end: the
          // few bytes behind the last boundary there are copied by hand
          const int64_t row_bytes = static_cast<int64_t>(nb) * kBlockBytes, end = row_bytes * a.n;
          const int bytes = min(8, nb - u * 8) * kBlockBytes;
          uint32_t total = 0;
#pragma unroll
          for (int i = 0; i < 4 * MATS; ++i) {
            const int row = w0 + (i & 3) * 32 + lane;
            if (row >= a.n) continue;
            const int64_t at = row * row_bytes + u * 144, lo = at & ~int64_t{15};
            const int64_t hi = min((at + bytes + 15) & ~int64_t{15}, end & ~int64_t{15});
            total += static_cast<uint32_t>(max(hi - lo, int64_t{0}));
            if (at + bytes > (end & ~int64_t{15})) {
              char* d = to + ((i >> 2) * 128 + (i & 3) * 32 + lane) * G::PITCH;
              for (int64_t b = max(end & ~int64_t{15}, lo); b < at + bytes; b += 2)
                *reinterpret_cast<uint16_t*>(d + (b - lo)) = *reinterpret_cast<const uint16_t*>(a.w[i >> 2] + b);
            }
          }
          fence_async();
          total = __reduce_add_sync(~0u, total);
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&c->w_full[r.slot], total);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4 * MATS; ++i) {
            const int row = w0 + (i & 3) * 32 + lane;
            if (row >= a.n) continue;
            const int64_t at = row * row_bytes + u * 144, lo = at & ~int64_t{15};
            const int64_t hi = min((at + bytes + 15) & ~int64_t{15}, end & ~int64_t{15});
            if (hi > lo)
              bulk_g2s(to + ((i >> 2) * 128 + (i & 3) * 32 + lane) * G::PITCH, a.w[i >> 2] + lo, static_cast<uint32_t>(hi - lo),
                       &c->w_full[r.slot]);
          }
        }
        __syncwarp();
        r.step(p.nw);
      }
    }
    for (int64_t u = n > p.nw ? n - p.nw : 0; u < n; ++u) gm_drain(&c->w_full[u % p.nw], static_cast<uint32_t>(u / p.nw) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- copies of x
    Ring r;
    int64_t n = 0;
    for (int64_t t = first; t < tiles; t += stride) {
      const int x0 = gm_tile(p, t).tok * p.bn + half * (p.bn / 2);
      for (int s = 0; s < steps; ++s, ++n) {
        if (n >= p.nx) gm_wait_warp(c, &c->x_empty[r.slot], r.before());
        if (lane == 0) {
          if (half == 0) mbar_arrive_expect_tx(&c->x_full[r.slot], 2 * x_stage);
          tma2_load_2d(s_x + r.slot * x_stage, &maps.x, u0 * 256 + s * 64, x0, cluster_addr(&c->x_full[r.slot], leader));
        }
        __syncwarp();
        r.step(p.nx);
      }
    }
    if (half == 0)      // (both CTAs' copies)
      for (int64_t u = n > p.nx ? n - p.nx : 0; u < n; ++u) gm_drain(&c->x_full[u % p.nx], static_cast<uint32_t>(u / p.nx) & 1);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- products
    if (half == 0) {
      const uint32_t idesc = mma_idesc(p.bn, false, 256);
      const bool one = elect_one();
      Ring rx, ra, rd;
      for (int64_t t = first; t < tiles; t += stride) {
        if (t != first) gm_wait_warp(c, &c->d_empty, rd.before());
        tm_after();
        for (int s = 0; s < steps; ++s) {
          gm_wait_warp(c, &c->x_full[rx.slot], rx.turn);
          gm_wait_warp(c, &c->a_full[ra.slot], ra.turn);
          tm_after();
          if (one) {
            const uint64_t b = mma_sdesc(smem_u32(s_x) + rx.slot * x_stage, 0);
            const uint32_t at = tmem + G::A_COL + ra.slot * G::A_STEP;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int m = 0; m < MATS; ++m)
                tm2_mma_ts(tmem + m * G::D_STEP, at + m * 32 + k * 8, b + 2 * k, idesc, s > 0 || k > 0);
            tm2_commit(&c->a_empty[ra.slot], pair_mask);
            tm2_commit(&c->x_empty[rx.slot], pair_mask);
          }
          __syncwarp();
          rx.step(p.nx);
          ra.step(G::NA);
        }
        if (one) tm2_commit(&c->d_full, pair_mask);
        __syncwarp();
        rd.step(1);
      }
    }
  } else if (warp >= kGmConvert && warp < kGmEpilogue) {
    // ---------------------------------------------------------------- conversion
    // Warps q + 4 and q + 8 hold rows 32 q .. of the CTA: of one matrix the groups of 256 columns in turn, of two a
    // matrix each.
    const int q = warp & 3, mine = (warp - kGmConvert) >> 2;
    const int mat = MATS == 2 ? mine : 0;
    const uint32_t to = tmem + G::A_COL + mat * 32 + (static_cast<uint32_t>(q * 32) << 16);
    Ring rw, ra;
    int64_t n = 0, step = 0;
    for (int64_t t = first; t < tiles; t += stride) {
      const int w0 = gm_tile(p, t).row * 256 + half * 128 + q * 32 + lane;
      const int shift = RAGGED ? static_cast<int>((static_cast<int64_t>(w0) * nb * kBlockBytes) & 15) : 0;
      for (int u = u0; u < u1; ++u, ++n) {
        const int here = min(4, (nb - u * 8 + 1) / 2);
        if (MATS == 1 && (n & 1) != mine) {
          rw.step(p.nw);
          for (int j = 0; j < here; ++j) ra.step(G::NA);
          step += here;
          continue;
        }
        gm_wait_warp(c, &c->w_full[rw.slot], rw.turn);
        const char* row = s_w + rw.slot * G::W_STAGE + (mat * 128 + q * 32 + lane) * G::PITCH;
        uint32_t w[40];
        if (!RAGGED) {
#pragma unroll
          for (int i = 0; i < 9; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + 16 * i);
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&c->w_empty[rw.slot]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= here) break;
          uint32_t o[32];
          if (RAGGED) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(row + (shift & ~3) + 36 * j);
            uint32_t v[10];
#pragma unroll
            for (int i = 0; i < 10; ++i) v[i] = src[i];
            const uint32_t by = (shift & 2) * 8;
#pragma unroll
            for (int i = 0; i < 9; ++i) w[9 * j + i] = __funnelshift_r(v[i], v[i + 1], by);
            if (j == here - 1) {
              __syncwarp();
              if (lane == 0) mbar_arrive(&c->w_empty[rw.slot]);
            }
          }
          q4_values64(w + 9 * j, o);
          if (RAGGED && u * 8 + 2 * j + 1 >= nb) {
#pragma unroll
            for (int i = 16; i < 32; ++i) o[i] = 0;      // (a row of an odd number of blocks)
          }
          if (step >= G::NA) gm_wait_warp(c, &c->a_empty[ra.slot], ra.before());
          tm_after();
          tm_st32(to + ra.slot * G::A_STEP, o);
          tm_st_wait();
          tm_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(cluster_addr(&c->a_full[ra.slot], leader));
          ra.step(G::NA);
          ++step;
        }
        rw.step(p.nw);
      }
    }
  } else if (warp >= kGmEpilogue) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;
    const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16);
    Ring rd;
    for (int64_t t = first; t < tiles; t += stride) {
      const GmTile tile = gm_tile(p, t);
      gm_wait_warp(c, &c->d_full, rd.turn);
      tm_after();
      rd.step(1);
      if (p.split > 1) break;
      const int i = tile.row * 256 + half * 128 + q * 32 + lane;
      const float bg = a.bias[0] && i < a.n ? __ldg(a.bias[0] + i) : 0.f, bu = MATS == 2 && a.bias[1] && i < a.n ? __ldg(a.bias[1] + i) : 0.f;
      for (int b = 0; b < p.bn; b += 32) {
        const int row0 = tile.tok * p.bn + b, rows = min(a.rows - row0, 32);
        if (rows <= 0) break;
        uint32_t g[32], u[32];
        tm_ld32(from + b, g);
        if (MATS == 2) tm_ld32(from + G::D_STEP + b, u);
        tm_ld_wait(g);
        if (MATS == 2) tm_ld_waited(u);
        finish<MATS, 32>(a, i, row0, rows, reinterpret_cast<float*>(g), reinterpret_cast<float*>(u), bg, bu);
      }
      tm_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&c->d_empty, leader));
    }
  }
  __syncwarp();
  // The barriers that the last products' ends are told to are not gone before they are.
  if (warp == 3) {
    int64_t mine = 0;
    for (int64_t t = first; t < tiles; t += stride) mine += steps;
    for (int64_t s = mine > G::NA ? mine - G::NA : 0; s < mine; ++s)
      gm_drain(&c->a_empty[s % G::NA], static_cast<uint32_t>(s / G::NA) & 1);
    for (int64_t s = mine > p.nx ? mine - p.nx : 0; s < mine; ++s)
      gm_drain(&c->x_empty[s % p.nx], static_cast<uint32_t>(s / p.nx) & 1);
  }
  __syncwarp();
  tm_before();
  __syncthreads();
  tm_after();

  if (p.split > 1 && first < tiles) {
    // The pairs' parts of the one tile: pair j adds up columns [j w, (j + 1) w).  The others' parts of them lie in the
    // rings' place, [pair][matrix][column][row of W] fp32.
    const int w = p.bn / p.split;
    const int q = warp & 3, own = part;
    float* recv = reinterpret_cast<float*>(s_x);
    const uint32_t from = tmem + (static_cast<uint32_t>(q * 32) << 16);
    cluster_sync();
    if (warp >= kGmEpilogue) {
      for (int j = 0; j < p.split; ++j) {
        if (j == own) continue;
        const uint32_t to = cluster_addr(recv, 2 * j + half);
        for (int m = 0; m < MATS; ++m)
          for (int b = 0; b < w; b += 32) {
            uint32_t v[32];
            tm_ld32(from + m * G::D_STEP + j * w + b, v);
            tm_ld_wait(v);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (b + e < w)
                asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + (((own * MATS + m) * w + b + e) * 128 + q * 32 + lane) * 4),
                             "r"(v[e])
                             : "memory");
          }
      }
    }
    cluster_sync();
    if (warp >= kGmEpilogue) {
      const GmTile tile = gm_tile(p, first);
      const int i = tile.row * 256 + half * 128 + q * 32 + lane;
      const float bg = a.bias[0] && i < a.n ? __ldg(a.bias[0] + i) : 0.f, bu = MATS == 2 && a.bias[1] && i < a.n ? __ldg(a.bias[1] + i) : 0.f;
      for (int b = 0; b < w; b += 32) {
        const int col = own * w + b, row0 = tile.tok * p.bn + col;
        const int rows = min(min(w - b, a.rows - row0), 32);
        if (rows <= 0) break;
        uint32_t v[MATS][32];
        float sum[MATS][32];
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          tm_ld32(from + m * G::D_STEP + col, v[m]);
          tm_ld_wait(v[m]);
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[m][e] = 0.f;
          for (int j = 0; j < p.split; ++j) {
            const float* src = recv + ((j * MATS + m) * w + b) * 128 + q * 32 + lane;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e < rows) sum[m][e] += j == own ? __uint_as_float(v[m][e]) : src[e * 128];
          }
        }
        finish<MATS, 32>(a, i, row0, rows, sum[0], sum[MATS - 1], bg, bu);
      }
    }
    tm_before();
    __syncthreads();
  }
  cluster_sync();
  if (warp == 3) {
    tm_after();
    tm2_free(tmem, 512);
  }
}

// ------------------------------------------------------------------ host

// Time of a plan in cycles, roughly: waves of tiles, each as long as the slowest of its products, its conversion and its
// copies, and its epilogue.
GmPlan plan(const GemmArgs& a, int sms, int mats, int w_stage) {
  const int pairs = sms / 2, units = (a.k + 255) / 256, most = 256 / mats;
  GmPlan best = {};
  best.row_tiles = (a.n + 255) / 256;
  double least = 0;
  const int fewest = (a.rows + most - 1) / most;
  for (int i = 0; i < 24; ++i) {
    const int tok = fewest + i;
    const int bn = ((a.rows + tok - 1) / tok + 31) / 32 * 32;
    if (i > 0 && (bn < 64 || (a.rows + bn - 1) / bn != tok)) break;
    const int64_t tiles = static_cast<int64_t>(tok) * best.row_tiles;
    for (int split = 1; split <= kGmMaxSplit; split *= 2) {
      if (split > 1 && (tiles * split > pairs || units < 2 * split)) break;
      const int64_t waves = (tiles + pairs - 1) / pairs;
      const double step = 2. * bn * mats > 260. * mats ? 2. * bn * mats : 260. * mats;
      const double time = waves * ((units + split - 1) / split * 4 * step + 1500 + 8. * bn * mats) + (split > 1 ? 3000 + 4. * bn * mats : 0);
      if (least == 0 || time < least) least = time, best.bn = bn, best.split = split, best.tok_tiles = tok;
    }
  }
  // rows of x that stay in L2 while W passes by
  const int64_t group = (int64_t{48} << 20) / (static_cast<int64_t>(best.bn) * a.k * 2);
  best.group = group < 1 ? 1 : group > best.tok_tiles ? best.tok_tiles : static_cast<int>(group);
  best.nw = best.bn * mats <= 128 ? 6 : 4;
  if (best.nw * w_stage > 140 * 1024) best.nw = 140 * 1024 / w_stage;
  const int room = kGmSmem - 2048 - best.nw * w_stage;
  best.nx = room / (best.bn * 64);
  if (best.nx > kGmMaxX) best.nx = kGmMaxX;
  return best;
}

template <int MATS, bool RAGGED>
cudaError_t launch(const GemmArgs& a, int sms, cudaStream_t s) {
  using G = Gm<MATS, RAGGED>;
  const GmPlan p = plan(a, sms, MATS, G::W_STAGE);
  GmMaps maps = {};
  if (!encode_f16_tile(&maps.x, a.x, a.rows, a.k, a.x_ld, p.bn / 2)) return cudaErrorInvalidValue;
  for (int m = 0; m < MATS && !RAGGED; ++m)
    if (!encode_bytes_tile(&maps.w[m], a.w[m], a.n, static_cast<int64_t>(a.k / kQK) * kBlockBytes, 144, 128)) return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>(p.tok_tiles) * p.row_tiles;
  const int64_t clusters = p.split > 1 || tiles < sms / 2 ? tiles : sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * p.split));
  cfg.blockDim = dim3(kGmThreads);
  cfg.dynamicSmemBytes = kGmSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2 * p.split, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_kernel<MATS, RAGGED>, a, maps, p);
}

template <int MATS, bool RAGGED>
cudaError_t prepare() {
  return cudaFuncSetAttribute(gemm_kernel<MATS, RAGGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGmSmem);
}

}  // namespace

cudaError_t gemm_prepare() {
  const cudaError_t e[4] = {prepare<1, false>(), prepare<1, true>(), prepare<2, false>(), prepare<2, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t gemm_launch(const GemmArgs& a, int sms, cudaStream_t s) {
  const bool ragged = a.k % 256 != 0;
  if (a.w[1]) return ragged ? launch<2, true>(a, sms, s) : launch<2, false>(a, sms, s);
  return ragged ? launch<1, true>(a, sms, s) : launch<1, false>(a, sms, s);
}

cudaError_t gemm_read_status(int* out) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status_gm, sizeof(int));
  if (e != cudaSuccess || *out == 0) return e;
  return cudaMemcpyToSymbol(g_status_gm, &zero, sizeof(int));
}

}  // namespace q4
