// Products of many rows with Q4_0 weights, with an epilogue (sm_103a):
//   y[r][i] = f16(residual + scale * act(sum_k W[i][k] x[r][k] + bias[i])),  or  f16(act(g) * u) of two matrices.
//
// The weights are the first operand of the tensor cores, 256 rows of W per
// pair of CTAs (128 in each), and bn <= 256 rows of x the second (192 with two
// matrices).  A pair walks tiles of 256 x bn outputs along k:
//   copies      W as it lies in memory, 256 columns at a time, by 16-byte cp.async; the
//               CTA's half of x's rows by tensor copies (128-byte swizzle): two rings
//   conversion  a thread per row of W: nibbles to f16((q - 8) * d) in registers,
//               stored into a ring of operands in tensor memory
//   products    one thread of the leading CTA: tcgen05.mma over both CTAs, operand A
//               in tensor memory, B in shared memory, fp32 sums in tensor memory
//   epilogue    a thread per row of W: bias, activation, residual, one rounding
// Weights never exist in binary16 outside tensor memory, so that a step of 64
// columns moves 36 bytes of shared memory per row of W where an unpacked operand
// would move 128 in and out, and with a pair each CTA fetches half of x only.  W's blocks
// are converted again for every bn rows of x: about 340 cycles of a scheduler
// per 32 rows and 64 columns (106 instructions, 64 of them on the half-rate
// binary16 pipe), beside products of 2 bn (two matrices 4 bn) cycles a step, which
// is why tiles are as wide as tensor memory lets them be and the plan weighs
// both times.
//
// With few tiles, a cluster of 4, 8 or 16 CTAs shares one tile: each pair takes a part
// of k and the parts are added, in a fixed order, over distributed shared memory.
//
// The tensor cores cut the fp32 sums at every step instead of rounding them:
// 1.7e-5 of a sum of 14336 products, far below the rounding to binary16.
//
// Measured in a graph, other inputs every time: 2048 rows, gated 14336 x 4096 289 us, 1666 TFLOP/s (88 % of a library
// matrix product's rate); 4096 x 14336 with a residual 154 us, 1557 (two rounds of tiles where 1.68 would do); 300 rows, gated
// 28672 x 8192 171 us, 1646.  16 rows, gated 14336 x 4096 25 to 28 us, 2.4 to 2.7 TB/s of W: the conversion bounds it, and 56 of
// the 76 pairs have a tile.
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_frag.cuh"
#include "q4_gemm.cuh"
#include "q4_tensor.cuh"

namespace q4 {

namespace {

constexpr uint32_t kGmWaitLimit = 1u << 21;
__device__ int g_status_gm;

constexpr int kGmThreads = 768;
constexpr int kGmConvert = 4, kGmEpilogue = 20;     // first warps of these roles
constexpr int kGmSplits = 4;                        // 1, 2, 4 or 8 pairs share a tile
constexpr int kGmTeams = 5;                         // of four warps, that finish the last tile
constexpr int kGmMaxX = 16, kGmMaxW = 8;            // stages of the rings at most
constexpr int kGmSmem = 232448 - 1024;              // dynamic shared memory at most
// Columns of a tile's sums up to which stages are twice as long: 9 rows of 4096 x 4096 take 14.6 us so and 16.2
// otherwise; from 128 on there is no tensor memory for three such stages.
constexpr int kGmWide = 64;
constexpr int kGmCols = 512;                        // columns of tensor memory
constexpr int kGmMaxA = 7;                          // operand stages at most

// WIDE: for few rows of x, where waits and signals cost more than the products, stages twice as long.
template <int MATS, bool RAGGED, bool WIDE>
struct Gm {
  // a staged row of W: the 16-byte pieces that hold 256 columns, and the bytes between rows (a multiple of 16 whose
  // 16-byte loads by 8 threads side by side fall in different banks)
  static constexpr int PIECES = RAGGED ? 10 : 9;
  static constexpr int PITCH = RAGGED ? 176 : 144;
  static constexpr int W_STAGE = MATS * 128 * PITCH;
  // steps of 64 columns of k of a stage of x and of a stage of operands, and the latter's columns of tensor memory
  static constexpr int XS = WIDE ? 4 : 2, AS = XS / MATS, A_COLS = AS * MATS * 32;
};

struct GmPlan {
  int bn;             // rows of x of a tile, a multiple of 32 (what a pair's product takes)
  int split;          // pairs that share a tile
  int sums;           // tiles whose sums have a place: with two, one is finished while the next one is formed
  int na, nx, nw;     // stages of the rings: operands in tensor memory, x, W
  int tok_tiles, row_tiles, group;      // tiles; tiles of x that follow one another before the next rows of W
};

struct GmCtl {
  uint64_t w_full[kGmMaxW], w_empty[kGmMaxW], x_full[kGmMaxX], x_empty[kGmMaxX], a_full[kGmMaxA], a_empty[kGmMaxA];
  uint64_t d_full[2], d_empty[2];
  uint64_t d_last;     // the last tile's sums are whole
  uint32_t tmem;
  int dead;
};
static_assert(sizeof(GmCtl) <= 1024, "control data fits its place");

// A wait that gives up at once when one has run out before: the roles walk on and the kernel ends (its results do not
// count: the status word says so).
__device__ __forceinline__ void gm_wait_one(GmCtl* c, uint64_t* bar, uint32_t parity) {
  if (mbar_test_wait(bar, parity)) return;
  for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i)
    if (i >= kGmWaitLimit || *reinterpret_cast<volatile int*>(&c->dead)) {
      *reinterpret_cast<volatile int*>(&c->dead) = 1;
      atomicOr(&g_status_gm, ST_FULL_TIMEOUT);
      break;
    }
}
__device__ __forceinline__ void gm_wait(GmCtl* c, uint64_t* bar, uint32_t parity) {
  gm_wait_one(c, bar, parity);
  __syncwarp();
}

// Before the CTA ends: what is still in flight (nothing is, unless a wait has run out), whatever ran out before.
__device__ __forceinline__ void gm_drain(uint64_t* bar, uint32_t parity) {
  if (!mbar_wait_bounded(bar, parity, kGmWaitLimit)) atomicOr(&g_status_gm, ST_DRAIN_TIMEOUT);
  __syncwarp();
}

// A place in a ring of n stages and the parity of its current turn.  Waiting for turn ^ 1 is waiting for the end of the
// turn before (a new barrier counts as having had one).
struct Ring {
  int slot = 0;
  uint32_t turn = 0;
  __device__ __forceinline__ void step(int n, int by = 1) {
    slot += by;
    if (slot >= n) slot -= n, turn ^= 1;
  }
};

// The tiles of one pair: tile t is rows 256 row .. of W and x0 .. of x, bn of them (the last ones fewer, in steps of 32).
struct GmTile {
  int row, x0, bn;
};
__device__ __forceinline__ GmTile gm_tile(const GmPlan& p, int rows, int64_t t) {
  const int64_t in_group = static_cast<int64_t>(p.group) * p.row_tiles;
  const int g = static_cast<int>(t / in_group);
  const int64_t rest = t - g * in_group;
  const int width = min(p.group, p.tok_tiles - g * p.group);
  GmTile r;
  r.row = static_cast<int>(rest / width);
  r.x0 = (g * p.group + static_cast<int>(rest - static_cast<int64_t>(r.row) * width)) * p.bn;
  r.bn = min(p.bn, (rows - r.x0 + 31) & ~31);
  return r;
}

// Step J (of the four of a staged row's 256 columns): its 9 words out of the 16-byte pieces that hold them.
template <int J>
__device__ __forceinline__ void staged_words(const char* row, uint32_t* w) {
  uint32_t v[12];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint4 f = *reinterpret_cast<const uint4*>(row + 32 * J + 16 * i);
    v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
  }
#pragma unroll
  for (int i = 0; i < 9; ++i) w[i] = v[J + i];
}

// The residual of N rows of x from row0 on (`rows` of them there), at this thread's row i of W.  The whole warp calls it, and
// has come together again behind it: instructions on tensor memory follow, which want every lane.
template <int N>
__device__ __forceinline__ void load_residual(const GemmArgs& a, int i, int row0, int rows, float* r) {
  if (i < a.n) {
    const int64_t at = row0 * a.residual.ld + i;
    if (a.residual.f32) {
      const float* p = static_cast<const float*>(a.residual.p) + at;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < rows) r[c] = p[c * a.residual.ld];
    } else {
      const __half* p = static_cast<const __half*>(a.residual.p) + at;
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < rows) r[c] = __half2float(p[c * a.residual.ld]);
    }
  }
  __syncwarp();
}

// N columns of sums of this thread's row i of W, of x's rows row0 .. : epilogue and store.  The whole warp, as load_residual.
template <int MATS, int N>
__device__ __forceinline__ void finish(const GemmArgs& a, int i, int row0, int rows, float* g, float* u, const float* r, float bg, float bu) {
#pragma unroll
  for (int c = 0; c < N; ++c) g[c] += bg;
  activate<N>(g, a.act);
#pragma unroll
  for (int c = 0; c < N; ++c) g[c] = MATS == 2 ? g[c] * (u[c] + bu) : a.residual.p ? fmaf(g[c], a.scale, r[c]) : g[c] * a.scale;
  if (i < a.n) {
    __half* y = a.y + row0 * a.y_ld + i;
    if (rows >= N) {
#pragma unroll
      for (int c = 0; c < N; ++c) {
        *y = __float2half_rn(g[c]);
        y += a.y_ld;
      }
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < rows) y[c * a.y_ld] = __float2half_rn(g[c]);
    }
  }
  __syncwarp();
}

template <int MATS, bool RAGGED, bool WIDE>
__global__ void __launch_bounds__(kGmThreads, 1)
    gemm_kernel(const __grid_constant__ GemmArgs a, const __grid_constant__ CUtensorMap x_map, const __grid_constant__ GmPlan p) {
  using G = Gm<MATS, RAGGED, WIDE>;
  extern __shared__ char smem_raw[];
  GmCtl* c = reinterpret_cast<GmCtl*>(smem_raw);
  // (the swizzle's period; the same offset in every CTA of the cluster)
  const uint32_t base = (smem_u32(smem_raw) + sizeof(GmCtl) + 1023) & ~1023u;
  char* s_x = smem_raw + (base - smem_u32(smem_raw));
  const int x_step = p.bn * 64, x_stage = G::XS * x_step;      // half of the rows, 128 bytes each, a step
  char* s_w = s_x + p.nx * x_stage;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
  const uint32_t rank = cluster_rank(), half = rank & 1, leader = rank & ~1u;
  const uint32_t pair_mask = 3u << leader;
  const int part = static_cast<int>(rank >> 1);        // of k
  const int nb = a.k / kQK, units = (nb + 7) / 8;      // blocks, and groups of 256 columns, of a row
  const int u0 = units * part / p.split, u1 = units * (part + 1) / p.split;
  const int64_t tiles = static_cast<int64_t>(p.tok_tiles) * p.row_tiles;
  const int64_t first = blockIdx.x / (2 * p.split), stride = gridDim.x / (2 * p.split);

  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kGmMaxW; ++i) mbar_init(&c->w_full[i], 64), mbar_init(&c->w_empty[i], 16);
    for (int i = 0; i < kGmMaxX; ++i) mbar_init(&c->x_full[i], 1), mbar_init(&c->x_empty[i], 1);
    for (int i = 0; i < kGmMaxA; ++i) mbar_init(&c->a_full[i], 8 * G::AS * MATS), mbar_init(&c->a_empty[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&c->d_full[i], 1), mbar_init(&c->d_empty[i], 8);
    mbar_init(&c->d_last, 1);
    c->dead = 0;
    fence_mbar_init();
  }
  if (warp == 2) tm2_alloc(&c->tmem, 512);
  tm_before();
  __syncthreads();
  // (the copies of W need no other CTA: they do not wait for it)
  cluster_arrive();
  griddep_wait();
  if (warp != 0 && warp != 3) cluster_wait();
  tm_after();
  const uint32_t tmem = __shfl_sync(~0u, c->tmem, 0);
  const int sums = p.bn * MATS;                        // columns of a tile's sums
  const uint32_t t_a = tmem + p.sums * sums;           // the operand stages

  if (warp == 0 || warp == 3) {
    // ---------------------------------------------------------------- copies of W
    // Two warps, a matrix each or half of the rows each: 8 threads to the first 128 bytes of a row, the rest of 16 or
    // 32 rows at a time behind them.
    constexpr int ROWS = MATS == 2 ? 128 : 64, REST = G::PIECES - 8;
    const int which = warp == 3, mat = MATS == 2 ? which : 0, r0 = MATS == 2 ? 0 : 64 * which;
    const int64_t row_bytes = static_cast<int64_t>(nb) * kBlockBytes, end = row_bytes * a.n;
    const uint8_t* const w = a.w[mat];
    const uint32_t to0 = smem_u32(s_w) + (mat * 128 + r0) * G::PITCH;
    Ring r;
    for (int64_t t = first; t < tiles; t += stride) {
      const int w0 = gm_tile(p, a.rows, t).row * 256 + half * 128 + r0;
      // every byte of the pieces lies in the matrix: those of the last row's last columns end last
      const bool whole = (w0 + ROWS - 1) * row_bytes + (units - 1) * 144 + G::PIECES * 16 <= end;
      for (int u = u0; u < u1; ++u) {
        gm_wait(c, &c->w_empty[r.slot], r.turn ^ 1);
        const uint32_t to = to0 + r.slot * G::W_STAGE;
        const uint32_t to_a = to + (lane >> 3) * G::PITCH + (lane & 7) * 16, to_b = to + (lane / REST) * G::PITCH + 128 + lane % REST * 16;
        // (where rows do not start 16-byte aligned, the bytes around them up to such boundaries)
        auto start = [&](int64_t at) { return RAGGED ? at & ~int64_t{15} : at; };
        if (whole) {
          int64_t at = (w0 + (lane >> 3)) * row_bytes;
          const uint8_t* const src = w + u * 144 + (lane & 7) * 16;
#pragma unroll 8
          for (int i = 0; i < ROWS; i += 4, at += 4 * row_bytes) cp16(to_a + i * G::PITCH, src + start(at));
          at = (w0 + lane / REST) * row_bytes;
#pragma unroll
          for (int i = 0; i < ROWS; i += 32 / REST, at += 32 / REST * row_bytes)
            cp16(to_b + i * G::PITCH, w + u * 144 + 128 + lane % REST * 16 + start(at));
        } else {
          auto copy = [&](uint32_t dst, int row, int piece) {
            const int64_t at = start((w0 + row) * row_bytes) + u * 144 + piece * 16;
            const int64_t left = w0 + row < a.n ? end - at : 0;
            const int bytes = static_cast<int>(left < 0 ? 0 : left > 16 ? 16 : left);
            cp16_part(dst, w + (bytes ? at : 0), bytes);
          };
          for (int i = 0; i < ROWS; i += 4) copy(to_a + i * G::PITCH, i + (lane >> 3), lane & 7);
          for (int i = 0; i < ROWS; i += 32 / REST) copy(to_b + i * G::PITCH, i + lane / REST, 8 + lane % REST);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&c->w_full[r.slot])) : "memory");
        r.step(p.nw);
      }
    }
    // the last copies have landed before the CTA ends
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    cluster_wait();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- copies of x
    Ring r;
    int64_t n = 0;
    for (int64_t t = first; t < tiles; t += stride) {
      const GmTile tile = gm_tile(p, a.rows, t);
      const int x0 = tile.x0 + half * (tile.bn / 2);
      for (int s = u0 * 4; s < u1 * 4; s += G::XS, ++n) {      // (past the end of a row: zeros)
        gm_wait(c, &c->x_empty[r.slot], r.turn ^ 1);
        if (lane == 0) {
          if (half == 0) mbar_arrive_expect_tx(&c->x_full[r.slot], 2 * x_stage);
          const uint32_t full = cluster_addr(&c->x_full[r.slot], leader);
#pragma unroll
          for (int i = 0; i < G::XS; ++i) tma2_load_2d(s_x + r.slot * x_stage + i * x_step, &x_map, (s + i) * 64, x0, full);
        }
        __syncwarp();
        r.step(p.nx);
      }
    }
    if (half == 0)      // (both CTAs' copies)
      for (int64_t u = n > p.nx ? n - p.nx : 0; u < n; ++u) gm_drain(&c->x_full[u % p.nx], static_cast<uint32_t>(u / p.nx) & 1);
  } else if (warp == 2) {
    // ---------------------------------------------------------------- products
    if (half == 0 && elect_one()) {
      Ring rx, ra, rd;
      for (int64_t t = first; t < tiles; t += stride) {
        const uint32_t idesc = mma_idesc(gm_tile(p, a.rows, t).bn, false, 256);
        const uint32_t d = tmem + rd.slot * sums;
        gm_wait_one(c, &c->d_empty[rd.slot], rd.turn ^ 1);
        for (int u = u0; u < u1; ++u) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i % G::XS == 0) gm_wait_one(c, &c->x_full[rx.slot], rx.turn);
            if (i % G::AS == 0) {
              gm_wait_one(c, &c->a_full[ra.slot], ra.turn);
              tm_after();
            }
            const uint64_t b = mma_sdesc(smem_u32(s_x) + rx.slot * x_stage + i % G::XS * x_step, 0);
            const uint32_t at = t_a + ra.slot * G::A_COLS + i % G::AS * (32 * MATS);
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
              for (int k = 0; k < 4; ++k) tm2_mma_ts(d + m * p.bn, at + m * 32 + k * 8, b + 2 * k, idesc, u > u0 || i > 0 || k > 0);
            if ((i + 1) % G::AS == 0) {
              tm2_commit(&c->a_empty[ra.slot], pair_mask);
              ra.step(p.na);
            }
            if ((i + 1) % G::XS == 0) {
              tm2_commit(&c->x_empty[rx.slot], pair_mask);
              rx.step(p.nx);
            }
          }
        }
        // (the last tile has a barrier of its own: the converting warps, which finish it too, have waited for no turn of d_full
        // before, and a parity alone does not tell its last turn from the one two before)
        tm2_commit(t + stride < tiles ? &c->d_full[rd.slot] : &c->d_last, pair_mask);
        rd.step(p.sums);
      }
    }
  } else if (warp >= kGmConvert && warp < kGmEpilogue) {
    // ---------------------------------------------------------------- conversion
    // Four warps hold rows 32 q .. of the CTA.  Of one matrix each takes one of the four 64 columns of every 256, of
    // two matrices two of one of them.
    const int q = warp & 3, mine = (warp - kGmConvert) >> 2;
    const int mat = MATS == 2 ? mine & 1 : 0;
    const int j0 = MATS == 2 ? mine >> 1 : mine;        // its first step of 256 columns
    const uint32_t to = t_a + j0 % G::AS * (32 * MATS) + mat * 32 + (static_cast<uint32_t>(q * 32) << 16);
    const char* const row0 = s_w + (mat * 128 + q * 32 + lane) * G::PITCH;
    const uint32_t full0 = cluster_addr(&c->a_full[0], leader);
    Ring rw, ra;
    ra.step(p.na, j0 / G::AS);
    for (int64_t t = first; t < tiles; t += stride) {
      const int w0 = gm_tile(p, a.rows, t).row * 256 + half * 128 + q * 32 + lane;
      const int shift = RAGGED ? static_cast<int>((static_cast<int64_t>(w0) * nb * kBlockBytes) & 15) : 0;
      for (int u = u0; u < u1; ++u) {
        gm_wait(c, &c->w_full[rw.slot], rw.turn);
        const char* row = row0 + rw.slot * G::W_STAGE;
#pragma unroll
        for (int i = 0; i < MATS; ++i) {
          const int j = j0 + 2 * i;
          uint32_t w[9], o[32];
          if (RAGGED) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(row + (shift & ~3) + 36 * j);
            const uint32_t by = (shift & 2) * 8;
            uint32_t v = src[0];
#pragma unroll
            for (int e = 0; e < 9; ++e) {
              const uint32_t next = src[e + 1];
              w[e] = __funnelshift_r(v, next, by);
              v = next;
            }
          } else {
            switch (j) {
              case 0: staged_words<0>(row, w); break;
              case 1: staged_words<1>(row, w); break;
              case 2: staged_words<2>(row, w); break;
              default: staged_words<3>(row, w); break;
            }
          }
          q4_first_block(w, o);
          q4_second_block(w, o + 16);
          if (RAGGED) {
            // (a row's last blocks: what lies behind them in memory is not its own)
            const int left = nb - u * 8 - 2 * j;
            if (left < 2) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e >= 16 || left < 1) o[e] = 0;
            }
          }
          if (i == MATS - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->w_empty[rw.slot]);
          }
          gm_wait(c, &c->a_empty[ra.slot], ra.turn ^ 1);
          tm_after();
          tm_st32(to + ra.slot * G::A_COLS, o);
          tm_st_wait();
          tm_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(full0 + ra.slot * 8);
          ra.step(p.na, MATS == 2 ? 2 / G::AS : 4 / G::AS);
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
      const GmTile tile = gm_tile(p, a.rows, t);
      const int i = tile.row * 256 + half * 128 + q * 32 + lane;
      const float bg = a.bias[0] && i < a.n ? __ldg(a.bias[0] + i) : 0.f, bu = MATS == 2 && a.bias[1] && i < a.n ? __ldg(a.bias[1] + i) : 0.f;
      const int last = min(tile.bn, a.rows - tile.x0);
      const bool res = MATS == 1 && a.residual.p;
      // (the tile's residual comes to L2 meanwhile: 8 rows of x a time, this warp's 32 values of each)
      if (res && i - lane < a.n)
        for (int b = lane >> 2; b < last; b += 8) {
          const int size = a.residual.f32 ? 4 : 2, at = i - lane + (lane & 3) * 32 / size;
          if (at < min(a.n, i - lane + 32))
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.residual.p) + ((tile.x0 + b) * a.residual.ld + at) * size));
        }
      if (t + stride >= tiles) break;                  // (the last one is every warp's)
      float ra[16], rb[16];
      if (res) load_residual<16>(a, i, tile.x0, last, ra);
      gm_wait(c, &c->d_full[rd.slot], rd.turn);
      tm_after();
      const uint32_t at = from + rd.slot * sums;
      auto chunk = [&](int b, const float* r, float* next) {
        uint32_t g[16], u[16];
        tm_ld16(at + b, g);
        if (MATS == 2) tm_ld16(at + p.bn + b, u);
        if (res && b + 16 < last) load_residual<16>(a, i, tile.x0 + b + 16, last - b - 16, next);
        tm_ld16_wait(g);
        if (MATS == 2) tm_ld16_waited(u);
        finish<MATS, 16>(a, i, tile.x0 + b, last - b, reinterpret_cast<float*>(g), reinterpret_cast<float*>(u), r, bg, bu);
      };
      for (int b = 0; b < last; b += 32) {
        chunk(b, ra, rb);
        if (b + 16 < last) chunk(b + 16, rb, ra);
      }
      tm_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_addr(&c->d_empty[rd.slot], leader));
      rd.step(p.sums);
    }
  }
  __syncwarp();
  // The barriers that the last products' ends are told to are not gone before they are.  (Behind d_last every turn of theirs but
  // the last has ended, or its stage could not have been filled again: a parity then tells the last one.)  A lane to a barrier:
  // one after the other they took 0.7 to 1.2 us.
  if (warp == 3) {
    const bool of_x = lane < kGmMaxX;
    const int slot = lane % kGmMaxX, ring = of_x ? p.nx : p.na;
    const int64_t turns = ((tiles - 1 - first) / stride + 1) * (u1 - u0) * (4 / (of_x ? G::XS : G::AS)) - slot;
    const uint32_t parity = static_cast<uint32_t>((turns - 1) / ring) & 1;
    gm_wait(c, &c->d_last, 0);
    if (slot < ring && turns > 0 && !mbar_wait_bounded(of_x ? &c->x_empty[slot] : &c->a_empty[slot], parity, kGmWaitLimit))
      atomicOr(&g_status_gm, ST_DRAIN_TIMEOUT);
  }
  __syncwarp();

  // The last tile (with a split: the only one) is finished by the converting warps too, 16 rows of x at a time.
  const int64_t before = (tiles - 1 - first) / stride;       // this pair's tiles before it
  const GmTile tile = gm_tile(p, a.rows, first + before * stride);
  const int q = warp & 3, team = (warp - kGmConvert) >> 2;
  const int i = tile.row * 256 + half * 128 + q * 32 + lane;
  const uint32_t from = tmem + static_cast<uint32_t>(before % p.sums) * sums + (static_cast<uint32_t>(q * 32) << 16);
  float bg = 0.f, bu = 0.f;
  if (warp >= kGmConvert) {
    if (a.bias[0] && i < a.n) bg = __ldg(a.bias[0] + i);
    if (MATS == 2 && a.bias[1] && i < a.n) bu = __ldg(a.bias[1] + i);
    gm_wait(c, &c->d_last, 0);
    tm_after();
  }
  if (p.split == 1) {
    const int last = min(tile.bn, a.rows - tile.x0);
    if (warp >= kGmConvert)
      for (int b = team * 16; b < last; b += kGmTeams * 16) {
        float r[16];
        if (MATS == 1 && a.residual.p) load_residual<16>(a, i, tile.x0 + b, last - b, r);
        uint32_t g[16], u[16];
        tm_ld16(from + b, g);
        if (MATS == 2) tm_ld16(from + p.bn + b, u);
        tm_ld16_wait(g);
        if (MATS == 2) tm_ld16_waited(u);
        finish<MATS, 16>(a, i, tile.x0 + b, last - b, reinterpret_cast<float*>(g), reinterpret_cast<float*>(u), r, bg, bu);
      }
  } else {
    // The pairs' parts: pair j adds up columns [j w, (j + 1) w).  The others' parts of them lie in the rings' place,
    // [pair][matrix][column][row of W] fp32.
    const int w = p.bn / p.split, own = part, chunks = (w + 15) / 16;
    float* recv = reinterpret_cast<float*>(s_x);
    cluster_sync();
    if (warp >= kGmConvert)
      for (int e = team; e < p.split * MATS * chunks; e += kGmTeams) {
        const int j = e / (MATS * chunks), m = e / chunks % MATS, b = e % chunks * 16;
        if (j == own) continue;
        const uint32_t to = cluster_addr(recv, 2 * j + half) + (((own * MATS + m) * w + b) * 128 + q * 32 + lane) * 4;
        uint32_t v[16];
        tm_ld16(from + m * p.bn + j * w + b, v);
        tm_ld16_wait(v);
#pragma unroll
        for (int col = 0; col < 16; ++col)
          if (b + col < w) asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + col * 512), "r"(v[col]) : "memory");
      }
    cluster_sync();
    if (warp >= kGmConvert)
      for (int b = team * 16; b < w; b += kGmTeams * 16) {
        const int col = own * w + b, row0 = tile.x0 + col, rows = min(min(w - b, a.rows - row0), 16);
        if (rows <= 0) break;
        float sum[MATS][16], r[16];
        if (MATS == 1 && a.residual.p) load_residual<16>(a, i, row0, rows, r);
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
          uint32_t v[16];
          tm_ld16(from + m * p.bn + col, v);
          tm_ld16_wait(v);
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[m][e] = 0.f;
          for (int j = 0; j < p.split; ++j) {
            const float* src = recv + ((j * MATS + m) * w + b) * 128 + q * 32 + lane;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < rows) sum[m][e] += j == own ? __uint_as_float(v[e]) : src[e * 128];
          }
        }
        finish<MATS, 16>(a, i, row0, rows, sum[0], sum[MATS - 1], r, bg, bu);
      }
  }
  __syncwarp();
  tm_before();
  __syncthreads();
  cluster_sync();
  if (warp == 2) {
    tm_after();
    tm2_free(tmem, 512);
  }
}

// ------------------------------------------------------------------ host

// Time of a plan in cycles, roughly: rounds of tiles, each as long as the slower of its products and its conversion, and
// its epilogue where nothing is formed meanwhile.  The conversion's 370 (two matrices 600) cycles a step decide between
// narrow and wide tiles: 500 rows of 4096 x 14336 46.3 us with 370 and 49.2 with 300, 500 rows of the gated 28672 x 8192
// 344 us with 740 and 326 with 600; 300 rows of that 262 us with tiles of at most 128 rows of x, 184 with up to 192.  Eight pairs to a
// tile (7 such clusters fit the GPU): 44 rows of the gated 277 x 27648 38 us, with four 60; 33 rows of 1024 x 8192 11.9 and
// 13.3, of 1024 x 4096 the same; 200 rows of 1024 x 8192 17.2 as one tile of 8 pairs and 15.4 as three of four.
GmPlan plan(const GemmArgs& a, const PromptDevice& d, int mats, int w_stage) {
  const int units = (a.k - 1) / 256 + 1, most = mats == 2 ? 192 : 256;
  const double convert = (mats == 2 ? 600. : 370.) * (a.k % 256 ? 1.2 : 1.);
  GmPlan best = {};
  best.row_tiles = (a.n + 255) / 256;
  double least = 0;
  for (int bn = 32; bn <= most; bn += 32) {
    const int tok = (a.rows + bn - 1) / bn;
    if (bn > 32 && (a.rows + bn - 33) / (bn - 32) == tok) continue;      // (a narrower tile does as well)
    const int64_t tiles = static_cast<int64_t>(tok) * best.row_tiles;
    for (int log = 0; log < kGmSplits; ++log) {
      const int split = 1 << log;
      if (log > 0 && (tiles > d.clusters[log] || units < 2 * split)) break;
      const int64_t waves = (tiles + d.clusters[log] - 1) / d.clusters[log];
      const double step = 2. * bn * mats > convert ? 2. * bn * mats : convert;
      const double time = waves * ((units + split - 1) / split * 4 * step + (bn * mats > 128 ? 12. * bn * mats : 0)) + (log ? (3000 + 4. * bn * mats) * (log == 3 ? 1.5 : 1.) : 0);
      if (least == 0 || time < least) least = time, best.bn = bn, best.split = split, best.tok_tiles = tok;
    }
  }
  // rows of x that stay in L2 while W passes by
  const int64_t group = (int64_t{48} << 20) / (static_cast<int64_t>(best.bn) * a.k * 2);
  best.group = group < 1 ? 1 : group > best.tok_tiles ? best.tok_tiles : static_cast<int>(group);
  const int sums = best.bn * mats;
  best.sums = sums <= 128 ? 2 : 1;
  const bool wide = sums <= kGmWide;
  best.na = (kGmCols - best.sums * sums) / (wide ? 128 : 64);
  if (best.na > kGmMaxA) best.na = kGmMaxA;
  // (what shared memory holds beside two to four stages of x)
  best.nw = sums <= 128 ? 6 : 4;
  if (best.nw * w_stage > 140 * 1024) best.nw = 140 * 1024 / w_stage;
  const int room = kGmSmem - 2048 - best.nw * w_stage;
  best.nx = room / (best.bn * (wide ? 256 : 128));
  if (best.nx > kGmMaxX) best.nx = kGmMaxX;
  return best;
}

cudaLaunchConfig_t config(int clusters, int split, cudaLaunchAttribute* at) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * split));
  cfg.blockDim = dim3(kGmThreads);
  cfg.dynamicSmemBytes = kGmSmem;
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = 2 * split, at->val.clusterDim.y = 1, at->val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

template <int MATS, bool RAGGED>
cudaError_t launch(const GemmArgs& a, const PromptDevice& d, cudaStream_t s) {
  const GmPlan p = plan(a, d, MATS, Gm<MATS, RAGGED, false>::W_STAGE);
  CUtensorMap x_map;
  if (!encode_f16_tile(&x_map, a.x, a.rows, a.k, a.x_ld, p.bn / 2)) return cudaErrorInvalidValue;
  const int64_t tiles = static_cast<int64_t>(p.tok_tiles) * p.row_tiles;
  const int clusters = static_cast<int>(tiles < d.clusters[0] ? tiles : d.clusters[0]);
  void (*const kernel)(GemmArgs, CUtensorMap, GmPlan) = p.bn * MATS <= kGmWide ? gemm_kernel<MATS, RAGGED, true> : gemm_kernel<MATS, RAGGED, false>;
  cudaLaunchAttribute at[2];
  cudaLaunchConfig_t cfg = config(clusters, p.split, at);
  cfg.stream = s;
  // It may start while the kernel before it on the stream ends (its CTAs take their places and wait before they touch
  // global memory): 1 to 2 us less in a chain of products.  Where several CTAs share an SM, as in the kernels of few
  // rows, norms and rotations, the waiting ones took more than that.
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, x_map, p);
}

template <int MATS, bool RAGGED, bool WIDE>
cudaError_t prepare(PromptDevice* d) {
  cudaError_t e = cudaFuncSetAttribute(gemm_kernel<MATS, RAGGED, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kGmSmem);
  // (clusters of 16 CTAs are no portable size)
  if (e == cudaSuccess) e = cudaFuncSetAttribute(gemm_kernel<MATS, RAGGED, WIDE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int log = 0; e == cudaSuccess && log < kGmSplits; ++log) {
    cudaLaunchAttribute at;
    const cudaLaunchConfig_t cfg = config(1, 1 << log, &at);
    e = cudaOccupancyMaxActiveClusters(&d->clusters[log], gemm_kernel<MATS, RAGGED, WIDE>, &cfg);
    if (e == cudaSuccess && d->clusters[log] < 1 && log < 3) e = cudaErrorInvalidConfiguration;
  }
  return e;
}

}  // namespace

cudaError_t gemm_prepare(PromptDevice* d) {
  const cudaError_t e[9] = {prepare<1, false, false>(d), prepare<1, true, false>(d), prepare<2, false, false>(d), prepare<2, true, false>(d),
                            prepare<1, false, true>(d),  prepare<1, true, true>(d),  prepare<2, false, true>(d),  prepare<2, true, true>(d),
                            gemm_few_prepare()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t gemm_launch(const GemmArgs& a, const PromptDevice& d, cudaStream_t s) {
  if (a.rows <= kFewRows) return gemm_few_launch(a, d, s);
  const bool ragged = a.k % 256 != 0;
  if (a.w[1]) return ragged ? launch<2, true>(a, d, s) : launch<2, false>(a, d, s);
  return ragged ? launch<1, true>(a, d, s) : launch<1, false>(a, d, s);
}

cudaError_t gemm_read_status(int* out) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status_gm, sizeof(int));
  if (e != cudaSuccess || *out == 0) return e;
  return cudaMemcpyToSymbol(g_status_gm, &zero, sizeof(int));
}

}  // namespace q4
