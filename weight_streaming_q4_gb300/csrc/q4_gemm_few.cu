// Products of few rows with Q4_0 weights, with an epilogue (sm_103a): single
// tokens and small steps, where reading W is all there is to do.
//
// Tiles are 32 rows of W (16 of each of two matrices) over all of k, which a
// CTA's warps share out: two by the rows, four by columns, 1024 of them a stage
// (576 bytes of a row in one piece).  A CTA walks its tiles with one ring of
// stages, so that the next tile's first ones are on their way while a tile is
// finished.  W as it lies in memory and x's rows come by
// 16-byte cp.async into a ring.  The products are mma.sync m16n8k16 with 16 rows
// of W as its rows and 8 rows of x as its columns: the order of k in a product
// is free, so a thread takes 36 bytes of its two rows of W, two whole
// blocks, and the same 64 columns of x, and nothing is exchanged.  9 words
// apart, the four threads of a row and the eight rows of a load fall in 32
// different banks.  The warps' sums meet in shared memory, in a fixed order; few
// tiles are shared by clusters of 2, 4 or 8 CTAs, each with a part of k, whose
// sums meet over distributed shared memory (1024 x 4096, one row: 5.7 -> 4.4 us;
// 6176 x 17824, five: 39 -> 31; the gated 328 x 15616, two: 18.7 -> 7.0).
//
// Measured in a graph: one row, 4096 x 4096 with a residual 5.5 us (the kernel of many rows 14.4); gated 14336 x 4096
// 21.7 us, 3.0 TB/s, with 8 rows 27 (the other kernel 25 to 27 for any number up to 32).  No pipe bounds it: issue slots 57 %,
// integer and binary16 pipes 40 and 38 % busy; what is seen is a barrier of the whole CTA per 1024 columns and instructions
// from nibbles to binary16 that take two cycles each.  Two, three or four CTAs of an SM, and two or four chains of sums, measure
// the same.  With 7 and 8 rows only two of the CTAs fit an SM's memory, and the rest of the grid runs behind them.
#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_frag.cuh"
#include "q4_gemm.cuh"
#include "q4_tensor.cuh"

namespace q4 {

namespace {

constexpr int kFwThreads = 256;
constexpr int kFwCtas = 3;                // of an SM (with 7 and 8 rows two fit)
constexpr int kFwRowsW = 32;              // rows of W of a CTA
constexpr int kFwSlices = 4;              // warps along k
constexpr int kFwChunk = 144;             // bytes between 64 columns of a staged row of x (128 and a shift of the banks)
constexpr int kFwXRow = 16 * kFwChunk + 64;     // ... between its rows: 16 banks apart, so that loads of two rows do not collide

template <bool RAGGED>
struct Fw {
  // 16-byte pieces of a staged row of W (1024 columns), and the bytes between rows (each 4 words from another)
  static constexpr int PIECES = RAGGED ? 37 : 36;
  static constexpr int PITCH = RAGGED ? 624 : 592;
  static constexpr int W_BYTES = kFwRowsW * PITCH;
};

__device__ __forceinline__ float cluster_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int MATS, bool RAGGED, bool SHARED>
__global__ void __launch_bounds__(kFwThreads, kFwCtas) few_kernel(const __grid_constant__ GemmArgs a, int stages, int stage_bytes, int members) {
  using F = Fw<RAGGED>;
  constexpr int ROWS = kFwRowsW / MATS, COLS = kFewRows + 4;   // rows of each matrix; floats between the rows of the sums
  extern __shared__ __align__(128) char smem[];
  __shared__ float sums[kFwSlices][kFwRowsW][COLS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int nb = a.k / kQK, units = (nb + 7) / 8, count = (units + kFwSlices - 1) / kFwSlices;
  const int tiles = (a.n + ROWS - 1) / ROWS;
  // SHARED: the CTAs of a cluster, `split` of them, share a tile, and this one takes these stages of it
  const int split = SHARED ? members : 1;
  const int part = SHARED ? static_cast<int>(cluster_rank()) : 0, s0 = count * part / split, s1 = count * (part + 1) / split;
  const int first = blockIdx.x / split, stride = gridDim.x / split;
  const int64_t row_bytes = static_cast<int64_t>(nb) * kBlockBytes, end = row_bytes * a.n;

  // The copies, a stage ahead of another: tile c_tile, columns 1024 c_s ...  Row r of a tile is its row r % ROWS of matrix
  // r / ROWS; eight threads take 128 bytes of a row at a time.
  const int r = tid >> 3;
  const uint8_t* const w = a.w[MATS == 2 ? r >> 4 : 0];
  auto start = [&](int64_t row) { return RAGGED ? (row * row_bytes) & ~int64_t{15} : row * row_bytes; };
  const uint32_t base = smem_u32(smem);
  int c_tile = first, c_s = s0, c_slot = 0;
  int64_t from = start(c_tile * ROWS + (MATS == 2 ? r & 15 : r));
  auto copy = [&]() {
    if (c_tile < tiles) {
      const uint32_t to = base + c_slot * stage_bytes;
      const int w0 = c_tile * ROWS;
      constexpr int REST = F::PIECES - 32;
      auto piece = [&](int rr, int i) {
        const int row = w0 + (MATS == 2 ? rr & 15 : rr);
        const int64_t at = start(row) + c_s * 576 + i * 16, left = row < a.n ? end - at : 0;
        const int bytes = static_cast<int>(left < 0 ? 0 : left > 16 ? 16 : left);
        cp16_part(to + rr * F::PITCH + i * 16, a.w[MATS == 2 ? rr >> 4 : 0] + (bytes ? at : 0), bytes);
      };
      // (every byte of the pieces lies in the matrix: those of the last row end last)
      if (static_cast<int64_t>(w0 + ROWS - 1) * row_bytes + c_s * 576 + F::PIECES * 16 <= end) {
        const uint8_t* src = w + from + c_s * 576 + (tid & 7) * 16;
        const uint32_t dst = to + r * F::PITCH + (tid & 7) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) cp16(dst + i * 128, src + i * 128);
        if (!RAGGED) {
          if ((tid & 7) < REST) cp16(dst + 512, src + 512);
        } else if (tid < 32 * REST) {
          piece(tid / REST, 32 + tid % REST);
        }
      } else {
        for (int i = 0; i < 4; ++i) piece(r, i * 8 + (tid & 7));
        if (tid < 32 * REST) piece(tid / REST, 32 + tid % REST);
      }
      // x: 128 pieces of a row, what lies behind the row's end as zeros
      for (int i = tid; i < a.rows * 128; i += kFwThreads) {
        const int rr = i >> 7, p = i & 127, col = c_s * 1024 + p * 8, left = a.k - col;
        const int bytes = left < 0 ? 0 : left > 8 ? 16 : left * 2;
        cp16_part(to + F::W_BYTES + rr * kFwXRow + (p >> 3) * kFwChunk + (p & 7) * 16, a.x + (bytes ? rr * a.x_ld + col : 0), bytes);
      }
      if (++c_slot == stages) c_slot = 0;
      if (++c_s == s1) {
        c_s = s0, c_tile += stride;
        from = start(static_cast<int64_t>(c_tile) * ROWS + (MATS == 2 ? r & 15 : r));
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int s = 0; s < stages - 1; ++s) copy();

  const int group = warp & 1, slice = warp >> 1, r0 = group * 16 + g;      // this thread's rows of a tile: r0 and r0 + 8
  const bool there = g < a.rows;                                           // (rows that x has not are not staged)
  const int x_at = F::W_BYTES + (there ? g : 0) * kFwXRow + (slice * 4 + t) * kFwChunk;
  const int w_at = r0 * F::PITCH + slice * 144 + 36 * t;
  int slot = 0;
  for (int tile = first; tile < tiles; tile += stride) {
    const int w0 = tile * ROWS;
    float acc[2][4] = {};                                     // two sums that do not wait for one another
    int shift[2] = {0, 0};
    if (RAGGED)
      for (int h = 0; h < 2; ++h) shift[h] = static_cast<int>(((w0 + (MATS == 2 ? (r0 + 8 * h) & 15 : r0 + 8 * h)) * row_bytes) & 15);
    for (int s = s0; s < s1; ++s) {
      // (the group of this stage is done when at most stages - 2 later ones are not)
      switch (stages) {
        case 2: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 3: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 4: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
      }
      __syncthreads();
      copy();
      const char* stage = smem + slot * stage_bytes;
      if (++slot == stages) slot = 0;
      const int u = s * kFwSlices + slice;
      if (u >= units) continue;
      uint32_t v[2][9];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(stage + w_at + 8 * h * F::PITCH + (shift[h] & ~3));
        if (RAGGED) {
          const uint32_t by = (shift[h] & 2) * 8;
          uint32_t now = src[0];
#pragma unroll
          for (int e = 0; e < 9; ++e) {
            const uint32_t after = src[e + 1];
            v[h][e] = __funnelshift_r(now, after, by);
            now = after;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 9; ++e) v[h][e] = src[e];
        }
      }
      const int left = nb - u * 8 - 2 * t;                    // blocks of the row from this thread's first one on
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t o[2][16], x[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 f = *reinterpret_cast<const uint4*>(stage + x_at + b * 64 + e * 16);
          x[4 * e] = f.x, x[4 * e + 1] = f.y, x[4 * e + 2] = f.z, x[4 * e + 3] = f.w;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (b == 0)
            q4_first_block(v[h], o[h]);
          else
            q4_second_block(v[h], o[h]);
          if (RAGGED && left <= b) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[h][e] = 0;
          }
        }
        // (a column that stands for no row of x is a copy of row 0's, and not stored)
#pragma unroll
        for (int j = 0; j < 8; ++j) mma16816(acc[j & 1], o[0][2 * j], o[1][2 * j], o[0][2 * j + 1], o[1][2 * j + 1], x[2 * j], x[2 * j + 1]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[slice][r0 + (e >> 1) * 8][2 * t + (e & 1)] = acc[0][e] + acc[1][e];
    __syncthreads();
    if (SHARED) {
      // (a CTA's slices are added up before the others read them)
      for (int i = tid; i < kFwRowsW * a.rows; i += kFwThreads) {
        const int rr = i % kFwRowsW, c = i / kFwRowsW;
        float f = sums[0][rr][c];
#pragma unroll
        for (int j = 1; j < kFwSlices; ++j) f += sums[j][rr][c];
        sums[0][rr][c] = f;
      }
      __syncwarp();
      cluster_sync();
    }
    // (the next sums are stored behind another barrier)
    for (int i = part * kFwThreads + tid; i < ROWS * a.rows; i += split * kFwThreads) {
      const int rr = i % ROWS, c = i / ROWS, n = w0 + rr;
      if (n >= a.n) continue;
      float f[MATS];
#pragma unroll
      for (int m = 0; m < MATS; ++m) {
        f[m] = 0.f;
        if (SHARED) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (q < split) f[m] += cluster_load(cluster_addr(&sums[0][m * 16 + rr][c], q));
        } else {
#pragma unroll
          for (int j = 0; j < kFwSlices; ++j) f[m] += sums[j][m * 16 + rr][c];
        }
        if (a.bias[m]) f[m] += __ldg(a.bias[m] + n);
      }
      activate<1>(f, a.act);
      if (MATS == 2) {
        f[0] *= f[MATS - 1];
      } else {
        f[0] *= a.scale;
        if (a.residual.p) {
          const int64_t at = c * a.residual.ld + n;
          f[0] += a.residual.f32 ? static_cast<const float*>(a.residual.p)[at] : __half2float(static_cast<const __half*>(a.residual.p)[at]);
        }
      }
      a.y[c * a.y_ld + n] = __float2half_rn(f[0]);
    }
    if (SHARED) {
      __syncwarp();
      cluster_sync();                // (the sums have been read)
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------ host

constexpr int kFwSmemMost = 204 * 1024;          // of an SM

template <int MATS, bool RAGGED>
cudaError_t launch(const GemmArgs& a, const PromptDevice& d, cudaStream_t s) {
  const int stage = Fw<RAGGED>::W_BYTES + a.rows * kFwXRow;
  const int64_t tiles = (static_cast<int64_t>(a.n) + kFwRowsW / MATS - 1) / (kFwRowsW / MATS);
  // Few tiles: clusters share them, while all their CTAs run at once, if the SM with most to do then has fewer stages, by more
  // than what the meeting of a cluster takes (about one stage with one row of x, two with eight).
  const int count = (a.k - 1) / 1024 + 1;
  auto most = [&](int split) { return (tiles * split + d.sms - 1) / d.sms * ((count + split - 1) / split); };
  int split = 1;
  for (int other = 2; other <= 8 && other * tiles <= d.sms * kFwCtas && other <= count; other *= 2)
    if (most(other) + (split == 1) * (1 + a.rows / 8) < most(split)) split = other;
  // what runs on an SM shares its memory
  const int64_t all = tiles * split;
  const int ctas = all <= d.sms ? 1 : all <= 2 * d.sms ? 2 : kFwCtas;
  int stages = kFwSmemMost / ctas / stage;
  stages = stages < 2 ? 2 : stages > 5 ? 5 : stages;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = split, at.val.clusterDim.y = 1, at.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(all < d.sms * ctas ? all : d.sms * ctas));
  cfg.blockDim = dim3(kFwThreads);
  cfg.dynamicSmemBytes = stages * stage;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, split > 1 ? few_kernel<MATS, RAGGED, true> : few_kernel<MATS, RAGGED, false>, a, stages, stage, split);
}

template <int MATS, bool RAGGED>
cudaError_t prepare() {
  const cudaError_t e = cudaFuncSetAttribute(few_kernel<MATS, RAGGED, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFwSmemMost);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(few_kernel<MATS, RAGGED, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFwSmemMost);
}

}  // namespace

cudaError_t gemm_few_prepare() {
  const cudaError_t e[4] = {prepare<1, false>(), prepare<1, true>(), prepare<2, false>(), prepare<2, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t gemm_few_launch(const GemmArgs& a, const PromptDevice& d, cudaStream_t s) {
  if (a.w[1]) return a.k % 256 ? launch<2, true>(a, d, s) : launch<2, false>(a, d, s);
  return a.k % 256 ? launch<1, true>(a, d, s) : launch<1, false>(a, d, s);
}

}  // namespace q4
