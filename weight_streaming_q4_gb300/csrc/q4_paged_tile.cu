// Attention of chunks of new tokens over a paged KV cache on the fifth
// generation's tensor cores (sm_103a).
//
// One persistent CTA per SM (q4_paged_sched.cuh splits the work), R = 256 query
// rows of a value head per item (two tiles of 128; one at head_dim above 128 or
// with fp32 queries), key tiles of BN positions.  Per query tile and key tile:
//   S = Q K^T       tcgen05.mma, Q and K in shared memory, S [128][BN] in tensor memory
//   P = 2^(S c - m) 128 threads, a row each: no exchange between threads
//   O += P V        tcgen05.mma, P (binary16) in tensor memory over S's columns,
//                   V in shared memory as it lies in the page ([position][head_dim])
// with the running maximum m and sum l of a row in its thread.  m is only raised,
// and O rescaled, when a tile's maximum exceeds it by more than 8 (a factor of
// 256: P stays far inside binary16, sums are fp32), so O is seldom touched.
// The two query tiles take turns: while the threads of one work on its scores,
// the tensor cores work for the other.
//
// Warps 0-3 and 4-7: the softmax of query tile 0 and 1; the warps behind them fill
// the ring of key and value tiles, the last warp issues the products.
//
// A tile is made of pieces of pages.  Binary16: a tensor copy (TMA, 128-byte
// swizzle) per 64 columns and page or 16 .. BN rows of it, issued by the lanes of
// one warp side by side; a copy through the threads (16-byte cp.async) took 6700
// cycles a tile where the products take 2050.  Q8: bulk copies of codes and
// scales into a staging place, from which six warps take them into registers
// and store them as f16(code * d).
// Positions that no row of the item sees must count as zeros in the product with
// P = 0 (a stale or later value may be NaN, and 0 * NaN is NaN), and so must
// values that are not finite in a tile that some rows see only in part: such
// tiles (the last one or two of an item, a window's edge, holes) are cleaned in
// shared memory, what was not finite is noted, and the rows that do see it get
// it added at the end.  Keys need no cleaning: their scores are replaced.
//
// Precision: binary16 queries enter as they are, fp32 queries as two binary16
// parts (22 bits of a scaled row, QueryScale; two products into the same S); P is rounded to binary16
// (2^-11 relative, as much as the output's own rounding; a second product with what that leaves out
// would cost half again the products), the sum l is taken of the unrounded weights.
//
// Measured, back to back in a graph: 2048 tokens of the 8B heads over 16384 positions 351 us, 1470 TFLOP/s, 76 %
// of a library matrix product's rate (fp32 queries, one query tile and half again the products: 562 us); the scores -> weights -> product chain of one
// query tile that the other one does not cover bounds it (tensor pipe 65 % busy), and power.  512
// tokens of the 70B heads over 8192 positions of Q8 135 us, 985 TFLOP/s: the conversion
// shares the issue slots with the softmax.  Eight ragged sequences of up to 2049 tokens 184 us,
// 792 TFLOP/s: outputs 23 us of it, cleaning 14 (each by leaving it out).
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "q4_paged_sched.cuh"
#include "q4_tensor.cuh"

namespace q4 {

namespace {

constexpr uint32_t kPtWaitLimit = 1u << 21;
__device__ int g_status_pt;

__device__ __forceinline__ void cp16_zfill(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Whether one of eight binary16 values is infinite or NaN: an exponent of all
// ones carries into the sign's place.
__device__ __forceinline__ bool h2_any_bad(const uint4& u) {
  constexpr uint32_t M = 0x7c007c00u, A = 0x04000400u;
  return ((((u.x & M) + A) | ((u.y & M) + A) | ((u.z & M) + A) | ((u.w & M) + A)) & 0x80008000u) != 0;
}

// ------------------------------------------------------------------ geometry

template <int HD, bool QF32, bool Q8>
struct Pt {
  static constexpr int BN = HD <= 128 ? 128 : 64;
  static constexpr int NQ = HD <= 128 && !QF32 ? 2 : 1;
  static constexpr int R = 128 * NQ;
  static constexpr int QB = 128 * HD * 2;               // bytes of a query tile (one part)
  static constexpr int KB = BN * HD * 2;                // bytes of a key or value tile
  static constexpr int LIMIT = 232448 - 1024 - 1024;    // control data, and the alignment of the tiles
  static constexpr int QALL = QB * (QF32 ? 2 : NQ);
  static constexpr int RAW = Q8 ? BN * HD + BN * HD / 16 : 0;   // a staged Q8 tile: codes, then scales
  static constexpr int NRAW = Q8 ? 1 : 0;
  static constexpr int OUT = NQ * 4 * 2048;             // per softmax warp: 32 rows of 64 bytes on their way out
  static constexpr int FIT = (LIMIT - QALL - OUT - NRAW * RAW) / KB;
  static constexpr int NS = FIT > 8 ? 8 : FIT;          // ring of key and value tiles
  static constexpr int SMEM = 2048 + QALL + NS * KB + NRAW * RAW + OUT;
  // tensor memory columns: S of query tile q at q * 128, then O; with one query tile S has two places
  // that take turns, so that the next scores are computed while the softmax works on these
  static constexpr int O_COL = 256;
  static constexpr int H = 64, NH = BN / 64;            // P is handed over 64 positions at a time ("halves")
  // warpgroups: two of softmax, then binary16: copies (warp 8), cleaning (9, 10), products (11);
  // Q8: conversion (8 to 13), copies (14), products (15)
  static constexpr int GROUPS = Q8 ? 4 : 3, THREADS = 128 * GROUPS;
  static constexpr int W_SIDE = Q8 ? 8 : 9, CONV = Q8 ? 6 : 2;      // the cleaning or converting warps
  static constexpr int W_COPY = Q8 ? 14 : 8, W_MMA = 4 * GROUPS - 1;
  // registers per thread after the split: softmax warpgroups, the others
  static constexpr int REG_S = Q8 ? 152 : 184;
  static constexpr int REG_O = Q8 ? 104 : (NQ == 2 ? 136 : 152);
  static constexpr int REGS = (NQ * REG_S + (GROUPS - NQ) * REG_O) * 128;
  static_assert(NS >= (NQ == 2 ? 3 : 2), "a key and a value tile, and the next key tile beside two query tiles");
};

// Tensor copies of binary16 pages: rows of HD values, boxes of 64 values by
// 2^box_log2 rows.
struct PtMaps {
  CUtensorMap k, v;
  int box_log2;
};

struct PtCtl {
  uint64_t full[8], empty[8], q_full[2];
  uint64_t s_full[2];      // scores of query tile q are there (one query tile: in place 0, 1)
  uint64_t p_full[2][2];   // weights of query tile q (one query tile: in place 0, 1, since the softmax
                           // may be a tile ahead of the products), half h
  uint64_t o_full[2][2];   // the product with half h is done
  uint64_t fixed[8];       // the value tile in a ring slot has been looked at, and cleaned if need be
  uint64_t raw, raw_free;  // a staged Q8 tile has landed; its place is free again
  uint64_t done;           // every product is done
  uint32_t tmem;
  int dead;
  // Where the loaders met infinities or NaN among a segment's values: per query tile its own count of the segments in
  // which it has rows (+ 1), by count mod 8.  A value tile's place in the ring is free only when every query tile with
  // rows has used it, so the loaders are at most five key tiles, and five of a query tile's own segments, ahead of
  // its softmax.  (Any number of segments without rows of the second query tile may pass while that one ends an item.)
  int bad[2][8];
  int second[16];          // Q8: the second query tile's count, by each converting warp
  uint32_t there[8];       // per key tile, by number mod 8: bit g = rows 16 g .. of the tile are in a page
  CtaWork work;
  long long scan[17];
};
static_assert(sizeof(PtCtl) <= 1024, "control data fits its place");

// A wait that gives up at once when one has run out before: the roles walk on
// and the kernel ends (its results do not count: the status word says so).
__device__ __forceinline__ void pt_wait(PtCtl* c, uint64_t* bar, uint32_t parity) {
  if (mbar_test_wait(bar, parity)) return;
  const uint32_t limit = *reinterpret_cast<volatile int*>(&c->dead) ? 0 : kPtWaitLimit;
  if (!mbar_wait_bounded(bar, parity, limit)) {
    *reinterpret_cast<volatile int*>(&c->dead) = 1;
    atomicOr(&g_status_pt, ST_FULL_TIMEOUT);
  }
}

// Before the CTA ends: a copy or product of its own that is still in flight
// (none is, unless a wait has run out), whatever ran out before.
__device__ __forceinline__ void pt_drain(uint64_t* bar, uint32_t parity) {
  if (!mbar_wait_bounded(bar, parity, kPtWaitLimit)) atomicOr(&g_status_pt, ST_DRAIN_TIMEOUT);
  __syncwarp();
}

// As pt_wait for a whole warp, which is together again afterwards.
__device__ __forceinline__ void pt_wait_warp(PtCtl* c, uint64_t* bar, uint32_t parity) {
  pt_wait(c, bar, parity);
  __syncwarp();
}

// A place in the ring and the parity of its current turn.
template <int NS>
struct RingAt {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void step() {
    if (++slot == NS) slot = 0, parity ^= 1;
  }
  // which value tile of its slot the n-th value tile of the ring is (an odd ring holds keys and values
  // in turn in every slot, an even one values in its odd slots)
  static __device__ __forceinline__ uint32_t turn(uint32_t n) { return NS & 1 ? n / NS : n / (NS / 2); }
};

// What of a key tile an item's rows see.
struct TileView {
  int base;             // first position of the tile
  bool whole;           // every row sees every position of it (holes aside)
};
template <int BN>
__device__ __forceinline__ TileView tile_view(const PagedAttnArgs& a, const ItemTiles& it, int i) {
  TileView v;
  v.base = it.tile(i) * BN;
  v.whole = v.base + BN - 1 <= it.p0 && (!a.window || v.base > it.p1 - a.window || v.base + BN <= a.sinks);
  return v;
}

// Values that were taken out of tiles seen in part, back into columns b .. of a
// row at position p that sees them (rare, so out of the way of the registers).
template <int R, int BN, int HD, bool Q8>
__device__ __noinline__ void add_taken_out(const PagedAttnArgs& a, const SegmentWalk<R, BN>& w, int p, int b, float* of) {
  for (int i = w.i0; i < w.i1; ++i) {
    const TileView tv = tile_view<BN>(a, w.it, i);
    if (tv.whole) continue;
    for (int t = tv.base; t < tv.base + BN && t <= p; ++t) {
      if (a.window && t <= p - a.window && t >= a.sinks) continue;
      const int row = paged_row(a.kv, a.b, w.seq, t, w.head);
      if (row < 0) continue;
      for (int e = 0; e < 32; ++e) {
        const size_t at = static_cast<size_t>(row) * HD + b + e;
        const __half h = Q8 ? __hmul(__int2half_rn(static_cast<const int8_t*>(a.kv.v)[at]), a.kv.vs[at / 32])
                            : static_cast<const __half*>(a.kv.v)[at];
        if (__hisinf(h) || __hisnan(h)) of[e] += __half2float(h);
      }
    }
  }
}

// ------------------------------------------------------------------ kernel

template <int HD, bool QF32, bool Q8>
__global__ void __launch_bounds__(Pt<HD, QF32, Q8>::THREADS, 1)
    paged_tile_kernel(const __grid_constant__ PagedAttnArgs a, PartSlots parts, const __grid_constant__ PtMaps maps) {
  using G = Pt<HD, QF32, Q8>;
  constexpr int BN = G::BN, NQ = G::NQ, R = G::R, NS = G::NS, H = G::H, NH = G::NH;
  extern __shared__ char smem_raw[];
  PtCtl* c = reinterpret_cast<PtCtl*>(smem_raw);
  // tiles start on 1024-byte boundaries (the swizzle's period)
  char* tiles = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1024 + 1023) & ~uintptr_t{1023});
  const uint32_t s_q = smem_u32(tiles), s_ring = s_q + G::QALL;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&c->full[i], Q8 ? G::CONV : 1), mbar_init(&c->empty[i], 1), mbar_init(&c->fixed[i], G::CONV);
    for (int q = 0; q < 2; ++q) {
      mbar_init(&c->q_full[q], 128);
      mbar_init(&c->s_full[q], 1);
      for (int h = 0; h < 2; ++h) mbar_init(&c->p_full[q][h], 128), mbar_init(&c->o_full[q][h], 1);
    }
    mbar_init(&c->raw, 1), mbar_init(&c->raw_free, G::CONV), mbar_init(&c->done, 1);
    c->dead = 0;
    for (int i = 0; i < 16; ++i) c->bad[i >> 3][i & 7] = c->second[i] = 0;
    fence_mbar_init();
  }
  if (warp == G::W_MMA) tm_alloc(&c->tmem, 512);
  if (a.b.n_seqs > 32) cta_work<R, BN, G::THREADS>(a, c->scan, &c->work);
  const bool few = a.b.n_seqs <= 32;
  CtaWork work;
  if (few) work = warp_work<R, BN>(a);
  tm_before();
  __syncthreads();
  tm_after();
  const uint32_t tmem = __shfl_sync(~0u, c->tmem, 0);
  if (!few) work = c->work;
  SegmentWalk<R, BN> w;
  w.begin(a, work);
  JoinRecord rec = {};       // thread 0's

  if (warp < 4 * NQ)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::REG_S));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::REG_O));
  if (warp < 4 * NQ) {
    // ---------------------------------------------------------------- softmax of query tile q
    const int q = warp >> 2, wl = warp & 3;
    const uint32_t t_s = tmem + q * 128 + (static_cast<uint32_t>(wl * 32) << 16);
    const uint32_t t_o = tmem + G::O_COL + q * 128 + (static_cast<uint32_t>(wl * 32) << 16);
    uint32_t n_s = 0;       // S tiles seen: parity of s_full, and of the product before it
    int seg = 0;            // segments in which this query tile had rows
    uint32_t n_k = 0;       // key tiles of the CTA before the current one
    float scale = a.scale;  // of this thread's row's scores
    // The queries of this tile of an item into shared memory: the warp's 32 rows,
    // 16-byte pieces of a row side by side.  The products that read the last ones
    // are done (their scores have been taken).
    auto load_q = [&](const SegmentWalk<R, BN>& g) {
      const int rows = g.rows();
      if (q * 128 >= rows) return;
      constexpr int PIECES = HD / 8;
      const int own = q * 128 + wl * 32 + lane, r = g.j * R + own;
      const int64_t own_at = own < rows ? a.row_at(g.sp.t0, g.head, r, a.q_ld) : -1;
      if (!QF32) {
#pragma unroll 4
        for (int x = lane; x < 32 * PIECES; x += 32) {
          const int rl = x / PIECES, rr = wl * 32 + rl, pc = x % PIECES;
          const int64_t at = __shfl_sync(~0u, own_at, rl);
          const uint32_t off = (pc >> 3) * (128 * 128) + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4);
          cp16_zfill(s_q + q * G::QB + off, static_cast<const __half*>(a.q) + (at < 0 ? 0 : at + pc * 8), at >= 0);
        }
      } else {
        // a row at a time, 8 bytes per lane: its largest element is wanted (QueryScale)
#pragma unroll 8
        for (int rl = 0; rl < 32; ++rl) {
          const int rr = wl * 32 + rl;
          const int64_t at = __shfl_sync(~0u, own_at, rl);
          float2 f[HD / 64];
          uint32_t most = 0;
#pragma unroll
          for (int j = 0; j < HD / 64; ++j) {
            f[j] = make_float2(0.f, 0.f);
            if (at >= 0) f[j] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + j * 64 + lane * 2));
            most = max(most, abs_bits(f[j]));
          }
          const QueryScale qs(__reduce_max_sync(~0u, most));
          if (lane == rl) scale = a.scale * qs.down;
          char* const to = tiles + rr * 128 + (((lane >> 2) ^ (rr & 7)) << 4) + (lane & 3) * 4;
#pragma unroll
          for (int j = 0; j < HD / 64; ++j) {
            __half2 hi, lo;
            query_parts(f[j], qs.up, &hi, &lo);
            *reinterpret_cast<__half2*>(to + j * (128 * 128)) = hi;
            *reinterpret_cast<__half2*>(to + G::QB + j * (128 * 128)) = lo;
          }
        }
      }
    };
    auto loaded_q = [&](const SegmentWalk<R, BN>& g) {       // ... are there
      if (q * 128 >= g.rows()) return;
      if (!QF32) asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async();
      mbar_arrive(&c->q_full[q]);
    };
    if (w.live()) {
      load_q(w);
      loaded_q(w);
    }
    while (w.live()) {
      const int rows = w.rows(), row0 = w.j * R;
      join_note(&rec, w, work.per);
      const bool active = q * 128 < rows;
      const int r = row0 + q * 128 + wl * 32 + lane;       // this thread's row
      const bool mine = q * 128 + wl * 32 + lane < rows;
      const int p = mine ? w.sp.len - w.sp.n_new + a.token_of(r) : -1;
      float m = -INFINITY, l = 0.f;
      if (!active) n_k += w.i1 - w.i0;
      for (int i = active ? w.i0 : w.i1; i < w.i1; ++i, ++n_s, ++n_k) {
        const TileView tv = tile_view<BN>(a, w.it, i);
        const uint32_t turn = NQ == 2 ? 0 : n_s & 1;
        if (NQ == 2)
          pt_wait_warp(c, &c->s_full[q], n_s & 1);
        else
          pt_wait_warp(c, &c->s_full[turn], (n_s >> 1) & 1);
        tm_after();
        const uint32_t there = *reinterpret_cast<volatile uint32_t*>(&c->there[n_k & 7]);
        const bool part = !tv.whole || there != (1u << (BN / 16)) - 1;
        const uint32_t t_x = t_s + turn * BN;
#pragma unroll 1
        for (int h = 0; h < NH; ++h) {
          uint32_t x[H];
          float* f = reinterpret_cast<float*>(x);
          float2 sum;
          // The weights with the maximum as it is; where that turns out to be too low, once
          // more.  So the maximum of a half costs no time before its weights.
#pragma unroll 1
          for (;;) {
#pragma unroll
            for (int b = 0; b < H; b += 32) tm_ld32(t_x + h * H + b, x + b);
            tm_ld_wait(x);
#pragma unroll
            for (int b = 32; b < H; b += 32) tm_ld_waited(x + b);
            if (part) {
              const int hi = p - tv.base - h * H;
              const int lo = a.window ? hi - a.window + 1 : 0, sk = a.sinks - tv.base - h * H;
              const uint32_t in_page = there >> (h * (H / 16));
#pragma unroll
              for (int b = 0; b < H; b += 32) {
                // bit e: this row sees column b + e
                uint32_t see = hi - b >= 31 ? ~0u : hi < b ? 0u : (2u << (hi - b)) - 1;
                const uint32_t in = lo <= b ? ~0u : lo - b > 31 ? 0u : ~0u << (lo - b);
                const uint32_t sink = sk - b > 31 ? ~0u : sk <= b ? 0u : (1u << (sk - b)) - 1;
                see &= (in | sink) &
                       (((in_page >> (b >> 4)) & 1 ? 0xffffu : 0u) | ((in_page >> (b >> 4)) & 2 ? 0xffff0000u : 0u));
#pragma unroll
                for (int e = 0; e < 32; ++e) f[b + e] = (see >> e) & 1 ? f[b + e] : -INFINITY;
              }
            }
            const float mm = m == -INFINITY ? 0.f : m;
            const float2 sc2 = make_float2(scale, scale), mm2 = make_float2(-mm, -mm);
            float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            float2 sum2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int e = 0; e < H; e += 2) {
              top4[(e >> 1) & 3] = fmaxf(top4[(e >> 1) & 3], fmaxf(f[e], f[e + 1]));
              const float2 t = f2_fma(make_float2(f[e], f[e + 1]), sc2, mm2);
              float2 y;
              asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(t.x));
              asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(t.y));
              sum2[(e >> 1) & 1] = f2_add(sum2[(e >> 1) & 1], y);
              x[e / 2] = pack_h2(y.x, y.y);
            }
            sum = f2_add(sum2[0], sum2[1]);
            const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * scale;
            const bool raise = top > m + 8.f || (m == -INFINITY && top > m);
            if (!__any_sync(~0u, raise)) break;
            // raise the warp's maxima and rescale what O and l hold, after the product before this half's
            const float m2 = fmaxf(m, top);
            const float fac = m == m2 ? 1.f : exp2f(m - m2);
            if (i > w.i0 || h > 0) {
              pt_wait_warp(c, &c->o_full[q][h ? 0 : NH - 1], (h ? n_s : n_s - 1) & 1);
              tm_after();
#pragma unroll 1
              for (int b = 0; b < HD; b += 32) {
                uint32_t o[32];
                tm_ld32(t_o + b, o);
                tm_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fac);
                tm_st32(t_o + b, o);
              }
            }
            l *= fac;
            m = m2;
          }
          l += sum.x + sum.y;
          // With one query tile these scores came ahead of the last tile's product.  Before P goes out that
          // product is done (the next could not start earlier anyway): so a wait for a turn of o_full, here,
          // above or below, only ever finds that turn open or just over, never the one after it.
          if (NQ == 1 && h == 0 && n_s > 0) pt_wait_warp(c, &c->o_full[q][NH - 1], (n_s - 1) & 1);
          // P over the scores' first columns (their half has been read)
          tm_st32(t_x + h * (H / 2), x);
          tm_st_wait();
          tm_before();
          mbar_arrive(&c->p_full[NQ == 2 ? q : turn][h]);
        }
      }
      // the next item's queries, so that its first scores are computed meanwhile
      SegmentWalk<R, BN> next = w;
      next.next(a);
      if (next.live()) load_q(next);
      if (!active) {
        if (next.live()) loaded_q(next);
        w = next;
        continue;
      }
      // the item's (or the part's) end
      pt_wait_warp(c, &c->o_full[q][NH - 1], (n_s - 1) & 1);
      tm_after();
      if (next.live()) loaded_q(next);
      const bool whole_item = w.i0 == 0 && w.i1 == w.it.cnt;
      const bool bad = *reinterpret_cast<volatile int*>(&c->bad[q][seg & 7]) == seg + 1;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int slot = w.i0 == 0 ? 1 : 0;
      // A thread holds a row, but stores go out with four lanes to a row, over shared memory: 64 bytes of
      // each row at a time, the 16-byte pieces exchanged by row so that they fall into different banks.
      // (A store of 16 bytes in each of 32 rows costs 32 passes.)
      const int64_t out_at = mine ? a.row_at(w.sp.t0, w.head, r, a.out_ld) : 0;
      char* const turn_at = tiles + G::QALL + NS * G::KB + G::NRAW * G::RAW + warp * 2048;
      char* const turn_mine = turn_at + lane * 64;
      float* const part0 = parts.out(blockIdx.x, slot) + static_cast<size_t>(q * 128 + wl * 32) * HD;
      const int n_mine = rows - q * 128 - wl * 32;                // rows of this warp
      __half* to[4];                                              // of the rows this lane stores pieces of
#pragma unroll
      for (int k = 0; k < 4; ++k) to[k] = a.out + __shfl_sync(~0u, out_at, k * 8 + (lane >> 2)) + (lane & 3) * 8;
#pragma unroll 1
      for (int b = 0; b < HD; b += 32) {
        uint32_t o[32];
        __syncwarp();
        tm_ld32(t_o + b, o);
        tm_ld_wait(o);
        float* of = reinterpret_cast<float*>(o);
        if (bad) {
          float back[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) back[e] = of[e];
          add_taken_out<R, BN, HD, Q8>(a, w, p, b, back);
#pragma unroll
          for (int e = 0; e < 32; ++e) of[e] = back[e];
          __syncwarp();
        }
        if (whole_item) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(turn_mine + ((k ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pack_h2(of[8 * k] * inv, of[8 * k + 1] * inv), pack_h2(of[8 * k + 2] * inv, of[8 * k + 3] * inv),
                           pack_h2(of[8 * k + 4] * inv, of[8 * k + 5] * inv), pack_h2(of[8 * k + 6] * inv, of[8 * k + 7] * inv));
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = k * 8 + (lane >> 2), pc = lane & 3;
            const uint4 u = *reinterpret_cast<const uint4*>(turn_at + row * 64 + ((pc ^ ((row >> 1) & 3)) << 4));
            if (row < n_mine) *reinterpret_cast<uint4*>(to[k] + b) = u;
          }
        } else {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<float4*>(turn_mine + ((k ^ ((lane >> 1) & 3)) << 4)) =
                  make_float4(of[half * 16 + 4 * k], of[half * 16 + 4 * k + 1], of[half * 16 + 4 * k + 2], of[half * 16 + 4 * k + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = k * 8 + (lane >> 2), pc = lane & 3;
              const float4 u = *reinterpret_cast<const float4*>(turn_at + row * 64 + ((pc ^ ((row >> 1) & 3)) << 4));
              if (row < n_mine) *reinterpret_cast<float4*>(part0 + static_cast<size_t>(row) * HD + b + half * 16 + pc * 4) = u;
            }
            __syncwarp();
          }
        }
      }
      if (!whole_item && mine) {
        parts.max(blockIdx.x, slot)[q * 128 + wl * 32 + lane] = m;
        parts.sum(blockIdx.x, slot)[q * 128 + wl * 32 + lane] = l;
      }
      w = next;
      ++seg;
    }
  } else if (warp >= 8 && warp < G::W_MMA) {
    // ---------------------------------------------------------------- key and value tiles
    constexpr uint32_t ALL = (1u << (BN / 16)) - 1;
    const int bl = Q8 ? min(a.kv.page_log2, BN == 128 ? 7 : 6) : maps.box_log2;   // rows of a piece of a page: 2^bl
    constexpr int COLS = Q8 ? 1 : HD / 64;                                       // copies per piece
    // Piece `lane / COLS` of tile i of the walk's item: its page-memory row, or -1 (not there, or seen by no row)
    auto lookup = [&](const SegmentWalk<R, BN>& g, int i) {
      const int base = g.it.tile(i) * BN, t = base + ((lane / COLS) << bl);
      if ((lane / COLS) << bl >= BN || t > g.it.p1) return -1;
      if (a.window && t + (1 << bl) <= max(g.it.p0, 0) - a.window + 1 && t >= a.sinks) return -1;
      return paged_row(a.kv, a.b, g.seq, t, g.head);
    };
    // Values of segment number seg were not finite.  The second query tile's own count of segments is in a register where
    // there is one to spare (in shared memory: mixed_8 185.7 us, not 184.3), else in shared memory (in a register:
    // chunk_512_q8 147 us, not 134.6).
    int second = 0;
    auto note_bad = [&](int seg) {
      *reinterpret_cast<volatile int*>(&c->bad[0][seg & 7]) = seg + 1;
      if (w.rows() > 128) {
        const int own = Q8 ? *reinterpret_cast<volatile int*>(&c->second[warp]) : second;
        *reinterpret_cast<volatile int*>(&c->bad[1][own & 7]) = own + 1;
      }
    };
    auto next_segment = [&]() {
      if (NQ == 2 && w.rows() > 128) {
        if (!Q8)
          ++second;
        else if (lane == 0)
          *reinterpret_cast<volatile int*>(&c->second[warp]) += 1;
      }
      w.next(a);
    };
    // bit r / 16: rows r .. of the tile are in a page (and seen)
    auto there_of = [&](int row) {
      const int at = __shfl_sync(~0u, row, (((lane & 7) << 4) >> bl) * COLS);
      return __ballot_sync(~0u, at >= 0) & ALL;
    };
    if (!Q8 && warp == G::W_COPY) {
      uint32_t n = 0;                                            // tiles issued (keys and values)
      int row = w.live() ? lookup(w, w.i0) : -1;
      while (w.live()) {
        for (int i = w.i0; i < w.i1; ++i) {
          const int now = row;
          if (i + 1 < w.i1) row = lookup(w, i + 1);              // the next tile's page entries on their way
          const uint32_t there = there_of(now);
          const uint32_t bytes = __popc(__ballot_sync(~0u, now >= 0)) << (bl + 7);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const uint32_t slot = n % NS;
            pt_wait_warp(c, &c->empty[slot], ((n / NS) & 1) ^ 1);
            if (lane == 0) {
              if (kv == 0) *reinterpret_cast<volatile uint32_t*>(&c->there[(n / 2) & 7]) = there;
              mbar_arrive_expect_tx(&c->full[slot], bytes);
            }
            __syncwarp();
            if (now >= 0)
              tma_load_2d(tiles + G::QALL + slot * G::KB + (lane % COLS) * (BN * 128) + ((lane / COLS) << (bl + 7)),
                          kv ? &maps.v : &maps.k, (lane % COLS) * 64, now, &c->full[slot]);
          }
        }
        w.next(a);
        if (w.live()) row = lookup(w, w.i0);
      }
      for (uint32_t t = n > NS ? n - NS : 0; t < n; ++t) pt_drain(&c->full[t % NS], (t / NS) & 1);
    } else if (!Q8) {   // (warps 9 and 10)
      // value tiles to be cleaned
      uint32_t n = 1;
      int seg = 0;
      for (; w.live(); ++seg, next_segment()) {
        for (int i = w.i0; i < w.i1; ++i, n += 2) {
          pt_wait_warp(c, &c->full[n % NS], (n / NS) & 1);
          const TileView tv = tile_view<BN>(a, w.it, i);
          const uint32_t there = *reinterpret_cast<volatile uint32_t*>(&c->there[(n / 2) & 7]);
          if (tv.whole && there == ALL) {
            if (lane == 0) mbar_arrive(&c->fixed[n % NS]);
            continue;
          }
          // Positions that some row sees: up to `last`, from `first` on or below sk; that every row sees: up to
          // all_last, from all_first on or below sk.  Only what lies between, or in a hole, is looked at.
          const int last = min(w.it.p1 - tv.base, BN - 1), first = a.window ? max(w.it.p0, 0) - a.window + 1 - tv.base : 0;
          const int all_last = w.it.p0 - tv.base, all_first = a.window ? w.it.p1 - a.window + 1 - tv.base : 0, sk = a.sinks - tv.base;
          bool found = false;
          constexpr int PIECES = HD / 8;
          constexpr int N = G::CONV * 32;
          const int me = tid - G::W_SIDE * 32;
          char* const tile = tiles + G::QALL + (n % NS) * G::KB;
          auto piece = [&](int x) {
            const int row = x / PIECES, pc = x % PIECES;
            return reinterpret_cast<uint4*>(tile + (pc >> 3) * (BN * 128) + row * 128 + (((pc & 7) ^ (row & 7)) << 4));
          };
          auto clean = [&](uint4 u, uint4* v) {
            if (!h2_any_bad(u)) return;
            __half* h = reinterpret_cast<__half*>(&u);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (__hisinf(h[e]) || __hisnan(h[e])) h[e] = __ushort_as_half(0);
            *v = u;
            found = true;
          };
          auto clean_rows = [&](int from, int to) {        // four loads under way
            const int end = to * PIECES;
#pragma unroll 1
            for (int x = from * PIECES + me; x < end; x += 4 * N) {
              uint4 u[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) u[k] = *piece(min(x + N * k, end - 1));
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (x + N * k < end) clean(u[k], piece(x + N * k));
            }
          };
          auto zero_rows = [&](int from, int to) {
#pragma unroll 4
            for (int x = from * PIECES + me; x < to * PIECES; x += N) *piece(x) = make_uint4(0, 0, 0, 0);
          };
          // rows [lo, hi) are those some row sees, of which [lo, lo2) and [hi2, hi) are seen in part
          const int lo = max(first, 0), hi = last + 1, lo2 = min(max(all_first, lo), BN), hi2 = max(all_last + 1, 0);
          const uint32_t wanted = hi > lo ? ((2u << ((hi - 1) >> 4)) - 1) & ~((1u << (lo >> 4)) - 1) : 0;
          if (hi > lo && lo2 <= hi2 && (sk <= 0 || all_first <= 0) && (there & wanted) == wanted) {
            clean_rows(lo, lo2);
            clean_rows(hi2, hi);
            zero_rows(0, lo);
            zero_rows(hi, BN);
          } else {
#pragma unroll 1
            for (int x = me; x < BN * PIECES; x += N) {
              const int row = x / PIECES;
              const bool in = (there >> (row >> 4)) & 1;
              if (in && row <= all_last && (row >= all_first || row < sk)) continue;
              if (in && row <= last && (row >= first || row < sk))
                clean(*piece(x), piece(x));
              else
                *piece(x) = make_uint4(0, 0, 0, 0);
            }
          }
          if (found) note_bad(seg);
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c->fixed[n % NS]);
        }
      }
    } else if (Q8 && warp == G::W_COPY) {
      // Q8: codes and scales into the staging ring
      char* const raw = tiles + G::QALL + NS * G::KB;
      uint32_t n = 0;
      int row = w.live() ? lookup(w, w.i0) : -1;
      while (w.live()) {
        for (int i = w.i0; i < w.i1; ++i) {
          const int now = row;
          if (i + 1 < w.i1) row = lookup(w, i + 1);              // the next tile's page entries on their way
          const uint32_t there = there_of(now);
          const uint32_t bytes = __popc(__ballot_sync(~0u, now >= 0)) * ((HD + HD / 16) << bl);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv, ++n) {
            char* const to = raw;
            uint64_t* bar = &c->raw;
            pt_wait_warp(c, &c->raw_free, (n & 1) ^ 1);
            if (lane == 0) {
              if (kv == 0) *reinterpret_cast<volatile uint32_t*>(&c->there[(n / 2) & 7]) = there;
              mbar_arrive_expect_tx(bar, bytes);
            }
            __syncwarp();
            if (now >= 0) {
              const size_t at = static_cast<size_t>(now) * HD;
              bulk_g2s(to + (lane << bl) * HD, static_cast<const char*>(kv ? a.kv.v : a.kv.k) + at, HD << bl, bar);
              bulk_g2s(to + BN * HD + (lane << bl) * (HD / 16), reinterpret_cast<const char*>(kv ? a.kv.vs : a.kv.ks) + at / 16,
                       (HD / 16) << bl, bar);
            }
          }
        }
        w.next(a);
        if (w.live()) row = lookup(w, w.i0);
      }
      if (n > 0) pt_drain(&c->raw, (n - 1) & 1);
    } else if (Q8 && warp < 8 + G::CONV) {
      // Q8: staged codes to binary16
      constexpr int PIECES = BN * HD / 16;               // 16 codes each
      const char* const raw = tiles + G::QALL + NS * G::KB;
      uint32_t n = 0;                                    // tiles stored (keys and values)
      int seg = 0;
      for (; w.live(); ++seg, next_segment()) {
        for (int i = w.i0; i < w.i1; ++i) {
          const TileView tv = tile_view<BN>(a, w.it, i);
          const int last = w.it.p1 - tv.base, first = a.window ? max(w.it.p0, 0) - a.window + 1 - tv.base : 0, sk = a.sinks - tv.base;
          const int all_last = w.it.p0 - tv.base, all_first = a.window ? w.it.p1 - a.window + 1 - tv.base : 0;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const uint32_t slot = n % NS;
            pt_wait_warp(c, &c->raw, n & 1);
            const uint32_t there = *reinterpret_cast<volatile uint32_t*>(&c->there[(n / 2) & 7]);
            const bool clean = kv == 1 && !(tv.whole && there == ALL);
            // Groups of 32 pieces go round the warps from tile to tile.  A warp's are taken into registers at once, so
            // that the next tile is staged while they are converted (one staging place: two would cost a ring slot,
            // without which the conversion of a tile waits for the products with the last).
            constexpr int PARTS = PIECES / 32, MOST = (PARTS + G::CONV - 1) / G::CONV;
            const int j0 = (warp - G::W_SIDE + G::CONV - static_cast<int>(n * PARTS % G::CONV)) % G::CONV;
            uint4 codes[MOST];
            __half sc[MOST];
#pragma unroll
            for (int y = 0; y < MOST; ++y) {
              const int x = min(j0 + y * G::CONV, PARTS - 1) * 32 + lane;
              codes[y] = *reinterpret_cast<const uint4*>(raw + x * 16);
              sc[y] = *reinterpret_cast<const __half*>(raw + BN * HD + (x >> 1) * 2);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->raw_free);
            pt_wait_warp(c, &c->empty[slot], ((n / NS) & 1) ^ 1);
            char* const dst = tiles + G::QALL + slot * G::KB;
            bool found = false;
            auto convert = [&](auto cleaning) {          // (code of its own for the few tiles to be cleaned)
#pragma unroll
              for (int y = 0; y < MOST; ++y) {
                if (j0 + y * G::CONV >= PARTS) break;
                const int x = (j0 + y * G::CONV) * 32 + lane, row = x / (HD / 16), pc = x % (HD / 16);
                uint4 u[2];
                __half2* h = reinterpret_cast<__half2*>(u);
                const __half2 d = __half2half2(sc[y]);
                // the two halves of a piece in an order that keeps 8 lanes' stores in different banks
                const bool odd = (pc >> 2) & 1;
                q8_values4(odd ? codes[y].z : codes[y].x, d, h[0], h[1]);
                q8_values4(odd ? codes[y].w : codes[y].y, d, h[2], h[3]);
                q8_values4(odd ? codes[y].x : codes[y].z, d, h[4], h[5]);
                q8_values4(odd ? codes[y].y : codes[y].w, d, h[6], h[7]);
                if (decltype(cleaning)::value) {
                  // as binary16's: what every row sees stays as it is (add_taken_out passes over a tile of such positions
                  // alone, holes or not)
                  const bool in = (there >> (row >> 4)) & 1, all = in && row <= all_last && (row >= all_first || row < sk);
                  if (!all && in && row <= last && (row >= first || row < sk)) {
                    uint32_t* b = reinterpret_cast<uint32_t*>(u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                      if ((b[e] & 0x7c00u) == 0x7c00u) b[e] &= 0xffff0000u, found = true;
                      if ((b[e] & 0x7c000000u) == 0x7c000000u) b[e] &= 0x0000ffffu, found = true;
                    }
                  } else if (!all) {
                    u[0] = u[1] = make_uint4(0, 0, 0, 0);
                  }
                }
                char* to = dst + (pc >> 2) * (BN * 128) + row * 128;
                const int p0 = (pc & 3) * 2 + odd;
                *reinterpret_cast<uint4*>(to + ((p0 ^ (row & 7)) << 4)) = u[0];
                *reinterpret_cast<uint4*>(to + (((p0 ^ 1) ^ (row & 7)) << 4)) = u[1];
              }
            };
            if (clean)
              convert(std::true_type{});
            else
              convert(std::false_type{});
            if (found) note_bad(seg);
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->full[slot]);
          }
        }
      }
    }
  } else if (warp == G::W_MMA) {
    // ---------------------------------------------------------------- products
    // The whole warp walks; one elected lane issues.  Warp-uniform values let
    // the descriptors live in uniform registers.
    constexpr uint32_t ID_S = mma_idesc(BN, false), ID_O = mma_idesc(HD, true);
    constexpr uint64_t BLOCK = (BN * 128) >> 4;         // next 64 values of head_dim, in descriptor units
    const bool one = elect_one();
    RingAt<NS> at_k, at_v;                               // the next key and value tile
    at_v.step();
    uint32_t n_v = 0;                                    // value tiles: turns of their slots
    uint32_t par_q[2] = {0, 0}, par_p[2] = {0, 0}, par_s = 0;
    for (; w.live(); w.next(a)) {
      const int active = __shfl_sync(~0u, w.rows() > 128 ? NQ : 1, 0);
      const int cnt = __shfl_sync(~0u, w.i1 - w.i0, 0);
      auto wait_v = [&](const RingAt<NS>& at, uint32_t n) {
        pt_wait_warp(c, &c->full[at.slot], at.parity);
        if (!Q8) pt_wait_warp(c, &c->fixed[at.slot], at.turn(n) & 1);
      };
      auto scores = [&](int q) {                         // S of query tile q with the key tile at_k
        if (one) {
          const uint64_t k0 = mma_sdesc(s_ring + at_k.slot * G::KB, 0);
          const uint32_t d = NQ == 2 ? tmem + q * 128 : tmem + par_s * BN;
#pragma unroll
          for (int part = 0; part < (QF32 ? 2 : 1); ++part) {
            uint32_t q_at = s_q + (QF32 ? part : q) * G::QB;
            asm volatile("" : "+r"(q_at));               // (descriptors formed here, not kept in registers)
            const uint64_t q0 = mma_sdesc(q_at, 0);
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
              tm_mma_ss(d, q0 + (k >> 2) * ((128 * 128) >> 4) + (k & 3) * 2, k0 + (k >> 2) * BLOCK + (k & 3) * 2, ID_S,
                        part > 0 || k > 0);
          }
          tm_commit(&c->s_full[NQ == 2 ? q : par_s]);
        }
      };
      auto values = [&](int q, uint32_t p_at, int h, bool add) {     // O += P V, half h
        if (one) {
          const uint64_t v0 = mma_sdesc(s_ring + at_v.slot * G::KB, BN * 128) + h * (G::H / 16) * (2048 >> 4);
#pragma unroll
          for (int k = 0; k < G::H / 16; ++k)
            tm_mma_ts(tmem + G::O_COL + q * 128, p_at + h * (G::H / 2) + k * 8, v0 + k * (2048 >> 4), ID_O, add || k > 0);
          tm_commit(&c->o_full[q][h]);
        }
      };
      pt_wait_warp(c, &c->full[at_k.slot], at_k.parity);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (q >= active) break;
        pt_wait_warp(c, &c->q_full[q], par_q[q]);
        par_q[q] ^= 1;
        tm_after();
        scores(q);
      }
      if (one) tm_commit(&c->empty[at_k.slot]);
      at_k.step(), at_k.step();
      for (int i = 0; i < cnt; ++i) {
        const bool more = i + 1 < cnt;
        if (NQ == 1) {
          // the next scores go ahead of this tile's weights, into the other place
          const uint32_t now = par_s;
          par_s ^= 1;
          if (more) {
            pt_wait_warp(c, &c->full[at_k.slot], at_k.parity);
            tm_after();
            scores(0);
            if (one) tm_commit(&c->empty[at_k.slot]);
            at_k.step(), at_k.step();
          }
          wait_v(at_v, n_v);
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            pt_wait_warp(c, &c->p_full[now][h], par_p[now]);
            tm_after();
            values(0, tmem + now * BN, h, i > 0 || h > 0);
          }
          par_p[now] ^= 1;
        } else {
          wait_v(at_v, n_v);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (q >= active) break;
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              pt_wait_warp(c, &c->p_full[q][h], par_p[q]);
              tm_after();
              values(q, tmem + q * 128, h, i > 0 || h > 0);
            }
            par_p[q] ^= 1;
            if (more) {
              if (q == 0) pt_wait_warp(c, &c->full[at_k.slot], at_k.parity);
              tm_after();
              scores(q);
            }
          }
          if (more) {
            if (one) tm_commit(&c->empty[at_k.slot]);
            at_k.step(), at_k.step();
          }
        }
        if (one) tm_commit(&c->empty[at_v.slot]);
        at_v.step(), at_v.step();
        ++n_v;

      }
    }
    if (one) tm_commit(&c->done);
    __syncwarp();
    pt_drain(&c->done, 0);
  }
  if (tid == 0) *parts.record(blockIdx.x) = rec;
  __syncwarp();
  tm_before();
  __syncthreads();
  if (warp == G::W_MMA) {
    tm_after();
    tm_free(tmem, 512);
  }
}

template <int HD, bool QF32, bool Q8>
cudaError_t prepare_tile() {
  // the warps' register split must fit what a block is launched with (it waits for registers otherwise)
  cudaFuncAttributes at;
  const cudaError_t e = cudaFuncGetAttributes(&at, paged_tile_kernel<HD, QF32, Q8>);
  if (e != cudaSuccess) return e;
  if ((at.numRegs + 7) / 8 * 8 * Pt<HD, QF32, Q8>::THREADS < Pt<HD, QF32, Q8>::REGS) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(paged_tile_kernel<HD, QF32, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Pt<HD, QF32, Q8>::SMEM);
}

template <int HD>
cudaError_t prepare_hd() {
  const cudaError_t e[4] = {prepare_tile<HD, false, false>(), prepare_tile<HD, false, true>(),
                            prepare_tile<HD, true, false>(), prepare_tile<HD, true, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

template <int HD, bool QF32, bool Q8>
cudaError_t launch_tile(const PagedAttnArgs& a, void* ws, int grid, cudaStream_t s) {
  using G = Pt<HD, QF32, Q8>;
  PartSlots parts{static_cast<char*>(ws), G::R, HD};
  PtMaps maps = {};
  if (!Q8) {
    maps.box_log2 = a.kv.page_log2 < (G::BN == 128 ? 7 : 6) ? a.kv.page_log2 : (G::BN == 128 ? 7 : 6);
    const int64_t rows = static_cast<int64_t>(a.kv.n_pages) * a.kv.n_kv << a.kv.page_log2;
    if (!encode_f16_rows(&maps.k, a.kv.k, rows, HD, 1 << maps.box_log2) ||
        !encode_f16_rows(&maps.v, a.kv.v, rows, HD, 1 << maps.box_log2))
      return cudaErrorInvalidValue;
  }
  paged_tile_kernel<HD, QF32, Q8><<<grid, G::THREADS, G::SMEM, s>>>(a, parts, maps);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : paged_join_launch(a, parts, grid, s);
}

template <int HD>
cudaError_t launch_hd(const PagedAttnArgs& a, bool f32, bool q8, void* ws, int grid, cudaStream_t s) {
  if (f32) return q8 ? launch_tile<HD, true, true>(a, ws, grid, s) : launch_tile<HD, true, false>(a, ws, grid, s);
  return q8 ? launch_tile<HD, false, true>(a, ws, grid, s) : launch_tile<HD, false, false>(a, ws, grid, s);
}

}  // namespace

cudaError_t paged_tile_prepare() {
  const cudaError_t e[4] = {prepare_hd<64>(), prepare_hd<128>(), prepare_hd<192>(), prepare_hd<256>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t paged_tile_launch(const PagedAttnArgs& a, bool q_f32, bool q8, void* ws, int grid, cudaStream_t s) {
  switch (a.kv.hd) {
    case 64: return launch_hd<64>(a, q_f32, q8, ws, grid, s);
    case 128: return launch_hd<128>(a, q_f32, q8, ws, grid, s);
    case 192: return launch_hd<192>(a, q_f32, q8, ws, grid, s);
    default: return launch_hd<256>(a, q_f32, q8, ws, grid, s);
  }
}

cudaError_t paged_read_status(int* out) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_status_pt, sizeof(int));
  if (e != cudaSuccess || *out == 0) return e;
  return cudaMemcpyToSymbol(g_status_pt, &zero, sizeof(int));
}

}  // namespace q4
