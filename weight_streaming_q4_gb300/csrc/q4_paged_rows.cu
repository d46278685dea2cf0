// Attention of few query rows over a paged KV cache (sm_103a): single tokens and
// short drafts, where reading the keys and values is all there is to do.
//
// An item (q4_paged_sched.cuh) is R = 8 to 32 query rows of one value head, its
// units are 32 positions.  Persistent, one CTA per SM.  Within a CTA every warp
// works for itself: it takes every W-th group of 16 positions of the CTA's
// units, copies their keys and values into its own ring with 16-byte cp.async
// (several groups in flight per warp, no barrier between the warps), and keeps its own
// maximum, sum and output of every row, so that nothing but the memory paces it.
// The warps' results meet in shared memory once per item.  The ring runs across
// items: the next item's keys are on their way while an item is finished.
//
// Both products are mma.sync m16n8k16 (binary16 in, fp32 sums) with the positions,
// then the value's columns, as its 16 rows and the query rows as its 8 columns: a
// group of 4 or 8 query heads fills it, where a tcgen05 operand has 128 rows (with the query rows as
// the 16, half of products, weights and output registers of such a group were zeros: 64
// sequences of the 70B heads over Q8 175 us, so 133 at that step).  The scores' registers become the weights'
// operand by one 8 x 8 transposition each.  fp32 queries enter as two binary16 parts of a scaled row (QueryScale).
// The weights are rounded to binary16 once, as in the kernel of many rows (which one runs must not show beyond
// the rounding): 2^-11 relative, as much as the output's own rounding; their sum is taken before it, in fp32.
// Q8 pages stay codes in shared memory: a lane's 16 codes of a key are its share
// of four instructions (the order of head_dim in the product is free, the
// queries follow it), a transposed matrix load of value codes holds two columns of one
// position pair per register; f16(code * d) is formed in registers.
//
// Measured, back to back in a graph: 64 sequences of the 70B heads of up to 8192 positions, binary16 180 us, 6.3 TB/s
// (93 % of a copy's rate); Q8 127 us, 4.8 TB/s: the issue slots, 67 % busy, of which the
// conversion takes 7 instructions per 4 values.  One token of the 8B heads over 512 and 4096 positions 4.8 and
// 7.7 us (8.3 and 11.8 where the table is too wide for clusters): the launch and a chain of dependent loads.
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "q4_paged_sched.cuh"

namespace q4 {

namespace {

// CL: the CTAs of a cluster share every item (ClusterWalk).
constexpr int kPrCluster = 8;

template <int HD, int NR, bool QF32, bool Q8, bool CL>
struct Pr {
  // Positions of a group, a warp's step.  At head_dim 64 a step of 32 pays the comparison with the
  // maximum and the copies' addresses half as often (16 sequences under a window 12.7 us against 13.4); above, it
  // takes the registers of the warps that hide its latency.
  static constexpr int GP = HD == 64 && NR <= 2 ? 32 : 16;
  // Warps, as many as the registers allow (outputs: HD * NR / 4 of them) for Q8, whose conversion makes it the issue
  // slots that count: 64 sequences of the 70B heads 133 us with 16, 139 with 12, 144 with 14, whose rings hold no more than 16's.
  // binary16 pages wait for memory, and the slots of the rings count.
  // At head_dim 64 12 of them hide more (the window's case 12.0 us against 12.8, 64 sequences over Q8 82 against 92), and a cluster,
  // which has few steps, meets sooner with 8 (one token over 4096 positions 5.8 against 5.9).
  static constexpr int W = HD > 128                          ? 4
                           : HD == 128 && Q8 && NR <= 2 ? (NR == 1 ? 16 : 12)
                           : HD == 64 && NR == 1 && !CL ? 12
                                                        : 8;
  static constexpr int NT = W * 32;
  static constexpr int R = 8 * NR;
  static constexpr int KS = HD / 16;                        // products of a key group
  static constexpr int ROW = Q8 ? HD : 2 * HD;              // bytes of a staged key
  static constexpr int SC = Q8 ? HD / 32 * 2 * GP : 0;      // bytes of a group's scales
  static constexpr int STAGE = 2 * GP * ROW + 2 * SC;       // keys, values, their scales
  static constexpr int PITCH = HD + 4;                      // floats of a row of the warps' results
  static constexpr bool QREG = NR == 1 && W <= 8;           // queries stay in registers (one token, 4096 positions: 7.8 us against 8.1)
  static constexpr int QB = NR * KS * 32 * (QF32 ? 16 : 8); // queries as operands
  static constexpr int RM = NR == 1 ? 8 : 16;               // rows that meet at a time
  static constexpr int MERGE = (W * RM * PITCH * 4 + 2 * W * R * 4 + 511) / 512 * 512;
  // In a cluster the ring is empty when the results meet, and they take its place.
  static constexpr int JOINED = CL ? R * (HD + 2) * 4 : 0;  // the CTA's result for the others of its cluster
  static constexpr int FIT = (231424 - 1024 - QB - (CL ? 0 : MERGE)) / (W * STAGE);
  static constexpr int NS = FIT > 6 ? 6 : FIT;              // stages per warp
  static constexpr int RING = W * NS * STAGE;
  static constexpr int SMEM = 1024 + QB + (CL ? (RING > MERGE + JOINED ? RING : MERGE + JOINED) : MERGE + RING);
  static_assert(NS >= 2, "a group is copied while one is read");
  static_assert(ROW > 512 || 512 % ROW || ((1024 + QB) % ROW == 0 && MERGE % ROW == 0 && STAGE % ROW == 0), "groups start on a multiple of the row");
};

struct PrCtl {
  CtaWork work;
  long long scan[17];
  int bad;                 // segment number + 1 in whose partly seen values a warp met infinities or NaN
  uint32_t there[16][8];   // per warp and stage: bit i = positions 16 i .. of the group are in a page
  alignas(8) float scale[32];      // fp32 queries: what a row's scores are multiplied by
};
static_assert(sizeof(PrCtl) <= 1024, "control data fits its place");

__device__ __forceinline__ void pr_cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void pr_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void pr_ldsm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void pr_ldsm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ uint4 pr_lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// The 8 x 8 matrix of which lane (g, t) holds row g, columns 2t and 2t + 1, transposed.
__device__ __forceinline__ uint32_t pr_transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void pr_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// All CTAs of the cluster, with what they wrote to shared memory.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this CTA's shared-memory address `at` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_at(uint32_t at, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float cluster_ld(uint32_t at) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ float pr_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// u with infinities and NaN replaced by zero; *found is set if there were any.
__device__ __forceinline__ uint32_t pr_finite(uint32_t u, bool* found) {
  if ((u & 0x7c00u) == 0x7c00u) u &= 0xffff0000u, *found = true;
  if ((u & 0x7c000000u) == 0x7c000000u) u &= 0x0000ffffu, *found = true;
  return u;
}

// The place of 16-byte piece `c` in row `r` of a staged group.  Matrix loads
// take the same piece of 8 consecutive rows: the pieces of 128 bytes' worth of banks
// are exchanged by row so that these fall apart.  Keys as Q8 are read by lanes
// of two rows and four pieces at a time instead.
template <int ROW, bool KEY8>
__device__ __forceinline__ int place(int r, int c) {
  if (KEY8) return ROW % 128 == 0 ? r * ROW + ((c ^ ((r & 1) << 2)) << 4) : r * ROW + (c << 4);
  if (ROW % 128 == 0) return r * ROW + ((c ^ (r & 7)) << 4);
  return r * ROW + ((c ^ ((r >> 1) & 3)) << 4);
}

// Rows whose pieces' numbers are whole bits of the address (a group starts on a multiple of the row): the place of
// piece c ^ x is that of piece c, xored with x * 16.
template <int ROW>
constexpr bool kByXor = ROW == 128 || ROW == 256 || ROW == 512;

template <bool CL, int R>
struct WalkOf {
  using T = SegmentWalk<R, 32>;
};
template <int R>
struct WalkOf<true, R> {
  using T = ClusterWalk<R, 32>;
};

// A warp's groups, segment by segment: those of the copies run ahead of those
// of the products.
template <int R, int W, int GP, bool CL>
struct GroupWalk {
  typename WalkOf<CL, R>::T w;
  int g, n;             // the warp's current group of the segment, and the segment's groups
  __device__ __forceinline__ void count() {
    n = 32 / GP * (w.i1 - w.i0);
    if (GP == 16 && n > 0 && w.i1 == w.it.cnt && (w.it.p1 & 31) < 16) --n;      // the last tile's second half holds no position seen
    if (w.it.p1 < 0) n = 0;
  }
  __device__ __forceinline__ int base_of(int g) const {
    return GP == 32 ? w.it.tile(w.i0 + g) * 32 : w.it.tile(w.i0 + (g >> 1)) * 32 + (g & 1) * 16;
  }
};

template <int HD, int NR, bool QF32, bool Q8, bool CL>
__global__ void __launch_bounds__(Pr<HD, NR, QF32, Q8, CL>::NT, 1)
    paged_rows_kernel(const __grid_constant__ PagedAttnArgs a, PartSlots parts) {
  using G = Pr<HD, NR, QF32, Q8, CL>;
  constexpr int W = G::W, R = G::R, NS = G::NS, KS = G::KS, ROW = G::ROW, PIECES = ROW / 16;
  constexpr int GP = G::GP, SUB = GP / 16;
  constexpr bool TWO = NR * SUB <= 2;     // few sums of scores: two each, of the parts of an fp32 query or of every other product
  extern __shared__ __align__(512) char smem_pr[];     // (kByXor)
  PrCtl* c = reinterpret_cast<PrCtl*>(smem_pr);
  using Query = typename std::conditional<QF32, uint4, uint2>::type;
  Query* s_q = reinterpret_cast<Query*>(smem_pr + 1024);                  // [NR][KS][lane]
  float* s_o = reinterpret_cast<float*>(smem_pr + 1024 + G::QB);          // [W][RM][PITCH]
  float* s_m = s_o + W * G::RM * G::PITCH;                                // [W][R]
  float* s_l = s_m + W * R;
  float* s_joined = s_l + W * R;                                          // CL: [R][HD], maxima [R], sums [R]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem_pr + 1024 + G::QB + (CL ? 0 : G::MERGE)) + warp * NS * G::STAGE;

  if (!CL) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) c->bad = 0;
  JoinRecord rec = {};       // thread 0's
  long long per = 1;
  GroupWalk<R, W, GP, CL> u, cp;
  if constexpr (CL) {
    u.w.begin(a, blockIdx.x / kPrCluster, gridDim.x / kPrCluster, blockIdx.x % kPrCluster, kPrCluster);
  } else {
    CtaWork work;
    if (a.b.n_seqs <= 32) {
      work = warp_work<R, 32>(a);
    } else {
      cta_work<R, 32, G::NT>(a, c->scan, &c->work);
      work = c->work;
    }
    per = work.per;
    u.w.begin(a, work);
  }

  // ------------------------------------------------------------------ copies
  cp.w = u.w;
  int st_cp = 0, st_use = 0;      // the next stage to copy into, to read
  // Page rows of the warp's next 32 / SUB groups in cp's segment, 16 positions per lane, from its group rows0 on.
  int rows_of = -1, rows0 = 0;
  auto look_up = [&]() {
    const int g = cp.g + lane / SUB * W;
    rows0 = cp.g;
    const int at = g < cp.n ? cp.base_of(g) + lane % SUB * 16 : 0;
    rows_of = g < cp.n && at <= cp.w.it.p1 ? paged_row(a.kv, a.b, cp.w.seq, at, cp.w.head) : -1;
  };
  auto enter = [&]() {      // cp's segment
    cp.g = warp;
    cp.count();
    look_up();
  };
  // 16 rows of keys or values to `to`.  Where a row's pieces divide a warp's 32, a lane's pieces lie 512 bytes apart, but
  // for the exchange, whose part that changes from one to the next is a constant: no addresses to compute
  // (64 sequences over Q8 127.5 us against 132.7, 32 rows 37.7 against 38.4).
  auto pieces = [&](uint32_t to, const char* from, auto key8) {
    constexpr bool K8 = decltype(key8)::value;
    if constexpr (32 % PIECES == 0) {
      const uint32_t d = to + place<ROW, K8>(lane / PIECES, lane % PIECES);
      const char* f = from + lane * 16;
#pragma unroll
      for (int i = 0; i < PIECES / 2; ++i)
        pr_cp16((d ^ (kByXor<ROW> && !K8 ? (i * (32 / PIECES) & 7) << 4 : 0)) + i * 512, f + i * 512);
    } else {
#pragma unroll
      for (int x = lane; x < 16 * PIECES; x += 32) pr_cp16(to + place<ROW, K8>(x / PIECES, x % PIECES), from + x * 16);
    }
  };
  auto copy = [&]() {       // the warp's next group into the next stage; always one commit
    if (!CL) {
      while (cp.w.live() && cp.g >= cp.n) {
        cp.w.next(a);
        if (cp.w.live()) enter();
      }
    }
    if (cp.w.live() && cp.g < cp.n) {
      if (cp.g - rows0 >= 32 / SUB * W) look_up();
      const int stage = st_cp;
      const uint32_t to = ring + stage * G::STAGE;
      uint32_t there = 0;
#pragma unroll
      for (int sub = 0; sub < SUB; ++sub) {
        const int r0 = __shfl_sync(~0u, rows_of, (cp.g - rows0) / W * SUB + sub);
        if (r0 < 0) {
          // no page, or positions that no row sees: what counts beside weights of zero is that the values are finite
          if (SUB > 1) {
            constexpr int N = Q8 ? G::SC / SUB / 16 : 16 * PIECES;
            const uint32_t at = Q8 ? to + 2 * GP * ROW + G::SC + sub * (G::SC / SUB) : to + GP * ROW + sub * 16 * ROW;
#pragma unroll 1
            for (int x = lane; x < N; x += 32)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + x * 16), "r"(0) : "memory");
          }
          continue;
        }
        there |= 1u << sub;
        const char* k = static_cast<const char*>(a.kv.k) + static_cast<size_t>(r0) * ROW;
        const char* v = static_cast<const char*>(a.kv.v) + static_cast<size_t>(r0) * ROW;
        pieces(to + sub * 16 * ROW, k, std::integral_constant<bool, Q8>{});
        if (Q8) {
          constexpr int SP = G::SC / SUB / 16;               // 16-byte pieces of 16 positions' scales
          const char* ks = reinterpret_cast<const char*>(a.kv.ks) + static_cast<size_t>(r0) * (HD / 16);
          const char* vs = reinterpret_cast<const char*>(a.kv.vs) + static_cast<size_t>(r0) * (HD / 16);
          const uint32_t sc = to + 2 * GP * ROW + sub * SP * 16;
          const bool of_v = lane >= SP;
          const int x = (of_v ? lane - SP : lane) * 16;
          if (lane < 2 * SP) pr_cp16(sc + (of_v ? G::SC : 0) + x, (of_v ? vs : ks) + x);
        }
        pieces(to + GP * ROW + sub * 16 * ROW, v, std::false_type{});
      }
      if (lane == 0) c->there[warp][stage] = there;
      st_cp = st_cp + 1 == NS ? 0 : st_cp + 1;
      cp.g += W;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (cp.w.live()) enter();

  // ------------------------------------------------------------------ items
  int seg = 0;
  for (; u.w.live(); u.w.next(a), ++seg) {
    const auto& w = u.w;
    const int rows = w.rows(), row0 = w.j * R, first = w.sp.len - w.sp.n_new;
    if constexpr (!CL) join_note(&rec, w, per);
    if (CL && seg > 0) {
      cp.w = u.w;
      enter();
    }
    // queries in operand order: lane (g, t) of product ks holds row g
    constexpr int RW = QF32 ? (R + W - 1) / W : 1;       // fp32: a warp per row, whose largest element it needs (QueryScale)
    float2 qf[RW][HD / 64];                              // element pairs j * 64 + 2 * lane
    if constexpr (QF32) {
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const int rr = k * W + warp;
        const int64_t at = rr < rows ? a.row_at(w.sp.t0, w.head, row0 + rr, a.q_ld) + lane * 2 : -1;
#pragma unroll
        for (int j = 0; j < HD / 64; ++j) {
          qf[k][j] = make_float2(0.f, 0.f);
          if (at >= 0) qf[k][j] = __ldg(reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at + j * 64));
        }
      }
    } else {
      for (int x = tid; x < NR * KS * 32; x += G::NT) {
        const int nr = x / (KS * 32), ks = x / 32 % KS, xl = x & 31, xt = xl & 3, rr = nr * 8 + (xl >> 2);
        const int e0 = Q8 ? (xt + 4 * (ks >> 2)) * 16 + 4 * (ks & 3) : ks * 16 + xt * 2;
        uint32_t hi[2] = {0, 0};
        if (rr < rows) {
          const int64_t at = a.row_at(w.sp.t0, w.head, row0 + rr, a.q_ld) + e0;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            hi[i] = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __half*>(a.q) + at + i * (Q8 ? 2 : 8)));
        }
        s_q[x] = make_uint2(hi[0], hi[1]);
      }
    }
    if (CL || seg == 0) {
#pragma unroll 1
      for (int i = 0; i < NS - 1; ++i) copy();
    }
    if constexpr (QF32) {      // (after the copies are on their way: it waits for the queries)
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        const int rr = k * W + warp;
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < HD / 64; ++j) most = max(most, abs_bits(qf[k][j]));
        const QueryScale qs(__reduce_max_sync(~0u, most));
        if (rr >= R) break;
        if (lane == 0) c->scale[rr] = a.scale * qs.down;
        uint32_t* const to = reinterpret_cast<uint32_t*>(s_q + rr / 8 * KS * 32 + rr % 8 * 4);
#pragma unroll
        for (int j = 0; j < HD / 64; ++j) {
          const int e = j * 64 + lane * 2, in = e & 15;
          const int ks = Q8 ? e / 64 * 4 + in / 4 : e / 16, xt = Q8 ? e / 16 & 3 : in / 2 & 3, i = Q8 ? in / 2 & 1 : in / 8;
          __half2 hi, lo;
          query_parts(qf[k][j], qs.up, &hi, &lo);
          to[(ks * 32 + xt) * 4 + i] = as_u32(hi);
          to[(ks * 32 + xt) * 4 + i + 2] = as_u32(lo);
        }
      }
    }
    // of this lane's rows 2t, 2t + 1 of every 8
    int p[NR][2];              // positions
    float m[NR][2], l[NR][2];
    float o[NR][KS][4];        // columns g (two of them) of 16, in rows 2t, 2t + 1
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rr = nr * 8 + 2 * t + h;
        p[nr][h] = rr < rows ? first + a.token_of(row0 + rr) : -1;
        m[nr][h] = -INFINITY, l[nr][h] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < KS; ++n) o[nr][n][0] = o[nr][n][1] = o[nr][n][2] = o[nr][n][3] = 0.f;
    }
    __syncthreads();           // queries are there
    u.count();
    bool found = false;
    Query qr[G::QREG ? KS : 1];
    if (G::QREG) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qr[G::QREG ? ks : 0] = s_q[ks * 32 + lane];
    }
    float scale[NR][2];        // of this lane's rows' scores
    auto scales = [&]() {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        scale[nr][0] = scale[nr][1] = a.scale;
        if (QF32)
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(scale[nr][0]), "=f"(scale[nr][1]) : "r"(smem_u32(&c->scale[nr * 8 + 2 * t])));
      }
    };
    scales();
    for (u.g = warp; u.g < u.n; u.g += W) {
      copy();
      pr_wait<NS - 1>();
      __syncwarp();
      const int stage = st_use;
      st_use = st_use + 1 == NS ? 0 : st_use + 1;
      const uint32_t at = ring + stage * G::STAGE;
      const int base = u.base_of(u.g);
      const uint32_t there = c->there[warp][stage];
      if (there) {
        const bool whole = there == (1u << SUB) - 1 && base + GP - 1 <= w.it.p0 &&
                           (!a.window || base > w.it.p1 - a.window || base + GP <= a.sinks);
        if (!whole) {
          // Values that no row sees become zeros (Q8: their scales), and are not noted: what lies behind the last
          // position may be anything.
          constexpr int N = Q8 ? HD / 32 : PIECES;       // stores per position
#pragma unroll 1
          for (int x = lane; x < GP * N; x += 32) {
            const int r = x / N, pos = base + r;
            if (pos <= w.it.p1 && (!a.window || pos > w.it.p0 - a.window || pos < a.sinks)) continue;
            if (Q8)
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 2 * GP * ROW + G::SC + x * 2), "h"(static_cast<uint16_t>(0)) : "memory");
            else
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + GP * ROW + x * 16), "r"(0) : "memory");
          }
          __syncwarp();
        }
        // where this lane's first pieces lie
        const uint32_t kat = at + (Q8 ? place<ROW, true>(g, t) : place<ROW, false>(lane & 7, lane >> 3));
        const uint32_t vat = at + GP * ROW + place<ROW, false>((lane & 7) + (lane & 8), lane >> 4);
        // ---- scores: of positions g, g + 8 (of 16), rows 2t, 2t + 1
        float s[NR][SUB][4], s2[NR][SUB][4];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 4 * SUB; ++e) s[nr][e >> 2][e & 3] = s2[nr][e >> 2][e & 3] = 0.f;
        auto product = [&](int sub, int ks, uint32_t k0, uint32_t k1, uint32_t k2, uint32_t k3) {
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            const Query q = G::QREG ? qr[G::QREG ? ks : 0] : s_q[(nr * KS + ks) * 32 + lane];
            pr_mma(TWO && !QF32 && (ks & 1) ? s2[nr][sub] : s[nr][sub], k0, k1, k2, k3, q.x, q.y);
            if constexpr (QF32) pr_mma(TWO ? s2[nr][sub] : s[nr][sub], k0, k1, k2, k3, q.z, q.w);
          }
        };
        if (!Q8) {
#pragma unroll
          for (int k2 = 0; k2 < KS / 2; ++k2)
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
              uint32_t r[2][4];
#pragma unroll
              for (int i = 0; i < 2; ++i)
                pr_ldsm(r[i], kByXor<ROW> ? (kat ^ (k2 << 6)) + (sub * 16 + i * 8) * ROW
                                          : at + place<ROW, false>(sub * 16 + i * 8 + (lane & 7), k2 * 4 + (lane >> 3)));
              product(sub, 2 * k2, r[0][0], r[1][0], r[0][1], r[1][1]);
              product(sub, 2 * k2 + 1, r[0][2], r[1][2], r[0][3], r[1][3]);
            }
        } else {
#pragma unroll
          for (int j = 0; j < HD / 64; ++j)
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
              __half2 h[2][8];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int pos = sub * 16 + i * 8 + g;
                const uint4 q = pr_lds16(kByXor<ROW> ? (kat ^ (j << 6)) + (sub * 16 + i * 8) * ROW : at + place<ROW, true>(pos, t + 4 * j));
                uint16_t d;
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=h"(d)
                             : "r"(at + 2 * GP * ROW + pos * (HD / 16) + ((t >> 1) + 2 * j) * 2)
                             : "memory");
                const __half2 d2 = __half2half2(__ushort_as_half(d));
                q8_values4(q.x, d2, h[i][0], h[i][1]);
                q8_values4(q.y, d2, h[i][2], h[i][3]);
                q8_values4(q.z, d2, h[i][4], h[i][5]);
                q8_values4(q.w, d2, h[i][6], h[i][7]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                product(sub, 4 * j + k, as_u32(h[0][2 * k]), as_u32(h[1][2 * k]), as_u32(h[0][2 * k + 1]), as_u32(h[1][2 * k + 1]));
            }
        }
        if (TWO) {
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 4 * SUB; ++e) s[nr][e >> 2][e & 3] += s2[nr][e >> 2][e & 3];
        }
        if (!whole) {
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 4 * SUB; ++e) {
              const int pr = p[nr][e & 1], x = base + (e >> 1) * 8 + g;
              if (x > pr || (a.window && x <= pr - a.window && x >= a.sinks) || !((there >> (e >> 2)) & 1))
                s[nr][e >> 2][e & 3] = -INFINITY;
            }
        }
        // ---- weights
        if (QF32 && NR > 1) scales();        // (loaded again: kept in registers, they spill)
        // (a row's maximum is wanted of all lanes only when one of them has raised it)
        float top[NR][2];
        bool raise = false;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = -INFINITY;
#pragma unroll
            for (int e = h; e < 4 * SUB; e += 2) x = fmaxf(x, s[nr][e >> 2][e & 3]);
            x *= scale[nr][h];
            top[nr][h] = x;
            raise |= x > m[nr][h] + 8.f || (m[nr][h] == -INFINITY && x > m[nr][h]);
          }
        if (__any_sync(~0u, raise)) {
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            float f[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float m2 = fmaxf(m[nr][h], top[nr][h]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) m2 = fmaxf(m2, __shfl_xor_sync(~0u, m2, d));
              f[h] = m2 == m[nr][h] ? 1.f : pr_exp2(m[nr][h] - m2);
              m[nr][h] = m2;
              l[nr][h] *= f[h];
            }
#pragma unroll
            for (int n = 0; n < KS; ++n)
              o[nr][n][0] *= f[0], o[nr][n][1] *= f[1], o[nr][n][2] *= f[0], o[nr][n][3] *= f[1];
          }
        }
        uint32_t pw[NR][SUB][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          float mm[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) mm[h] = m[nr][h] == -INFINITY ? 0.f : m[nr][h];
#pragma unroll
          for (int e = 0; e < 4 * SUB; e += 2) {
            const float w0 = pr_exp2(fmaf(s[nr][e >> 2][e & 3], scale[nr][0], -mm[0]));
            const float w1 = pr_exp2(fmaf(s[nr][e >> 2][(e & 3) + 1], scale[nr][1], -mm[1]));
            l[nr][0] += w0, l[nr][1] += w1;
            pw[nr][e >> 2][(e >> 1) & 1] = pr_transposed(as_u32(__floats2half2_rn(w0, w1)));
          }
        }
        // ---- values, 16 positions at a time
        auto values = [&](auto cleaning) {      // (code of its own for the few groups to be cleaned)
          const int vr = (lane & 7) + (lane & 8);
#pragma unroll
          for (int sub = 0; sub < SUB; ++sub) {
            __half2 d0[HD / 32], d1[HD / 32];       // Q8: scales of positions 2t, 2t + 1 and of 8 further on
            if (Q8) {
              const uint32_t sc = at + 2 * GP * ROW + G::SC + sub * 16 * (HD / 16);
#pragma unroll
              for (int b = 0; b < HD / 64; ++b) {   // two blocks' scales at a time
                uint32_t x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[i]) : "r"(sc + (2 * t + (i & 1) + (i >> 1) * 8) * (HD / 16) + b * 4) : "memory");
                uint32_t y;
                asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(y) : "r"(x[0]), "r"(x[1]));
                d0[2 * b] = as_h2(y);
                asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(y) : "r"(x[0]), "r"(x[1]));
                d0[2 * b + 1] = as_h2(y);
                asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(y) : "r"(x[2]), "r"(x[3]));
                d1[2 * b] = as_h2(y);
                asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(y) : "r"(x[2]), "r"(x[3]));
                d1[2 * b + 1] = as_h2(y);
              }
            }
#pragma unroll
            for (int i = 0; i < PIECES / 2; ++i) {
              uint32_t r[4];
              pr_ldsm_t(r, kByXor<ROW> ? (vat ^ (i << 5)) + sub * 16 * ROW : at + GP * ROW + place<ROW, false>(sub * 16 + vr, 2 * i + (lane >> 4)));
              if (!Q8) {
                if (decltype(cleaning)::value) {
#pragma unroll
                  for (int e = 0; e < 4; ++e) r[e] = pr_finite(r[e], &found);
                }
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) pr_mma(o[nr][i], r[0], r[2], r[1], r[3], pw[nr][sub][0], pw[nr][sub][1]);
              } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {       // two pieces; of each the 16 codes' even columns, then the odd ones
                  const int pc = 2 * i + k;
                  const uint32_t x0 = r[2 * k] ^ 0x80808080u, x1 = r[2 * k + 1] ^ 0x80808080u;
                  uint32_t v[4] = {as_u32(__hmul2(q8_pair(x0, 0x4240u), d0[pc / 2])), as_u32(__hmul2(q8_pair(x0, 0x4341u), d0[pc / 2])),
                                   as_u32(__hmul2(q8_pair(x1, 0x4240u), d1[pc / 2])), as_u32(__hmul2(q8_pair(x1, 0x4341u), d1[pc / 2]))};
                  if (decltype(cleaning)::value) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = pr_finite(v[e], &found);
                  }
#pragma unroll
                  for (int nr = 0; nr < NR; ++nr) pr_mma(o[nr][pc], v[0], v[1], v[2], v[3], pw[nr][sub][0], pw[nr][sub][1]);
                }
              }
            }
          }
        };
        if (whole)
          values(std::false_type{});
        else
          values(std::true_type{});
      }
      __syncwarp();            // the stage may be written again
    }
    if (found) *reinterpret_cast<volatile int*>(&c->bad) = seg + 1;
    if (CL) __syncthreads();   // (the results take the ring's place)
    // ---- the warps' results meet, RM rows at a time
    const bool whole_item = w.i0 == 0 && w.i1 == w.it.cnt;
    const int slot = w.i0 == 0 ? 1 : 0;
#pragma unroll
    for (int r8 = 0; r8 < NR; r8 += G::RM / 8) {
      float* mine = s_o + warp * G::RM * G::PITCH;
#pragma unroll
      for (int i = 0; i < G::RM / 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int nr = r8 + i;
          if (nr >= NR) break;
          const int rr = (nr - r8) * 8 + 2 * t + h;
          float sum = l[nr][h];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
          if (g == 0) s_m[warp * R + r8 * 8 + rr] = m[nr][h], s_l[warp * R + r8 * 8 + rr] = sum;
#pragma unroll
          for (int n = 0; n < KS; ++n) {
            float* to = mine + rr * G::PITCH + n * 16;
            if (Q8)
              *reinterpret_cast<float2*>(to + 2 * g) = make_float2(o[nr][n][h], o[nr][n][2 + h]);
            else
              to[g] = o[nr][n][h], to[8 + g] = o[nr][n][2 + h];
          }
        }
      __syncthreads();
      const bool bad = c->bad == seg + 1;
      const int n_rows = min(G::RM, rows - r8 * 8);
      for (int x = tid; x < n_rows * (HD / 4); x += G::NT) {
        const int rr = x / (HD / 4), e = x % (HD / 4) * 4, r = row0 + r8 * 8 + rr;
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < W; ++k) top = fmaxf(top, s_m[k * R + r8 * 8 + rr]);
        float sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const float mk = s_m[k * R + r8 * 8 + rr], f = mk == -INFINITY ? 0.f : pr_exp2(mk - top);
          const float4 y = *reinterpret_cast<const float4*>(s_o + (k * G::RM + rr) * G::PITCH + e);
          sum += s_l[k * R + r8 * 8 + rr] * f;
          v[0] += y.x * f, v[1] += y.y * f, v[2] += y.z * f, v[3] += y.w * f;
        }
        if (bad) {
          // values that were taken out of groups seen in part: back into the rows that see them
          const int pr = first + a.token_of(r);
          for (int i = w.i0; i < w.i1; ++i)
            for (int b = 0; b < 32; b += 16) {
              const int base = w.it.tile(i) * 32 + b, from_g = base & ~(GP - 1);
              // (the values that were looked at are those of groups not seen whole; a hole makes a group one)
              if (from_g + GP - 1 <= w.it.p0 && (!a.window || from_g > w.it.p1 - a.window || from_g + GP <= a.sinks) &&
                  paged_row(a.kv, a.b, w.seq, from_g, w.head) >= 0 && paged_row(a.kv, a.b, w.seq, from_g + GP - 16, w.head) >= 0)
                continue;
              for (int q = base; q < base + 16 && q <= pr; ++q) {
                if (a.window && q <= pr - a.window && q >= a.sinks) continue;
                const int vrow = paged_row(a.kv, a.b, w.seq, q, w.head);
                if (vrow < 0) continue;
                for (int k = 0; k < 4; ++k) {
                  const size_t from = static_cast<size_t>(vrow) * HD + e + k;
                  const __half h = Q8 ? __hmul(__int2half_rn(static_cast<const int8_t*>(a.kv.v)[from]), a.kv.vs[from / 32])
                                      : static_cast<const __half*>(a.kv.v)[from];
                  if (__hisinf(h) || __hisnan(h)) v[k] += __half2float(h);
                }
              }
            }
        }
        if (CL) {
          *reinterpret_cast<float4*>(s_joined + (r8 * 8 + rr) * HD + e) = make_float4(v[0], v[1], v[2], v[3]);
          if (e == 0) s_joined[R * HD + r8 * 8 + rr] = top, s_joined[R * (HD + 1) + r8 * 8 + rr] = sum;
        } else if (whole_item) {
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          __half* out = a.out + a.row_at(w.sp.t0, w.head, r, a.out_ld) + e;
          const uint2 y = make_uint2(as_u32(__floats2half2_rn(v[0] * inv, v[1] * inv)), as_u32(__floats2half2_rn(v[2] * inv, v[3] * inv)));
          *reinterpret_cast<uint2*>(out) = y;
        } else {
          *reinterpret_cast<float4*>(parts.out(blockIdx.x, slot) + static_cast<size_t>(r8 * 8 + rr) * HD + e) =
              make_float4(v[0], v[1], v[2], v[3]);
          if (e == 0) {
            parts.max(blockIdx.x, slot)[r8 * 8 + rr] = top;
            parts.sum(blockIdx.x, slot)[r8 * 8 + rr] = sum;
          }
        }
      }
      if (r8 + G::RM / 8 < NR) __syncthreads();        // the next item's queries are waited for anyway
    }
    if constexpr (CL) {
      // ---- the cluster's results meet: every CTA finishes its share of the outputs
      cluster_sync();
      const uint32_t own = smem_u32(s_joined);
      for (int x = tid + w.rank * G::NT; x < rows * (HD / 4); x += G::NT * kPrCluster) {
        const int rr = x / (HD / 4), e = x % (HD / 4) * 4;
        float m8[kPrCluster], l8[kPrCluster];
        float4 y[kPrCluster];
#pragma unroll
        for (int k = 0; k < kPrCluster; ++k) {
          const uint32_t at = cluster_at(own, k);
          m8[k] = cluster_ld(at + (R * HD + rr) * 4);
          l8[k] = cluster_ld(at + (R * (HD + 1) + rr) * 4);
          y[k] = cluster_ld4(at + (rr * HD + e) * 4);
        }
        float top = m8[0], sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 1; k < kPrCluster; ++k) top = fmaxf(top, m8[k]);
#pragma unroll
        for (int k = 0; k < kPrCluster; ++k) {
          const float f = m8[k] == -INFINITY ? 0.f : pr_exp2(m8[k] - top);
          sum += l8[k] * f;
          v[0] += y[k].x * f, v[1] += y[k].y * f, v[2] += y[k].z * f, v[3] += y[k].w * f;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        __half* out = a.out + a.row_at(w.sp.t0, w.head, row0 + rr, a.out_ld) + e;
        *reinterpret_cast<uint2*>(out) = make_uint2(as_u32(__floats2half2_rn(v[0] * inv, v[1] * inv)),
                                                    as_u32(__floats2half2_rn(v[2] * inv, v[3] * inv)));
      }
      cluster_sync();          // read by all before it is written again, or its CTA ends
    }
  }
  if (!CL && tid == 0) *parts.record(blockIdx.x) = rec;
}

template <int HD, int NR, bool QF32, bool Q8>
cudaError_t prepare_rows() {
  const cudaError_t e = cudaFuncSetAttribute(paged_rows_kernel<HD, NR, QF32, Q8, false>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Pr<HD, NR, QF32, Q8, false>::SMEM);
  if constexpr (NR <= 2) {
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(paged_rows_kernel<HD, NR, QF32, Q8, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Pr<HD, NR, QF32, Q8, true>::SMEM);
  }
  return e;
}

template <int HD, int NR>
cudaError_t prepare_nr() {
  const cudaError_t e[4] = {prepare_rows<HD, NR, false, false>(), prepare_rows<HD, NR, false, true>(),
                            prepare_rows<HD, NR, true, false>(), prepare_rows<HD, NR, true, true>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

template <int HD, int NR, bool QF32, bool Q8>
cudaError_t launch_rows(const PagedAttnArgs& a, void* ws, int grid, cudaStream_t s) {
  if constexpr (NR <= 2) {
    // Few items and a table of no great length: a cluster each.  One token of the 8B heads over 512, 2048, 4096, 8192
    // and 32768 positions 4.7, 6.1, 7.8, 11.9 and 30.0 us, split evenly over all CTAs 8.3, 8.9, 11.9, 16.7 and 31.1
    // (64 CTAs draw less of the bandwidth than 152, so longer tables are split).  16 items are more clusters than the
    // GPU holds at once (a CTA fills an SM): 16.9 against 15.6 for 2 sequences of 4096 positions.
    const int items = a.b.n_seqs * a.kv.n_kv;
    if (items * kPrCluster * 2 <= grid && (a.b.width << a.kv.page_log2) <= 32768) {
      using G = Pr<HD, NR, QF32, Q8, true>;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(items * kPrCluster);
      cfg.blockDim = dim3(G::NT);
      cfg.dynamicSmemBytes = G::SMEM;
      cfg.stream = s;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = kPrCluster, at[0].val.clusterDim.y = 1, at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      return cudaLaunchKernelEx(&cfg, paged_rows_kernel<HD, NR, QF32, Q8, true>, a, PartSlots{});
    }
  }
  using G = Pr<HD, NR, QF32, Q8, false>;
  PartSlots parts{static_cast<char*>(ws), G::R, HD};
  paged_rows_kernel<HD, NR, QF32, Q8, false><<<grid, G::NT, G::SMEM, s>>>(a, parts);
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : paged_join_launch(a, parts, grid, s);
}

template <int HD, int NR>
cudaError_t launch_nr(const PagedAttnArgs& a, bool f32, bool q8, void* ws, int grid, cudaStream_t s) {
  if (f32) return q8 ? launch_rows<HD, NR, true, true>(a, ws, grid, s) : launch_rows<HD, NR, true, false>(a, ws, grid, s);
  return q8 ? launch_rows<HD, NR, false, true>(a, ws, grid, s) : launch_rows<HD, NR, false, false>(a, ws, grid, s);
}

// As many rows at once as the item has; above head_dim 128, whose outputs fill the registers, at most 16.
template <int HD>
cudaError_t launch_hd(const PagedAttnArgs& a, bool f32, bool q8, int rows, void* ws, int grid, cudaStream_t s) {
  if (rows <= 8) return launch_nr<HD, 1>(a, f32, q8, ws, grid, s);
  if constexpr (HD <= 128) {
    if (rows > 24) return launch_nr<HD, 4>(a, f32, q8, ws, grid, s);
    if (rows > 16) return launch_nr<HD, 3>(a, f32, q8, ws, grid, s);
  }
  return launch_nr<HD, 2>(a, f32, q8, ws, grid, s);
}

}  // namespace

cudaError_t paged_rows_prepare() {
  const cudaError_t e[12] = {prepare_nr<64, 1>(),  prepare_nr<64, 2>(),  prepare_nr<64, 3>(),  prepare_nr<64, 4>(),
                             prepare_nr<128, 1>(), prepare_nr<128, 2>(), prepare_nr<128, 3>(), prepare_nr<128, 4>(),
                             prepare_nr<192, 1>(), prepare_nr<192, 2>(), prepare_nr<256, 1>(), prepare_nr<256, 2>()};
  for (cudaError_t x : e)
    if (x != cudaSuccess) return x;
  return cudaSuccess;
}

cudaError_t paged_rows_launch(const PagedAttnArgs& a, bool q_f32, bool q8, int rows, void* ws, int grid, cudaStream_t s) {
  switch (a.kv.hd) {
    case 64: return launch_hd<64>(a, q_f32, q8, rows, ws, grid, s);
    case 128: return launch_hd<128>(a, q_f32, q8, rows, ws, grid, s);
    case 192: return launch_hd<192>(a, q_f32, q8, rows, ws, grid, s);
    default: return launch_hd<256>(a, q_f32, q8, rows, ws, grid, s);
  }
}

}  // namespace q4
