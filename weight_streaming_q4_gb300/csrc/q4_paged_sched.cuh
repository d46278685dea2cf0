// How the attention over pages is split over the CTAs, on the device (sm_103a).
//
// An item is one tile of R query rows of one value head of one sequence: row r
// of a head is query head r % group of new token r / group, so that the group's
// queries share each key and value that is read.  An item walks the key tiles
// (BN positions each) that its rows see: the sinks' tiles, then the tiles from
// the first row's window to the last row's position.  All items' key tiles in
// a row (sequence, row tile, head, key tile) are the units; every CTA takes the
// same number of consecutive units, whatever the lengths, so a long sequence
// spreads over many CTAs and short ones share one.  An item that a CTA does not
// hold whole leaves partial results (maximum, sum, unnormalised output per row):
//   slot 0 of a CTA: its first item, begun by an earlier CTA
//   slot 1 of a CTA: its last item, begun there and not finished
// so an item begun by CTA c is slot 1 of c, then slot 0 of c + 1, ...: joined in
// that order by a second kernel, whose result depends on the lengths alone.
// Everything is computed from the arrays in device memory by every CTA for
// itself (one scan over the sequences, about a microsecond), so a captured
// graph serves any content of them and there is no plan to keep.
#pragma once

#include <stdint.h>

#include "q4_paged.cuh"

namespace q4 {

constexpr int kPagedMaxCtas = 160;      // CTAs a workspace has slots for

// The key tiles of one item.
struct ItemTiles {
  int p0, p1;       // positions of its first and last row (p1 < 0: the rows see nothing)
  int n_sink;       // tiles 0 .. n_sink - 1 come first
  int lo;           // then tiles lo ..
  int cnt;          // tiles in all, at least 1 (an item without work still writes its zeros)
  __device__ __forceinline__ int tile(int i) const { return i < n_sink ? i : lo + i - n_sink; }
};

template <int R, int BN>
__device__ __forceinline__ ItemTiles item_tiles(const PagedAttnArgs& a, const SeqSpan& sp, int j) {
  ItemTiles t;
  const int rows = sp.n_new * a.group;
  const int first = sp.len - sp.n_new;
  t.p0 = first + a.token_of(j * R);
  t.p1 = first + a.token_of(min(rows, j * R + R) - 1);
  t.n_sink = 0, t.lo = 0, t.cnt = 1;
  if (t.p1 < 0) return t;
  const int seen = a.window ? max(0, t.p0 - a.window + 1) : 0;     // first position inside the first row's window
  t.lo = seen / BN;
  t.n_sink = min((a.sinks + BN - 1) / BN, t.lo);
  t.cnt = t.n_sink + t.p1 / BN - t.lo + 1;
  return t;
}

// Units of the sequence of every lane (n_new 0: none), by the whole warp: a lane
// adds up a few row tiles for itself, the rest of a long chunk is shared by all
// (one lane alone took 26 us over the 382 row tiles of two chunks).
constexpr int kLaneTiles = 4;
template <int R, int BN>
__device__ __forceinline__ long long seq_units(const PagedAttnArgs& a, const SeqSpan& sp, int* most = nullptr) {
  const int lane = threadIdx.x & 31;
  const int n = (sp.n_new * a.group + R - 1) / R;
  long long sum = 0;
  for (int j = 0; j < min(n, kLaneTiles); ++j) {
    const int cnt = item_tiles<R, BN>(a, sp, j).cnt;
    if (most) *most = max(*most, cnt);
    sum += cnt;
  }
  for (unsigned more = __ballot_sync(~0u, n > kLaneTiles); more; more &= more - 1) {
    const int who = __ffs(more) - 1;
    const SeqSpan s = {__shfl_sync(~0u, sp.t0, who), __shfl_sync(~0u, sp.n_new, who), __shfl_sync(~0u, sp.len, who)};
    const int ns = __shfl_sync(~0u, n, who);
    long long part = 0;
    for (int j = kLaneTiles + lane; j < ns; j += 32) part += item_tiles<R, BN>(a, s, j).cnt;
#pragma unroll
    for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(~0u, part, d);
    if (lane == who) sum += part;
  }
  return sum * a.kv.n_kv;
}

// The item and tile of unit u (per value head: all of a row tile's heads follow
// one another) of a sequence, by the whole warp, the same in every lane.
template <int R, int BN>
__device__ __forceinline__ void find_unit(const PagedAttnArgs& a, const SeqSpan& sp, long long u, int* j, int* head, int* tile) {
  const int lane = threadIdx.x & 31;
  const int n = (sp.n_new * a.group + R - 1) / R;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int cnt = j0 + lane < n ? item_tiles<R, BN>(a, sp, j0 + lane).cnt : 0;
    const long long mine = static_cast<long long>(cnt) * a.kv.n_kv;
    long long end = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(~0u, end, d);
      if (lane >= d) end += o;
    }
    const unsigned at = __ballot_sync(~0u, u < end);
    if (at) {
      const int who = __ffs(at) - 1;
      const unsigned x = static_cast<unsigned>(u - __shfl_sync(~0u, end - mine, who)), c = __shfl_sync(~0u, cnt, who);
      *j = j0 + who, *head = static_cast<int>(x / c), *tile = static_cast<int>(x % c);
      return;
    }
    u -= __shfl_sync(~0u, end, 31);
  }
}

// Where a CTA starts and how many units it takes.
struct CtaWork {
  long long per;            // units of every CTA but the last ones
  int n;                    // units of this CTA (0: none)
  int seq, j, head, tile;   // its first unit
};

// (64-bit divisions are slow, and that many units are days of work)
__device__ __forceinline__ long long units_per_cta(long long total) {
  return total < 0x7fffffff ? (static_cast<unsigned>(total) + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
}

// One scan over the sequences by the whole block of NT threads (a multiple of
// 32); s_scan holds NT / 32 + 1 values.  Ends with the result in *out (shared
// memory) and the block synchronised.
template <int R, int BN, int NT>
__device__ void cta_work(const PagedAttnArgs& a, long long* s_scan, CtaWork* out) {
  constexpr int W = NT / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // inclusive scan of v over the block; *total its sum
  auto scan = [&](long long v, long long* total) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(~0u, v, d);
      if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const long long x = s_scan[w];
      before += w < warp ? x : 0;
      all += x;
    }
    *total = all;
    return v + before;
  };
  const int n_seqs = a.b.n_seqs;
  auto span = [&](int s) { return s < n_seqs ? paged_span(a.kv, a.b, s) : SeqSpan{0, 0, 0}; };
  long long total = 0, mine = 0;
  for (int base = 0; base < n_seqs; base += NT) mine += seq_units<R, BN>(a, span(base + tid));
  scan(mine, &total);
  const long long per = units_per_cta(total);
  const long long u0 = per * blockIdx.x;
  if (tid == 0) out->per = per, out->n = u0 < total ? static_cast<int>(min(per, total - u0)) : 0;
  long long carry = 0;
  for (int base = 0; base < n_seqs && carry <= u0 && u0 < total; base += NT) {
    const SeqSpan sp = span(base + tid);
    mine = seq_units<R, BN>(a, sp);
    long long sum;
    const long long end = carry + scan(mine, &sum);
    carry += sum;
    // the warp whose sequences hold u0 finds the unit
    const unsigned here = __ballot_sync(~0u, mine > 0 && u0 >= end - mine && u0 < end);
    if (here) {
      const int who = __ffs(here) - 1;
      const SeqSpan s = {__shfl_sync(~0u, sp.t0, who), __shfl_sync(~0u, sp.n_new, who), __shfl_sync(~0u, sp.len, who)};
      int j = 0, head = 0, tile = 0;
      find_unit<R, BN>(a, s, u0 - __shfl_sync(~0u, end - mine, who), &j, &head, &tile);
      if (lane == 0) out->seq = base + (tid & ~31) + who, out->j = j, out->head = head, out->tile = tile;
    }
  }
  __syncthreads();
}

// cta_work for at most 32 sequences, by every warp for itself: a sequence per
// lane, no barrier and no shared memory.
template <int R, int BN>
__device__ __forceinline__ CtaWork warp_work(const PagedAttnArgs& a) {
  const int lane = threadIdx.x & 31;
  SeqSpan sp = {};
  if (lane < a.b.n_seqs) sp = paged_span(a.kv, a.b, lane);
  int most = 0;                    // key tiles of the longest item, if every sequence has few
  const long long mine = seq_units<R, BN>(a, sp, &most);
  const int tiles = (sp.n_new * a.group + R - 1) / R;
  long long end = mine;
  int tiles_end = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(~0u, end, d);
    const int t = __shfl_up_sync(~0u, tiles_end, d);
    if (lane >= d) end += o, tiles_end += t;
  }
  const long long total = __shfl_sync(~0u, end, 31);
  CtaWork w = {};
  w.per = units_per_cta(total);
  // With no more items than CTAs and none much longer than an even share, an item each: nothing to join, and
  // one start and end per CTA instead of two.  16 sequences under a window, 33 tiles an item where an even share is
  // 28: 12.0 us against 15.8; 16 sequences of 1000 positions, 32 and 27: 16.1 against 18.4; 10 of 4000, 125 and 66,
  // are split: an item each takes 34.2 against 32.2.
  const int items = __shfl_sync(~0u, tiles_end, 31) * a.kv.n_kv;
  most = __reduce_max_sync(~0u, tiles > kLaneTiles ? 0x3fffffff : most);
  if (items <= static_cast<int>(gridDim.x) && items > 0 && most <= w.per + w.per / 2) {
    const int item = blockIdx.x;
    if (item < items) {
      w.seq = __ffs(__ballot_sync(~0u, item < tiles_end * a.kv.n_kv)) - 1;
      const int x = item - __shfl_sync(~0u, (tiles_end - tiles) * a.kv.n_kv, w.seq);
      w.j = x / a.kv.n_kv, w.head = x - w.j * a.kv.n_kv;
      const SeqSpan s = {__shfl_sync(~0u, sp.t0, w.seq), __shfl_sync(~0u, sp.n_new, w.seq), __shfl_sync(~0u, sp.len, w.seq)};
      w.n = item_tiles<R, BN>(a, s, w.j).cnt;
    }
    return w;
  }
  const long long u0 = w.per * blockIdx.x;
  w.n = u0 < total ? static_cast<int>(min(w.per, total - u0)) : 0;
  const unsigned here = __ballot_sync(~0u, mine > 0 && u0 >= end - mine && u0 < end);
  if (here) {
    w.seq = __ffs(here) - 1;
    const SeqSpan s = {__shfl_sync(~0u, sp.t0, w.seq), __shfl_sync(~0u, sp.n_new, w.seq), __shfl_sync(~0u, sp.len, w.seq)};
    find_unit<R, BN>(a, s, u0 - __shfl_sync(~0u, end - mine, w.seq), &w.j, &w.head, &w.tile);
  }
  return w;
}

// A CTA's units as segments: the tiles of one item that it holds.  Every role
// of the kernel walks its own copy.
template <int R, int BN>
struct SegmentWalk {
  int group;
  int left;                 // units not yet walked
  int seq, j, head;         // current item
  SeqSpan sp;
  ItemTiles it;
  int i0, i1;               // its tiles [i0, i1) in this segment

  __device__ __forceinline__ void begin(const PagedAttnArgs& a, const CtaWork& w) {
    group = a.group, left = w.n, seq = w.seq, j = w.j, head = w.head, i0 = w.tile;
    if (left > 0) {
      sp = paged_span(a.kv, a.b, seq);
      it = item_tiles<R, BN>(a, sp, j);
      i1 = min(it.cnt, i0 + left);
    }
  }
  __device__ __forceinline__ bool live() const { return left > 0; }
  __device__ __forceinline__ void next(const PagedAttnArgs& a) {
    left -= i1 - i0;
    if (left <= 0) return;
    i0 = 0;
    if (++head == a.kv.n_kv) {
      head = 0, ++j;
      while (j * R >= sp.n_new * group) {       // the next sequence with rows: there is one, units are left
        if (++seq >= a.b.n_seqs) {
          left = 0;
          return;
        }
        j = 0;
        sp = paged_span(a.kv, a.b, seq);
      }
      it = item_tiles<R, BN>(a, sp, j);
    }
    i1 = min(it.cnt, left);
  }
  __device__ __forceinline__ int rows() const { return min(R, sp.n_new * group - j * R); }
};

// For few items (at most 32 sequences): C CTAs of a cluster share every item,
// rank r the r-th part of its tiles, and join their results over distributed
// shared memory; no second kernel and no workspace.
template <int R, int BN>
struct ClusterWalk {
  int group;
  int item, items, step, rank, ranks;      // the cluster's current item; all items; clusters
  int seq, j, head;
  SeqSpan sp;
  ItemTiles it;
  int i0, i1;
  SeqSpan mine;                             // this lane's sequence
  int end, count;                           // ... its last item + 1, and how many

  __device__ __forceinline__ void begin(const PagedAttnArgs& a, int cluster, int clusters, int r, int n) {
    const int lane = threadIdx.x & 31;
    group = a.group, item = cluster, step = clusters, rank = r, ranks = n;
    mine = {};
    count = 0;
    if (lane < a.b.n_seqs) {
      mine = paged_span(a.kv, a.b, lane);
      count = (mine.n_new * group + R - 1) / R * a.kv.n_kv;
    }
    end = count;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(~0u, end, d);
      if (lane >= d) end += o;
    }
    items = __shfl_sync(~0u, end, 31);
    find(a);
  }
  __device__ __forceinline__ void find(const PagedAttnArgs& a) {
    if (item >= items) return;
    seq = __ffs(__ballot_sync(~0u, item < end && item >= end - count)) - 1;
    const int x = item - __shfl_sync(~0u, end - count, seq);
    j = x / a.kv.n_kv, head = x - j * a.kv.n_kv;
    sp.t0 = __shfl_sync(~0u, mine.t0, seq), sp.n_new = __shfl_sync(~0u, mine.n_new, seq);
    sp.len = __shfl_sync(~0u, mine.len, seq);
    it = item_tiles<R, BN>(a, sp, j);
    const int per = (it.cnt + ranks - 1) / ranks;
    i0 = min(it.cnt, rank * per), i1 = min(it.cnt, i0 + per);
  }
  __device__ __forceinline__ bool live() const { return item < items; }
  __device__ __forceinline__ void next(const PagedAttnArgs& a) {
    item += step;
    find(a);
  }
  __device__ __forceinline__ int rows() const { return min(R, sp.n_new * group - j * R); }
};

// Workspace: a record per CTA, then the partial results of its two slots.
struct JoinRecord {
  int n;                    // CTAs that hold a part of the item that slot 1 begins (0: none)
  int t0, row0, rows;       // the sequence's first token row; the item's first row and its rows
  int head;
};
constexpr size_t kPagedRecordBytes = kPagedMaxCtas * 32;
static_assert(sizeof(JoinRecord) <= 32, "records are 32 bytes apart");

// Notes in *rec the segment g if it begins an item that its CTA does not finish
// (per: units of every CTA).
template <int R, int BN>
__device__ __forceinline__ void join_note(JoinRecord* rec, const SegmentWalk<R, BN>& g, long long per) {
  if (g.i0 != 0 || g.i1 == g.it.cnt) return;
  rec->n = 1 + (g.it.cnt - g.i1 + static_cast<int>(per) - 1) / static_cast<int>(per);
  rec->t0 = g.sp.t0, rec->row0 = g.j * R, rec->rows = g.rows(), rec->head = g.head;
}

struct PartSlots {
  char* base;
  int rows, hd;             // R and head_dim
  __host__ __device__ __forceinline__ size_t slot_floats() const { return static_cast<size_t>(rows) * (hd + 2); }
  __device__ __forceinline__ JoinRecord* record(int cta) const { return reinterpret_cast<JoinRecord*>(base + cta * 32); }
  // [rows][hd] outputs, then [rows] maxima, then [rows] sums
  __device__ __forceinline__ float* out(int cta, int slot) const {
    return reinterpret_cast<float*>(base + kPagedRecordBytes) + (2 * cta + slot) * slot_floats();
  }
  __device__ __forceinline__ float* max(int cta, int slot) const { return out(cta, slot) + static_cast<size_t>(rows) * hd; }
  __device__ __forceinline__ float* sum(int cta, int slot) const { return max(cta, slot) + rows; }
};

// Launchers.  ws: the workspace; grid: CTAs, at most kPagedMaxCtas.
cudaError_t paged_tile_prepare();
cudaError_t paged_tile_launch(const PagedAttnArgs& a, bool q_f32, bool q8, void* ws, int grid, cudaStream_t s);
// For items of few rows: `rows` query rows of a head at most, as far as is known.
cudaError_t paged_rows_prepare();
cudaError_t paged_rows_launch(const PagedAttnArgs& a, bool q_f32, bool q8, int rows, void* ws, int grid, cudaStream_t s);
// Joins the parts that a kernel of `grid` CTAs left (q4_paged_join.cu).
cudaError_t paged_join_launch(const PagedAttnArgs& a, const PartSlots& parts, int grid, cudaStream_t s);

}  // namespace q4
