// Shared by the kernels of fa_decode (fa_decode.cu, bf16, and
// fa_decode_fp32.cu): how the work is shared out, and the joining of parts.
//
// Work.  An item is one sequence and one key-value head; a tile is kTile rows of
// an item.  All tiles of all items in order are
// cut into runs, one for each block.  A block finds its run from the lengths
// itself: the host knows none of them.  A run may end inside an item.  What a
// block has then goes to the workspace as (m, l, o), at most two such parts a
// run: one of an item that began in an earlier run and one of an item that
// goes on in the next one.  decode_join_kernel adds the parts of an item up, in
// the order of the runs: no atomics, the same sums each time.
//
// Query heads.  Up to 16 (8 in fp32) share one reading of the cache.  Larger
// groups are cut evenly, and as many blocks take each run, side by side, so
// that all but the first find its rows in L2.
//
// Small tables.  Where no item can have more than kClusterTiles tiles for each
// of a cluster's blocks, and a cluster an item fills no more than the GPU, each
// item is read by a cluster, whose blocks join their parts through one
// another's shared memory: no second kernel, no search for the run, no
// workspace.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "fa_paged.cuh"
#include "sm103_ptx.cuh"

namespace fa {
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxRuns = 1280;
constexpr int kMostBlocks = 16;  // of a cluster
constexpr int kMostHeads = 512;  // query heads that share a key-value head
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  const char *Q, *K, *V;
  char* O;
  float* L;
  const int32_t *table, *lengths;
  int32_t* status;
  float2* part_ml;    // [2 runs][split][heads of a piece, rounded up]
  float* part_o;      // the same, [d]
  FastDiv page_rows;
  int S, H, group;    // group: query heads that share a key-value head
  int split;          // blocks that take a run: pieces a group of query heads is cut into
  int piece_heads;    // query heads of a piece (the last of a group may have fewer)
  int items;          // of a sequence: H_kv
  int num_pages, max_pages;
  int cap;            // page_rows * max_pages
  int resident;       // blocks that run at a time
  int cluster;        // blocks an item, if each item has a cluster; else 0
  int64_t table_stride;
  int64_t qs, qh, os, oh;  // byte strides
  int64_t pp, ph, pn;
  float scale2;       // scale * log2(e)
};

// Of a cache in 8 bits.
struct E4m3Params : DecodeParams {
  const float *KS, *VS;
  FastDiv block_rows;
  int blocks;           // of a page and head
  int64_t page_scales;  // scales of a page
  uint64_t wait_ns;
};

// Blocks an SM holds of the kernel for that type and head dim: what its ring of
// tiles in shared memory (228 KB an SM) leaves room for.
constexpr int blocks_an_sm(bool bf16, int d) {
  return bf16 ? (d == 32 ? 4 : d == 64 ? 3 : d == 256 ? 1 : 2) : (d == 16 ? 4 : d == 32 ? 3 : d == 64 ? 2 : 1);
}

// ------------------------------------------------------------- sharing out
__device__ __forceinline__ int rows_of(const DecodeParams& a, int s) {
  const int n = a.lengths[s];
  if (n < 0 || n > a.cap) report_pages(a.status);
  return min(max(n, 0), a.cap);
}

template <int kTile>
__device__ __forceinline__ int tiles_of(int rows) {
  return rows <= kTile ? 1 : (rows + kTile - 1) / kTile;  // an empty item still writes its zeros
}

// What beginning and ending an item costs, in tiles: an item of n tiles is
// kItemCost + n units of work, and the runs are of equal units.  A run that
// begins inside the first kItemCost units of an item begins with its first
// tile.  So a run may be empty only between two items, never inside one.  1 is
// what measured best for rows as they are (those in 8 bits have a kCost of their own): 32 sequences of up to 2048 rows, 32 heads of d 64 (items
// of up to 32 tiles) took 56.5 us with 0, 46.3 with 1, 46.5 with 2, 47.4 with 3.
constexpr int kItemCost = 1;

// The runs.  SMs do not get equal shares of the memory's bandwidth: with equal
// runs the first was done after 74 % of the time, on average they were after
// 88 % (32 sequences of 8192 rows, 8 heads of d 128).  So where there is enough
// to do, the blocks that are resident from the start get kBigShare of the
// units, and the rest is cut into kSmallRuns times as many small runs, for
// blocks that the hardware starts where one has ended.  Who takes which changes
// from call to call, where the runs end does not.  64 sequences of up to 8192
// rows (100 units a resident block) took 164.1 us with equal runs, 158.7 with
// these, 157.9 to 159.7 with two or three times as many small ones; 32 of up to
// 2048 (33 units) took 44.9 and, with small runs, 47 to 50: a block's start
// costs as much as two tiles.  Hence kMinUnits.  With 24 instead, on one
// GPU: 82.4 -> 78.3 us (64 sequences of up to 4608 rows, 8 key heads of d 128: 48 units a
// resident block), 75.5 -> 73.9 (of up to 3584: 45), 92.9 -> 90.5 (4 of 8192, 16 heads of
// d 256: 54), 106.6 -> 103.2 (16 of up to 4000: 64), 54.6 -> 49.7 (16 of up to 2048: 28), but
// 43.4 -> 44.2 (64 of up to 2048, d 128: 24) and 50.5 -> 51.0 (32 of 1024, 32 heads of d 64: 38,
// items of 16 tiles): a lower border would suit long items, and 64 is on the safe side.
constexpr double kBigShare = 0.9;
constexpr int kSmallRuns = 1;
constexpr int kMinUnits = 64;  // of a resident block, for there to be small runs

// x / n, as one of 32 bits where that does (a division of 64 bits takes several
// times as long, and stands in front of all loads).
__device__ __forceinline__ int64_t divide(int64_t x, int64_t n) {
  return (uint64_t)(x | n) >> 32 ? x / n : (int64_t)((uint32_t)x / (uint32_t)n);
}

// `units` units in `runs` runs as equal as can be: the first `longer` of them
// have one more than `each`.
struct Cuts {
  int64_t units, each;
  int runs, longer;
  __device__ __forceinline__ Cuts(int64_t u, int r) : units(u), each(r > 0 ? divide(u, r) : 0), runs(r) {
    longer = (int)(u - each * r);
  }
  __device__ __forceinline__ int64_t first(int w) const { return each * w + min(w, longer); }
  // the run that holds unit x
  __device__ __forceinline__ int run_of(int64_t x) const {
    const int64_t in_longer = (each + 1) * longer;
    return x < in_longer ? (int)divide(x, each + 1) : longer + (int)divide(x - in_longer, each);
  }
};

struct Share {
  Cuts big, small;  // units of all items: in big and in small runs
  static __device__ __forceinline__ bool tail(int64_t total, int resident) {
    return total >= (int64_t)resident * kMinUnits;
  }
  static __device__ __forceinline__ int64_t of_big(int64_t total, int resident) {
    return tail(total, resident) ? total - (int64_t)((float)total * (float)(1 - kBigShare)) : total;
  }
  __device__ __forceinline__ Share(int64_t total, int resident)
      : big(of_big(total, resident), (int)(total < resident ? total : resident)),
        small(total - big.units, tail(total, resident) ? resident * kSmallRuns : 0) {}
  __device__ __forceinline__ int runs() const { return big.runs + small.runs; }
  __device__ __forceinline__ int64_t first(int w) const {
    return w <= big.runs ? big.first(w) : big.units + small.first(w - big.runs);
  }
  // the run that holds unit x: the largest w with first(w) <= x
  __device__ __forceinline__ int run_of(int64_t x) const {
    return x < big.units ? big.run_of(x) : big.runs + small.run_of(x - big.units);
  }
};

// Sum over the threads before this one (return value) and over the block of NT
// threads; sums: NT / 32 entries of shared memory.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t n, int64_t* sums, int64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the last call's readers of sums are done
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  x -= n;
  *all = 0;
#pragma unroll
  for (int k = 0; k < NT / 32; ++k) {
    if (k < warp) x += sums[k];
    *all += sums[k];
  }
  return x;
}

// The sequences' units, summed over a block of NT threads.  Thread t looks at
// sequences t, t + NT, ...: up to NT of them are loaded and summed once, of more
// the sums are taken twice, for the total and for a place among them.
template <int kTile, int NT, int kCost>
struct Units {
  const DecodeParams& a;
  int64_t* sums;     // NT / 32 entries of shared memory
  int64_t n, lo, all;  // of the first NT sequences: this thread's, those before it, all
  __device__ __forceinline__ int64_t of(int s) const {
    return s < a.S ? (int64_t)(kCost + tiles_of<kTile>(rows_of(a, s))) * a.items : 0;
  }
  __device__ __forceinline__ Units(const DecodeParams& p, int64_t* shared) : a(p), sums(shared) { restart(); }
  // the first NT sequences once more: find() goes on from them
  __device__ __forceinline__ void restart() {
    n = of(threadIdx.x);
    lo = block_scan<NT>(n, sums, &all);
  }
  __device__ __forceinline__ Share share() {
    int64_t total = all;
    if (a.S > NT) {
      int64_t more = 0;
      for (int s = NT + threadIdx.x; s < a.S; s += NT) more += of(s);
      block_scan<NT>(more, sums, &more);
      total += more;
    }
    return Share(total, a.resident);
  }
  // The sequence that holds unit x (x < 0: sequence `want`), and its first unit.
  __device__ __forceinline__ int find(int64_t x, int want, int64_t* base) {
    __shared__ int64_t found_base;
    __shared__ int found;
    for (int at = 0;;) {
      const int s = at + threadIdx.x;
      if (x < 0 ? s == want : n > 0 && lo <= x && x < lo + n) {
        found_base = lo;
        found = s;
      }
      at += NT;
      if (x < 0 ? want < at : all > x) break;
      n = of(at + threadIdx.x);
      int64_t here;
      lo = all + block_scan<NT>(n, sums, &here);
      all += here;
    }
    __syncthreads();
    *base = found_base;
    return found;
  }
};

// A place in the row of tiles: tile t of item `item` of sequence s, which is
// unit `unit` of all.
template <int kTile, int kCost = kItemCost>
struct Place {
  int s, item, t, rows, tiles;
  int64_t unit;
  // the first tile at or behind unit x of sequence s, whose first unit is base
  __device__ __forceinline__ void set(const DecodeParams& a, int seq, int64_t base, int64_t x) {
    s = seq;
    rows = rows_of(a, s);
    tiles = tiles_of<kTile>(rows);
    item = (int)divide(x - base, kCost + tiles);
    const int64_t begin = base + (int64_t)item * (kCost + tiles);
    t = max((int)(x - begin) - kCost, 0);
    unit = begin + kCost + t;
  }
  __device__ __forceinline__ void next(const DecodeParams& a) {
    ++unit;
    if (++t < tiles) return;
    t = 0;
    unit += kCost;
    if (++item < a.items) return;
    item = 0;
    if (++s < a.S) {
      rows = rows_of(a, s);
      tiles = tiles_of<kTile>(rows);
    }
  }
};

// A way through a run, item by item.
template <int kTile, int kCost = kItemCost>
struct Walk {
  int s, item, t;       // the item's sequence and head, and its first tile that is the run's
  int rows, tiles;      // of the item
  int count;            // of its tiles, those that are the run's
  int rows_next;        // of the next sequence, asked for in time
  int64_t unit, end;    // of tile t; the run's
  __device__ __forceinline__ void begin(const DecodeParams& a, const Place<kTile, kCost>& at, int64_t e) {
    s = at.s, item = at.item, t = at.t, rows = at.rows, tiles = at.tiles, unit = at.unit, end = e;
    count = (int)min((int64_t)(tiles - t), end - unit);
    rows_next = s + 1 < a.S ? rows_of(a, s + 1) : 0;
  }
  __device__ __forceinline__ bool some() const { return unit < end; }
  // the next item; false if the run ends before it has a tile
  __device__ __forceinline__ bool next(const DecodeParams& a) {
    unit += tiles - t + kCost;
    t = 0;
    if (unit >= end) return false;
    if (++item == a.items) {
      item = 0;
      ++s;
      rows = rows_next;
      tiles = tiles_of<kTile>(rows);
      if (s + 1 < a.S) rows_next = rows_of(a, s + 1);
    }
    count = (int)min((int64_t)tiles, end - unit);
    return true;
  }
};

// The piece of an item's query heads that this block takes, the first of them,
// and how many.
__device__ __forceinline__ int first_head(const DecodeParams& a, int item, int piece, int* heads) {
  *heads = min(a.piece_heads, a.group - piece * a.piece_heads);
  return item * a.group + piece * a.piece_heads;
}

__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

template <class T>
__device__ __forceinline__ void store4(char* row, int col, float4 x) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(row + 4 * col) = x;
  else
    *reinterpret_cast<uint2*>(row + 2 * col) = make_uint2(ptx::pack_bf16x2(x.x, x.y), ptx::pack_bf16x2(x.z, x.w));
}

// ------------------------------------------------------- asynchronous copies
__device__ __forceinline__ void cp_async16(uint32_t dst, const char* src, bool on) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}
__device__ __forceinline__ void prefetch_l1(const char* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------ shared-memory reads
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds4(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t at, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(at));
}

// A warp's copies of its rows of each tile, ahead of their use: rows warp *
// kRows ... of the tile, K then V, kPieces pieces of 16 bytes each, kPitch
// bytes apart, in a ring of kStages in shared memory.
template <int kTile, int kRows, int kPieces, int kPitch, int kStages>
struct Loader {
  static constexpr int kStageBytes = 2 * kRows * kPitch;
  static_assert(kStages >= 3 && kStages <= 5, "the masks of kStages - 1 tiles share 64 bits");
  const DecodeParams& a;
  Place<kTile> at;      // the tile that is copied next
  const int64_t end;    // of the run
  const uint32_t ring;  // of this warp
  const int piece;      // of the query heads
  uint64_t queue = 0;   // which rows of the tiles in flight are there, the oldest in the low 16 bits
  // The row that this lane looks up in that tile: its page is asked for one
  // tile ahead of the copies that need it.
  int page = -1;
  bool in = false;
  int64_t off = 0;

  __device__ __forceinline__ Loader(const DecodeParams& p, const Place<kTile>& first, int64_t e, uint32_t r, int h)
      : a(p), at(first), end(e), ring(r), piece(h) {
    look_up();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) produce(i);
  }
  __device__ __forceinline__ void look_up() {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = at.t * kTile + warp * kRows + (lane & (kRows - 1));
    uint32_t r;
    const uint32_t col = a.page_rows.div((uint32_t)j, &r);
    in = j < at.rows;
    page = in ? a.table[at.s * a.table_stride + col] : -1;
    off = at.item * a.ph + (int64_t)r * a.pn;
    if (at.t == 0) {  // a new item: its queries into L1
      int heads;
      const char* row = a.Q + at.s * a.qs + (int64_t)first_head(a, at.item, piece, &heads) * a.qh;
      constexpr int kLines = (kPieces * 16 + 127) / 128;
      for (int k = lane; k < heads * kLines; k += 32) prefetch_l1(row + (k / kLines) * a.qh + (k % kLines) * 128);
    }
  }
  // Copies of the tile looked up, into stage st; returns which of its rows are
  // there.  Rows that are not are filled with zeros, and not read.  The pieces
  // of a row go to neighbouring lanes, so that a request takes whole lines.
  __device__ __forceinline__ uint32_t copy(int st) {
    const int lane = threadIdx.x & 31;
    const bool ok = in && page >= 0 && page < a.num_pages;
    if (in && !ok) report_pages(a.status);
    const int64_t from_row = ok ? page * a.pp + off : 0;
    const uint32_t seen = __ballot_sync(0xffffffffu, ok) & ((1u << kRows) - 1);
    const uint32_t to = ring + st * kStageBytes;
#pragma unroll
    for (int i = 0; i < kRows * kPieces / 32; ++i) {
      const int row = (i * 32 + lane) / kPieces, piece = (i * 32 + lane) % kPieces;
      const int64_t from = __shfl_sync(0xffffffffu, from_row, row) + piece * 16;
      const bool on = (seen >> row) & 1;
      cp_async16(to + row * kPitch + piece * 16, a.K + from, on);
      cp_async16(to + (kRows + row) * kPitch + piece * 16, a.V + from, on);
    }
    return seen;
  }
  __device__ __forceinline__ void produce(int st) {
    uint32_t seen = 0;
    if (at.unit < end) {
      seen = copy(st);
      at.next(a);
      if (at.unit < end) look_up();
    }
    cp_commit();
    queue = (queue >> 16) | ((uint64_t)seen << (16 * (kStages - 2)));
  }
  // Waits for the oldest tile in flight, in stage st, asks for another, and
  // returns which rows of it are there.
  __device__ __forceinline__ uint32_t next(int st) {
    cp_wait<kStages - 2>();
    __syncwarp();  // the warp's copies are all there, and its reads of the stage refilled next are done
    const uint32_t seen = (uint32_t)queue & 0xffffu;
    produce(st == 0 ? kStages - 1 : st - 1);
    return seen;
  }
};

// This block's run: its first tile and its last unit; false if it has none.
template <int kTile, int kCost>
__device__ __forceinline__ bool run_of(const DecodeParams& a, Place<kTile, kCost>* at, int64_t* end) {
  __shared__ int64_t sums[kWarps];
  Units<kTile, kThreads, kCost> units(a, sums);
  const Share share = units.share();
  const int run = blockIdx.x / a.split;
  if (run >= share.runs()) return false;
  const int64_t x = share.first(run);
  *end = share.first(run + 1);
  int64_t base;
  const int s = units.find(x, 0, &base);
  at->set(a, s, base, x);
  return at->unit < *end;
}

// With a cluster an item (and piece of its heads): this block's tiles of its item, the k-th of n equal
// shares; false if it has none.
template <int kTile, int kCost>
__device__ __forceinline__ bool share_of_item(const DecodeParams& a, Place<kTile, kCost>* at, int64_t* end) {
  const int k = blockIdx.x % a.cluster, n = blockIdx.x / a.cluster / a.split;
  at->s = n / a.items;
  at->item = n - at->s * a.items;
  at->rows = rows_of(a, at->s);
  at->tiles = tiles_of<kTile>(at->rows);
  at->t = (int)((int64_t)at->tiles * k / a.cluster);
  at->unit = at->t;
  *end = (int64_t)at->tiles * (k + 1) / a.cluster;
  return at->unit < *end;
}

// Joins the parts of a cluster's blocks: o [heads][D] and ml [heads] in the
// shared memory of each, l = kNoPart of a block without tiles, whose o is not
// read.  m alone does not tell: it is -inf too where all scores are NaN, and
// that has to come out.  Every thread of the cluster calls it.
constexpr float kNoPart = -1.f;
template <class T, int D>
__device__ __forceinline__ void join_cluster(const DecodeParams& a, const float4* o_part, const float2* ml_part) {
  constexpr int kLanes = D / 4, kMost = kMostBlocks;
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int n = blockIdx.x / a.cluster / a.split, s = n / a.items;
  int heads;
  const int h0 = first_head(a, n - s * a.items, blockIdx.x / a.cluster % a.split, &heads);
  cluster.sync();  // the parts are there
  for (int k = cluster.block_rank() * kThreads + threadIdx.x; k < heads * kLanes; k += a.cluster * kThreads) {
    const int head = k / kLanes;
    float2 ml[kMost];
    float m = -INFINITY;
#pragma unroll
    for (int r = 0; r < kMost; ++r) {
      ml[r] = r < a.cluster ? cluster.map_shared_rank(ml_part, r)[head] : make_float2(-INFINITY, kNoPart);
      m = fmaxf(m, ml[r].x);
    }
    const float base = base_of(m);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll
    for (int r = 0; r < kMost; ++r) {
      if (ml[r].y == kNoPart) continue;
      const float4 v = cluster.map_shared_rank(o_part, r)[k];
      const float w = ptx::ex2(ml[r].x - base);
      o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
      l = fmaf(w, ml[r].y, l);
    }
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
    o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    store4<T>(a.O + s * a.os + (int64_t)(h0 + head) * a.oh, 4 * (k % kLanes), o);
    if (k % kLanes == 0) a.L[(int64_t)s * a.H + h0 + head] = none ? INFINITY : (m + log2f(l)) * kLn2;
  }
  cluster.sync();  // no block leaves while another reads its part
}

// ------------------------------------------------------------------- joining
// Block (r, y): some query heads and columns of one item, item r if there are no
// more items than runs (by_item), else the one that run r ends inside of if it
// also begins there: every item of several parts has one such run.  Which parts
// it has follows from the lengths, so the blocks can find that out while the
// kernel in front still runs.  `lanes` threads hold a slice of a row of o; of
// the block's groups of so many threads, `together` take a head each and the
// others share its parts, kAhead loads at a time.
// 128 threads and their 2.2 KB of shared memory fit beside the blocks of the
// kernel in front, so the join is there when those end.  With 256 threads, on the
// same GPU: 32 sequences of 1024 rows, 32 heads of d 64, 55.4 us instead of 50.5; of
// 4096 173.3 instead of 165.4; 64 of up to 8192, 8 key heads of d 128, 138.8 instead
// of 136.9; nothing at d 256.
constexpr int kJoinThreads = 128;
struct JoinShape {
  int by_item, part_heads;
  int together;  // heads a block takes
  int slices;    // blocks that a head's columns are cut into; 1 if together > 1
};

template <class T, int D, int kTile, int kCost>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeParams a,
                                                                   const JoinShape j) {
  constexpr int kAhead = 8;
  __shared__ float4 os[kJoinThreads];
  __shared__ float2 mls[kJoinThreads / (D / 16)];  // a group has D / 16 threads at least
  __shared__ int64_t sums[kJoinThreads / 32];
  int s = 0, item = 0, run = 0, slot = 0, following = 0;
  {
    Units<kTile, kJoinThreads, kCost> units(a, sums);
    const Share share = units.share();
    int64_t base = 0;
    if (j.by_item) {
      s = blockIdx.x / a.items;
      item = blockIdx.x - s * a.items;
      units.find(-1, s, &base);
    } else if ((int)blockIdx.x < share.runs()) {
      const int64_t x = share.first(blockIdx.x + 1) - 1;
      s = units.find(x, 0, &base);
      item = (int)divide(x - base, kCost + tiles_of<kTile>(rows_of(a, s)));
    }
    const int64_t tiles = tiles_of<kTile>(rows_of(a, s)), begin = base + item * (kCost + tiles);
    run = share.run_of(begin + kCost);
    if (j.by_item || run == (int)blockIdx.x) following = share.run_of(begin + kCost + tiles - 1) - run;
    // a run that holds tiles before the item has it as its second part
    slot = share.first(run) < begin ? 1 : 0;
  }
  const int head0 = blockIdx.y / j.slices * j.together;  // of the item's query heads
  const int lanes = D / 4 / j.slices, groups = kJoinThreads / lanes;
  const int grp = threadIdx.x / lanes, x = threadIdx.x - grp * lanes;
  const int col = 4 * (blockIdx.y % j.slices * lanes + x);
  const int sharing = groups / j.together, take = j.together * sharing;  // groups that share a head's parts, and all
  // What comes after this kernel on its stream waits for this kernel alone, so
  // it may not end before the one in front, even if it has nothing to join:
  // block (0, 0) waits in any case.
  if (following > 0 || (blockIdx.x == 0 && blockIdx.y == 0)) after_stream();
  if (following == 0) return;
  if (grp < take) {
    const int h = min(head0 + grp % j.together, a.group - 1), piece = h / a.piece_heads;
    const int head = h - piece * a.piece_heads;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for (int k0 = grp / j.together; k0 <= following; k0 += sharing * kAhead) {
      float2 ml[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int k = k0 + e * sharing;
        ml[e] = make_float2(-INFINITY, 0.f);
        v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k > following) continue;
        const int64_t p = ((int64_t)(2 * (run + k) + (k == 0 ? slot : 0)) * a.split + piece) * j.part_heads + head;
        ml[e] = a.part_ml[p];
        v[e] = *reinterpret_cast<const float4*>(a.part_o + p * D + col);
      }
      float top = m;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) top = fmaxf(top, ml[e].x);
      const float base = base_of(top), f = ptx::ex2(m - base);
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
      l *= f;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const float w = ptx::ex2(ml[e].x - base);
        o.x = fmaf(w, v[e].x, o.x), o.y = fmaf(w, v[e].y, o.y), o.z = fmaf(w, v[e].z, o.z), o.w = fmaf(w, v[e].w, o.w);
        l = fmaf(w, ml[e].y, l);
      }
      m = top;
    }
    os[threadIdx.x] = o;
    if (x == 0) mls[grp] = make_float2(m, l);
  }
  __syncthreads();
  if (grp >= j.together || head0 + grp >= a.group) return;
  float m = -INFINITY;
#pragma unroll 8
  for (int k = grp; k < take; k += j.together) m = fmaxf(m, mls[k].x);
  const float base = base_of(m);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 8
  for (int k = grp; k < take; k += j.together) {
    const float4 v = os[k * lanes + x];
    const float2 ml = mls[k];
    const float w = ptx::ex2(ml.x - base);
    o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
    l = fmaf(w, ml.y, l);
  }
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  const int64_t h = (int64_t)item * a.group + head0 + grp;
  store4<T>(a.O + s * a.os + h * a.oh, col, o);
  if (col == 0) a.L[(int64_t)s * a.H + h] = none ? INFINITY : (m + log2f(l)) * kLn2;
}

// ----------------------------------------------------------------- launching
// How a problem is cut: what the workspace's size and the launch go by.
struct Cut {
  int split, piece_heads, part_heads;  // pieces of a group, heads of a piece, the same rounded up
  int64_t tiles, most_tiles;          // at most: of all items, of one
  int cluster;                        // blocks an item, or 0: runs
  int cost = kItemCost;
  // units are tiles and cost for every item, and no item has less than one tile
  int64_t units() const { return tiles * (1 + cost); }
  int64_t parts() const { return 2 * (units() * split < kMaxRuns ? units() * split : kMaxRuns); }
};

// Rows of a tile.
inline int tile_rows(const fa_cache& c) { return c.dtype == FA_FP32 && c.d == 256 ? 32 : 64; }

// Each item gets a cluster of as many blocks (1, 2, 4, 8 or 16) as the GPU holds
// at a time, if that leaves at most kClusterTiles tiles a block.  Beyond that
// the runs are quicker, which use all SMs: a block alone on its SM takes 1.1 us a
// tile.  4 sequences of up to 4000 rows, 16 heads on one of d 128, took 8.3 us in
// runs, 9.1 with 16 blocks of 4 tiles and 12.6 with 8 of 8; 8 of 512, 32 heads on 8,
// 10.2 in runs and 7.7 with 4 blocks of 2 tiles.
constexpr int kClusterTiles = 2;
// Tiles a block at most, by a cluster's size.
struct ClusterTiles {
  int sixteen = kClusterTiles, some = kClusterTiles, one = kClusterTiles;
  int of(int blocks) const { return blocks == kMostBlocks ? sixteen : blocks == 1 ? one : some; }
};
// an_sm: blocks of the kernel that an SM holds.
inline int cluster_of(int an_sm, int64_t items, int64_t most_tiles, const ClusterTiles& most) {
  // clusters that the GPU holds of each size, for each block an SM, as a GB300 of 152 SMs answers when asked: a cluster
  // stays inside a GPC.  Written down, because the workspace's size goes by this too, which is asked for without a GPU;
  // one that holds other numbers of them computes the same, in more or fewer waves.
  struct {
    int blocks, fit;
  } sizes[] = {{kMostBlocks, 7}, {8, 15}, {4, 36}, {2, 76}, {1, 152}};
  for (const auto& z : sizes) {
    if (items > (int64_t)z.fit * an_sm || z.blocks / 2 >= most_tiles) continue;  // too many, or blocks without a tile
    return most_tiles <= (int64_t)z.blocks * most.of(z.blocks) ? z.blocks : 0;
  }
  return 0;
}

// A group of query heads in even pieces of at most `most`.
inline Cut pieces_of(int group, int most) {
  Cut k;
  k.split = (int)ceil_div(group, most);
  k.piece_heads = (int)ceil_div(group, k.split);
  k.part_heads = k.piece_heads <= 8 ? 8 : 16;
  return k;
}
inline Cut cut_tiles(Cut k, const fa_cache& c, int tile, int an_sm, int cost = kItemCost, const ClusterTiles& most = {}) {
  k.cost = cost;
  k.most_tiles = ceil_div(cache_rows(c), tile);
  k.tiles = (int64_t)c.S * c.H_kv * k.most_tiles;
  k.cluster = cluster_of(an_sm, (int64_t)c.S * c.H_kv * k.split, k.most_tiles, most);
  return k;
}

inline Cut cut_of(const fa_cache& c, int H) {
  Cut k = pieces_of(H / c.H_kv, c.dtype == FA_BF16 ? 16 : 8);
  if (c.dtype != FA_BF16) k.part_heads = k.piece_heads == 1 ? 1 : k.piece_heads <= 4 ? 4 : 8;
  return cut_tiles(k, c, tile_rows(c), blocks_an_sm(c.dtype == FA_BF16, c.d));
}
// The workspace's size: no parts where there are clusters, none in global memory where items are a tile.
inline size_t workspace_of(const Cut& k, int d) {
  if (k.cluster > 0 || k.most_tiles <= 1) return 0;
  return (size_t)k.parts() * k.part_heads * (sizeof(float2) + sizeof(float) * d);
}

// The runs that the lengths can lead to at most.  Sets a->resident.
inline int runs_of(const Cut& k, int resident, DecodeParams* a) {
  if (resident > kMaxRuns / (1 + kSmallRuns)) resident = kMaxRuns / (1 + kSmallRuns);
  resident /= k.split;  // at most kMostHeads / 8 = 64: some are left
  a->resident = resident;
  if (k.units() >= (int64_t)resident * kMinUnits) return resident * (1 + kSmallRuns);
  return (int)(k.units() < resident ? k.units() : resident);
}

template <class T, int D, int kTile, int kCost>
cudaError_t launch_join(const Cut& k, const DecodeParams& a, int runs, cudaStream_t s) {
  const int64_t items = (int64_t)a.S * a.items;
  JoinShape j = {items <= runs, k.part_heads, 1, 1};
  const int64_t x = j.by_item ? items : runs;
  // few items of many parts: a head and then a slice of its columns a block, so
  // that more threads read parts; many of few: several heads a block, as long as
  // a head's parts are still read in one go
  constexpr int kMost = kJoinThreads / (D / 4);
  while (x * a.group * j.slices < 304 && j.slices < 4) j.slices *= 2;
  while (x * ceil_div(a.group, j.together) > 304 && j.together < a.group && 2 * j.together <= kMost &&
         kMost / (2 * j.together) * 8 >= runs / x + 2)
    j.together *= 2;
  const dim3 grid((unsigned)x, (unsigned)(ceil_div(a.group, j.together) * j.slices));
  return launch_early(decode_join_kernel<T, D, kTile, kCost>, grid, kJoinThreads, 0, s, 1, a, j);
}

// How many blocks of a kernel the device holds at a time; raises the kernel's
// shared-memory limit.  Asked for once a device, and kept in known[device].
inline cudaError_t resident_blocks(const void* kernel, int smem, std::atomic<int>* known, int* blocks,
                                   int threads = kThreads) {
  int dev = 0, a_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  *blocks = known[dev].load(std::memory_order_acquire);
  if (*blocks > 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  // clusters of 16 blocks
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&a_sm, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *blocks = a_sm * sm_count();
  if (*blocks < 1) return cudaErrorInvalidConfiguration;
  known[dev].store(*blocks, std::memory_order_release);
  return cudaSuccess;
}

// Launches `alone` with a cluster an item, or `kernel` with a block a run and the join.
// P: DecodeParams, or what goes on from there.
template <class T, int D, int kTile, int kCost = kItemCost, class P>
cudaError_t launch_decode(const Cut& k, P a, void (*kernel)(P), void (*alone)(P), int smem,
                          std::atomic<int>* known, std::atomic<int>* known_alone, cudaStream_t s) {
  int resident = 0;
  a.cluster = k.cluster;
  cudaError_t e = resident_blocks(k.cluster > 0 ? (const void*)alone : (const void*)kernel, smem,
                                  k.cluster > 0 ? known_alone : known, &resident);
  if (e != cudaSuccess) return e;
  if (k.cluster > 0) return launch_early(alone, dim3((unsigned)(a.S * a.items * a.split * k.cluster)), kThreads, smem, s, k.cluster, a);
  const int runs = runs_of(k, resident, &a);
  e = launch_early(kernel, dim3((unsigned)(runs * a.split)), kThreads, smem, s, 1, a);
  if (e != cudaSuccess || k.most_tiles <= 1) return e;
  return launch_join<T, D, kTile, kCost>(k, a, runs, s);
}

// The arguments of fa_decode and fa_decode_e4m3, after H is known to fit: what is wrong with them, and the
// kernels' parameters.  es: bytes of an element of the pools.
struct DecodeCall {
  const fa_cache* c;
  int32_t H;
  float scale;
  const void* Q;
  int64_t q_stride_s, q_stride_h;
  const void *K_pages, *V_pages;
  const int32_t *page_table, *lengths;
  void* O;
  int64_t o_stride_s, o_stride_h;
  float* L;
  void* workspace;
  size_t workspace_bytes;
};
inline fa_status check_call(const DecodeCall& x, size_t need) {
  const int es = elem_size(x.c->dtype), d = x.c->d;
  if (!(x.scale > 0.f) || !isfinite(x.scale * kLog2e) || x.O == x.Q || !aligned16(x.Q) || !aligned16(x.K_pages) ||
      !aligned16(x.V_pages) || !aligned16(x.O) || !aligned4(x.page_table) || !aligned4(x.lengths) || !aligned4(x.L) ||
      !good_stride(x.q_stride_s, d, es, false) || !good_stride(x.q_stride_h, d, es, false) ||
      !good_stride(x.o_stride_s, d, es, true) || !good_stride(x.o_stride_h, d, es, true))
    return FA_ERR_INVALID_ARG;
  return need > 0 && (!aligned16(x.workspace) || x.workspace_bytes < need) ? FA_ERR_INVALID_ARG : FA_OK;
}
inline void fill(const DecodeCall& x, const Cut& k, size_t need, int es, DecodeParams* a) {
  const fa_cache& c = *x.c;
  const int qes = elem_size(c.dtype);
  a->Q = (const char*)x.Q;
  a->K = (const char*)x.K_pages;
  a->V = (const char*)x.V_pages;
  a->O = (char*)x.O;
  a->L = x.L;
  a->table = x.page_table;
  a->lengths = x.lengths;
  a->part_o = (float*)x.workspace;
  a->part_ml = (float2*)(a->part_o + (need > 0 ? (size_t)k.parts() * k.part_heads * c.d : 0));
  a->page_rows = FastDiv(c.page_rows);
  a->S = c.S;
  a->H = x.H;
  a->group = x.H / c.H_kv;
  a->split = k.split;
  a->piece_heads = k.piece_heads;
  a->items = c.H_kv;
  a->num_pages = c.num_pages;
  a->max_pages = c.max_pages;
  a->cap = (int)cache_rows(c);
  a->table_stride = c.table_stride;
  a->qs = x.q_stride_s * qes;
  a->qh = x.q_stride_h * qes;
  a->os = x.o_stride_s * qes;
  a->oh = x.o_stride_h * qes;
  a->pp = c.stride_page * es;
  a->ph = c.stride_h * es;
  a->pn = c.stride_n * es;
  a->scale2 = x.scale * kLog2e;
}
// H against a cache that has been checked.
inline fa_status check_heads(const fa_cache* c, int32_t H) {
  if (H < 1 || H % c->H_kv != 0) return FA_ERR_INVALID_ARG;
  return (int64_t)c->S * H > (1 << 24) || H / c->H_kv > kMostHeads ? FA_ERR_UNSUPPORTED : FA_OK;
}

cudaError_t launch_decode_bf16(const fa_cache& c, const Cut& k, const DecodeParams& a, cudaStream_t s);
cudaError_t launch_decode_fp32(const fa_cache& c, const Cut& k, const DecodeParams& a, cudaStream_t s);
// fa_decode_e4m3 with tcgen05: whether it takes the problem.
bool takes_sm103(const fa_cache& c, int H);
Cut cut_e4m3_sm103(const fa_cache& c, int H);
cudaError_t launch_e4m3_sm103(int d, const Cut& k, const E4m3Params& a, cudaStream_t s);

}  // namespace fa
