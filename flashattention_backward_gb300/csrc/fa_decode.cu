// Attention of one new token over a paged key-value cache (fa_decode).
//
//   s_j = scale q . k_j,  m = max_j s_j,  l = sum_j 2^(s_j - m),
//   O = sum_j 2^(s_j - m) v_j / l,  L = (m + log2 l) ln 2
// with scores in units of log 2 (the scale carries log2 e).  Over disjoint
// ranges of rows with (m_i, l_i, o_i), o unnormalised, m = max m_i and the l
// and o add up with the factors 2^(m_i - m).
//
// Every row of the cache is read once for the group of query heads that share
// it, 2 d elements a row against 4 d multiply-adds a query head: with 8 heads a
// group that is 8 flops a byte in bf16, far below what the tensor cores need
// to be the limit.  HBM is, so the design is about loads: all SMs have an
// equal share of the rows, whatever the lengths, and each keeps about 100 KB
// of loads in flight.
//
// Work.  An item is one sequence, one key-value head and up to 8 * NH of its
// query heads; a tile is kTile rows of an item.  All tiles of all items in
// order, numbered through, are cut into equal runs, one for each of `workers`
// blocks (as many as are resident at a time).  A block finds its run from the
// lengths itself: the host knows none of them.  A run may end inside an item.
// What a block has then goes to the workspace as (m, l, o), at most two such
// parts a block: one of an item that began in an earlier block's run and one
// of an item that goes on in the next one's.  decode_join_kernel adds the
// parts of an item up, in the order of the blocks.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "fa_paged.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWorkers = 1024;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  const char *Q, *K, *V;
  char* O;
  float* L;
  const int32_t *table, *lengths;
  int32_t* status;
  float2* part_ml;    // [2 workers][heads of an item]
  float* part_o;      // [2 workers][heads of an item][d]
  FastDiv page_rows;
  int S, H, group;    // group: query heads that share a key-value head
  int split;          // items a group is cut into
  int item_heads;     // query heads of an item (the last of a group may have fewer)
  int items;          // of a sequence: H_kv * split
  int num_pages, max_pages;
  int cap;            // page_rows * max_pages
  int workers;
  int64_t table_stride;
  int64_t qs, qh, os, oh;  // byte strides
  int64_t pp, ph, pn;
  float scale2;       // scale * log2(e)
};

// ------------------------------------------------------------- sharing out
__device__ __forceinline__ int rows_of(const DecodeParams& a, int s) {
  const int n = __ldg(a.lengths + s);
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
// what measured best: 32 sequences of up to 2048 rows, 32 heads of d 64 (items
// of up to 32 tiles) took 56.5 us with 0, 46.3 with 1, 46.5 with 2, 47.4 with 3.
constexpr int kItemCost = 1;

struct Share {
  int64_t total;  // units of all items
  int workers;    // blocks that have a run
  __device__ __forceinline__ int64_t first(int w) const { return total * w / workers; }
  // the block whose run holds unit x: the largest w with first(w) <= x
  __device__ __forceinline__ int block_of(int64_t x) const { return (int)(((x + 1) * workers - 1) / total); }
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
template <int kTile, int NT>
struct Units {
  const DecodeParams& a;
  int64_t* sums;     // NT / 32 entries of shared memory
  int64_t n, lo, all;  // of the first NT sequences: this thread's, those before it, all
  __device__ __forceinline__ int64_t of(int s) const {
    return s < a.S ? (int64_t)(kItemCost + tiles_of<kTile>(rows_of(a, s))) * a.items : 0;
  }
  __device__ __forceinline__ Units(const DecodeParams& p, int64_t* shared) : a(p), sums(shared) {
    n = of(threadIdx.x);
    lo = block_scan<NT>(n, sums, &all);
  }
  __device__ __forceinline__ Share share() {
    Share sh;
    sh.total = all;
    if (a.S > NT) {
      int64_t more = 0;
      for (int s = NT + threadIdx.x; s < a.S; s += NT) more += of(s);
      block_scan<NT>(more, sums, &more);
      sh.total += more;
    }
    sh.workers = (int)(sh.total < a.workers ? sh.total : a.workers);
    return sh;
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
template <int kTile>
struct Place {
  int s, item, t, rows, tiles;
  int64_t unit;
  // the first tile at or behind unit x of sequence s, whose first unit is base
  __device__ __forceinline__ void set(const DecodeParams& a, int seq, int64_t base, int64_t x) {
    s = seq;
    rows = rows_of(a, s);
    tiles = tiles_of<kTile>(rows);
    item = (int)((x - base) / (kItemCost + tiles));
    const int64_t begin = base + (int64_t)item * (kItemCost + tiles);
    t = max((int)(x - begin) - kItemCost, 0);
    unit = begin + kItemCost + t;
  }
  __device__ __forceinline__ void next(const DecodeParams& a) {
    ++unit;
    if (++t < tiles) return;
    t = 0;
    unit += kItemCost;
    if (++item < a.items) return;
    item = 0;
    if (++s < a.S) {
      rows = rows_of(a, s);
      tiles = tiles_of<kTile>(rows);
    }
  }
};

// The query heads of an item: the first one, and how many.
__device__ __forceinline__ int item_first_head(const DecodeParams& a, int item, int* kv, int* heads) {
  *kv = item / a.split;
  const int part = item - *kv * a.split;
  *heads = min(a.item_heads, a.group - part * a.item_heads);
  return *kv * a.group + part * a.item_heads;
}

__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }

template <class T>
__device__ __forceinline__ void store4(char* row, int col, float4 x) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4*>(row + 4 * col) = x;
  else
    *reinterpret_cast<uint2*>(row + 2 * col) = make_uint2(ptx::pack_bf16x2(x.x, x.y), ptx::pack_bf16x2(x.z, x.w));
}

// ------------------------------------------------------- bf16: tensor cores
// A warp takes 16 rows of each tile with mma.m16n8k16:
//
//  S = Q K^T     A = 16 query heads x 16 columns, B = 16 columns x 8 keys.
//                A sum may be taken in any order, so the 16 columns of a step are
//                those that make a lane's share of B a run of 16 bytes of a key,
//                two steps' worth, and the same columns of Q are A's.
//  O^T += V^T P^T  A = 16 columns x 16 keys, B = 16 keys x 8 heads: S's
//                accumulators are P^T's operand as they stand.  A's pairs of
//                keys come from two rows: lane (g, q) reads columns 64 c + 8 g
//                ... + 7 of keys 2q, 2q + 1, 2q + 8, 2q + 9, and byte permutes pair
//                them.  Column 64 c + 8 g + 2 i + r is row g + 8 r of product i.
//
// A warp copies its own 16 rows (cp.async into a ring of its own) and waits for
// them alone: no block barrier in the loop, no transposition, conflict-free
// 16-byte shared-memory reads.  tcgen05 would want 64 or 128 rows of A where
// there are 1 to 16 query heads, and a barrier a tile, for a product that is
// not the limit.
//
// P is multiplied as the sum of two bf16 numbers (p rounded, and what is left
// rounded): the second product costs nothing beside the loads, and leaves the
// rounding of the output as the only one to fewer than 16 bits.
template <int D>
struct Mma {
  static constexpr int kRows = 16;             // of a tile, a warp
  static constexpr int kTile = kWarps * kRows;
  static constexpr int kVW = D % 64 ? 32 : 64; // columns of V in a block: 8 or 16 bytes a lane
  static constexpr int kPieces = D / 8;        // of 16 bytes in a row
  // 16 bytes between rows: the 8 lanes of an access's quarter then take 8
  // different groups of 4 banks, of K (2 keys x 4 pieces, 2 apart) as of V (4 pairs
  // of keys, 2 pieces)
  static constexpr int kPitch = D * 2 + 16;
  static constexpr int kStageBytes = 2 * kRows * kPitch;  // K and V rows of a warp
  // Bytes in flight an SM: (stages - 1) of blocks x warps x 64 d.  Shared
  // memory holds 228 KB an SM, and 8 to 16 warps keep the issue slots fed.
  static constexpr int kBlocks = D == 32 ? 4 : D == 64 ? 3 : D == 256 ? 1 : 2;  // an SM
  static constexpr int kStages = D == 32 || D == 96 ? 4 : 3;
  // the place in a row of the piece that lane q multiplies in step c, in pieces
  __host__ __device__ static constexpr int k_piece(int c, int q) {
    return c == D / 32 - 1 && c % 2 == 0 ? 4 * c + q : 8 * (c / 2) + 2 * q + c % 2;
  }
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kPad = kVW + 4;         // floats of a row of the exchange buffer
  static constexpr int kExchange = kWarps * 8 * kPad * 4;
  static constexpr int kSmem = kRing + kExchange;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const char* src, bool on) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void prefetch_l1(const char* p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int D, int NH>
__global__ void __launch_bounds__(kThreads, Mma<D>::kBlocks) decode_mma_kernel(const __grid_constant__ DecodeParams a) {
  using M = Mma<D>;
  constexpr int kTile = M::kTile, kStages = M::kStages, VW = M::kVW;
  constexpr int kHeads = 8 * NH;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t sums[kWarps];
  __shared__ float2 ml[kWarps][kHeads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t ring = ptx::smem_addr(smem) + warp * kStages * M::kStageBytes;
  float* exchange = reinterpret_cast<float*>(smem + M::kRing);

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join's blocks may line up
  Place<kTile> load, at;
  int64_t end;
  {
    Units<kTile, kThreads> units(a, sums);
    const Share share = units.share();
    if ((int)blockIdx.x >= share.workers) return;
    const int64_t x = share.first(blockIdx.x);
    end = share.first(blockIdx.x + 1);
    int64_t base;
    const int s = units.find(x, 0, &base);
    at.set(a, s, base, x);
  }
  if (at.unit >= end) return;
  load = at;

  // The row that this lane looks up in the tile that is loaded next: its page
  // is asked for one tile ahead of the copies that need it.
  int row_page = -1;
  bool row_in = false;
  int64_t row_off = 0;
  auto look_up = [&]() {
    const int j = load.t * kTile + warp * M::kRows + (lane & 15);
    uint32_t r;
    const uint32_t col = a.page_rows.div((uint32_t)j, &r);
    row_in = j < load.rows;
    row_page = row_in ? __ldg(a.table + load.s * a.table_stride + col) : -1;
    row_off = (int64_t)(load.item / a.split) * a.ph + (int64_t)r * a.pn;
    if (load.t == 0) {  // a new item: its queries into L1
      int kv, heads;
      const char* row = a.Q + load.s * a.qs + (int64_t)item_first_head(a, load.item, &kv, &heads) * a.qh;
      constexpr int kLines = (D * 2 + 127) / 128;
      for (int k = lane; k < heads * kLines; k += 32) prefetch_l1(row + (k / kLines) * a.qh + (k % kLines) * 128);
    }
  };
  // Copies of the tile looked up, into stage st; returns which of its 16 rows
  // are there.  Rows that are not are filled with zeros, and not read.  The
  // pieces of a row go to neighbouring lanes, so that a request takes whole
  // lines of a row.
  auto copy = [&](int st) -> uint32_t {
    const bool ok = row_in && row_page >= 0 && row_page < a.num_pages;
    if (row_in && !ok) report_pages(a.status);
    const int64_t off = ok ? row_page * a.pp + row_off : 0;
    const uint32_t seen = __ballot_sync(0xffffffffu, ok) & 0xffffu;
    const uint32_t to = ring + st * M::kStageBytes;
#pragma unroll
    for (int i = 0; i < M::kPieces / 2; ++i) {
      const int row = (i * 32 + lane) / M::kPieces, piece = (i * 32 + lane) % M::kPieces;
      const int64_t from = __shfl_sync(0xffffffffu, off, row) + piece * 16;
      const bool on = (seen >> row) & 1;
      cp_async16(to + row * M::kPitch + piece * 16, a.K + from, on);
      cp_async16(to + M::kStageBytes / 2 + row * M::kPitch + piece * 16, a.V + from, on);
    }
    return seen;
  };
  // seen masks of the tiles in flight, the oldest in the low 16 bits
  uint64_t seen_queue = 0;
  auto produce = [&](int st) {
    uint32_t seen = 0;
    if (load.unit < end) {
      seen = copy(st);
      load.next(a);
      if (load.unit < end) look_up();
    }
    cp_commit();
    seen_queue = (seen_queue >> 16) | ((uint64_t)seen << (16 * (kStages - 2)));
  };
  look_up();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) produce(i);

  uint32_t qf[NH][D / 32][4];
  float acc[NH][D / VW][VW / 16][4];  // O^T, unnormalised
  float m[NH], l[NH];                 // of heads g, g + 8; l of this lane's keys alone
  int begin = at.t;                   // tile at which the item (or this block's part of it) began
  int stage = 0;
  bool first = true, last = false;    // item of the run

  for (bool fresh = true; !last; fresh = false) {
    Place<kTile> next = at;
    next.next(a);
    last = next.unit >= end;
    cp_wait<kStages - 2>();
    __syncwarp();  // the warp's copies are all there, and its reads of the stage refilled next are done
    const uint32_t seen = (uint32_t)seen_queue & 0xffffu;
    produce(stage == 0 ? kStages - 1 : stage - 1);

    if (fresh || at.t == 0) {
      int kv, heads;
      const int h0 = item_first_head(a, at.item, &kv, &heads);
      const char* row = a.Q + at.s * a.qs + (int64_t)h0 * a.qh;
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        const bool on = g + 8 * u < heads;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 x = on ? __ldg(reinterpret_cast<const uint4*>(row + (g + 8 * u) * a.qh + M::k_piece(c, q) * 16))
                             : make_uint4(0, 0, 0, 0);
          qf[u][c][0] = x.x, qf[u][c][1] = x.y, qf[u][c][2] = x.z, qf[u][c][3] = x.w;
        }
        m[u] = -INFINITY;
        l[u] = 0.f;
#pragma unroll
        for (int c = 0; c < D / VW; ++c)
#pragma unroll
          for (int e = 0; e < VW / 16; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[u][c][e][x] = 0.f;
      }
      begin = at.t;
    }

    if (seen) {
      const uint32_t k_at = ring + stage * M::kStageBytes + g * M::kPitch;
      float s[2][4] = {};
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint4 k0 = lds16(k_at + M::k_piece(c, q) * 16), k1 = lds16(k_at + 8 * M::kPitch + M::k_piece(c, q) * 16);
        const uint32_t b0 = NH > 1 ? qf[NH - 1][c][0] : 0u, b1 = NH > 1 ? qf[NH - 1][c][1] : 0u;
        const uint32_t b2 = NH > 1 ? qf[NH - 1][c][2] : 0u, b3 = NH > 1 ? qf[NH - 1][c][3] : 0u;
        mma16816(s[0], qf[0][c][0], b0, qf[0][c][1], b1, k0.x, k0.y);
        mma16816(s[1], qf[0][c][0], b0, qf[0][c][1], b1, k1.x, k1.y);
        mma16816(s[0], qf[0][c][2], b2, qf[0][c][3], b3, k0.z, k0.w);
        mma16816(s[1], qf[0][c][2], b2, qf[0][c][3], b3, k1.z, k1.w);
      }
      // rows 2q, 2q + 1 (s[0]) and 2q + 8, 2q + 9 (s[1]) of the warp's 16
      const uint32_t mine = seen >> (2 * q);
      uint32_t hi[NH][2], lo[NH][2];
      float alpha[NH];
      bool moved = false;
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        float x[4];
        x[0] = mine & 1 ? s[0][2 * u] * a.scale2 : -INFINITY;
        x[1] = mine & 2 ? s[0][2 * u + 1] * a.scale2 : -INFINITY;
        x[2] = mine & 256 ? s[1][2 * u] * a.scale2 : -INFINITY;
        x[3] = mine & 512 ? s[1][2 * u + 1] * a.scale2 : -INFINITY;
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float now = fmaxf(m[u], top), base = base_of(now);
        alpha[u] = ptx::ex2(m[u] - base);
        moved |= now != m[u];
        m[u] = now;
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ptx::ex2(x[e] - base);
        l[u] = l[u] * alpha[u] + ((p[0] + p[1]) + (p[2] + p[3]));
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          hi[u][e] = ptx::pack_bf16x2(p[2 * e], p[2 * e + 1]);
          lo[u][e] = ptx::pack_bf16x2(p[2 * e] - __uint_as_float(hi[u][e] << 16),
                                      p[2 * e + 1] - __uint_as_float(hi[u][e] & 0xffff0000u));
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
        // the factors belong to heads g, the accumulators to heads 2q, 2q + 1
#pragma unroll
        for (int u = 0; u < NH; ++u) {
          const float f0 = __shfl_sync(0xffffffffu, alpha[u], 8 * q), f1 = __shfl_sync(0xffffffffu, alpha[u], 8 * q + 4);
#pragma unroll
          for (int c = 0; c < D / VW; ++c)
#pragma unroll
            for (int e = 0; e < VW / 16; ++e) {
              acc[u][c][e][0] *= f0, acc[u][c][e][2] *= f0;
              acc[u][c][e][1] *= f1, acc[u][c][e][3] *= f1;
            }
        }
      }
      constexpr int kLaneV = VW / 4, kWords = VW / 16;
      const uint32_t v_at = ring + stage * M::kStageBytes + M::kStageBytes / 2 + 2 * q * M::kPitch + g * kLaneV;
#pragma unroll
      for (int c = 0; c < D / VW; ++c) {
        uint32_t w[4][kWords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t from = v_at + ((r & 1) + (r >> 1) * 8) * M::kPitch + c * VW * 2;
          if constexpr (VW == 64) {
            const uint4 x = lds16(from);
            w[r][0] = x.x, w[r][1] = x.y, w[r][2] = x.z, w[r][3] = x.w;
          } else {
            const uint2 x = lds8(from);
            w[r][0] = x.x, w[r][1] = x.y;
          }
        }
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
          const uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5410), a1 = __byte_perm(w[0][e], w[1][e], 0x7632);
          const uint32_t a2 = __byte_perm(w[2][e], w[3][e], 0x5410), a3 = __byte_perm(w[2][e], w[3][e], 0x7632);
#pragma unroll
          for (int u = 0; u < NH; ++u) {
            mma16816(acc[u][c][e], a0, a1, a2, a3, hi[u][0], hi[u][1]);
            mma16816(acc[u][c][e], a0, a1, a2, a3, lo[u][0], lo[u][1]);
          }
        }
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;

    if (at.t + 1 == at.tiles || last) {
      // ---- the item ends here, or goes on in the next block's run
      const bool whole = begin == 0 && at.t + 1 == at.tiles;
      // the part of an item that was being read when the run began is the
      // block's first, any other its second
      const int slot = 2 * blockIdx.x + (first ? 0 : 1);
      first = false;
      int kv, heads;
      const int h0 = item_first_head(a, at.item, &kv, &heads);
      __syncthreads();  // ml and the exchange buffer have been read
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if (q == 0) ml[warp][g + 8 * u] = make_float2(m[u], l[u]);
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        // this warp's factor of heads 2q, 2q + 1
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k][8 * u + 2 * q + e].x);
          f[e] = ptx::ex2(ml[warp][8 * u + 2 * q + e].x - base_of(top));
        }
        // the head and the four columns that this thread adds up
        const int head = threadIdx.x / (VW / 4), col = threadIdx.x % (VW / 4) * 4;
        float top = -INFINITY, sum = 0.f;
        if (head < 8) {
#pragma unroll
          for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k][8 * u + head].x);
#pragma unroll
          for (int k = 0; k < kWarps; ++k) sum += ml[k][8 * u + head].y * ptx::ex2(ml[k][8 * u + head].x - base_of(top));
        }
        const bool mine = head < 8 && 8 * u + head < heads;
        const bool none = sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
        for (int c = 0; c < D / VW; ++c) {
          if (u + c > 0) __syncthreads();
          float* mine_at = exchange + ((warp * 8 + 2 * q) * M::kPad + g * (VW / 8));
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < VW / 16; x += 2)
              *reinterpret_cast<float4*>(mine_at + e * M::kPad + 2 * x) =
                  make_float4(acc[u][c][x][e] * f[e], acc[u][c][x][2 + e] * f[e], acc[u][c][x + 1][e] * f[e],
                              acc[u][c][x + 1][2 + e] * f[e]);
          __syncthreads();
          if (mine) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
              const float4 x = *reinterpret_cast<const float4*>(exchange + (k * 8 + head) * M::kPad + col);
              o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
            }
            if (whole) {
              o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
              store4<__nv_bfloat16>(a.O + at.s * a.os + (int64_t)(h0 + 8 * u + head) * a.oh, c * VW + col, o);
            } else {
              *reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * kHeads + 8 * u + head) * D + c * VW + col) = o;
            }
          }
        }
        if (mine && col == 0) {
          if (whole)
            a.L[(int64_t)at.s * a.H + h0 + 8 * u + head] = none ? INFINITY : (top + log2f(sum)) * kLn2;
          else
            a.part_ml[(int64_t)slot * kHeads + 8 * u + head] = make_float2(top, sum);
        }
      }
    }
    at = next;
  }
}

// ------------------------------------------------------------ fp32: CUDA cores
// One block per (sequence, query head), whose warps take the rows in turn.
template <int D>
__global__ void __launch_bounds__(kThreads) decode_fp32_kernel(const __grid_constant__ DecodeParams a) {
  constexpr int E = (D + 31) / 32;  // columns a lane holds: lane, lane + 32, ...
  __shared__ float part[kWarps][D], ms[kWarps], ls[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.x / a.H, h = blockIdx.x % a.H, kv = h / a.group;
  const int n = rows_of(a, s);
  const float* q = (const float*)(a.Q + s * a.qs + h * a.qh);
  float qv[E], o[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = lane + 32 * e < D ? q[lane + 32 * e] : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < n; j += kWarps) {
    uint32_t r;
    const uint32_t col = a.page_rows.div(j, &r);
    const int page = __ldg(a.table + s * a.table_stride + col);
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) report_pages(a.status);
      continue;
    }
    const int64_t at = page * a.pp + kv * a.ph + (int64_t)r * a.pn;
    float x = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane + 32 * e;
      x = fmaf(c < D ? ((const float*)(a.K + at))[c] : 0.f, qv[e], x);
      v[e] = c < D ? ((const float*)(a.V + at))[c] : 0.f;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= a.scale2;
    const float now = fmaxf(m, x), base = base_of(now);
    const float alpha = ptx::ex2(m - base), p = ptx::ex2(x - base);
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + p * v[e];
    m = now;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane + 32 * e < D) part[warp][lane + 32 * e] = o[e];
  if (lane == 0) ms[warp] = m, ls[warp] = l;
  __syncthreads();
  float top = -INFINITY, sum = 0.f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ms[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = ptx::ex2(ms[w] - base_of(top));
    sum += f[w] * ls[w];
  }
  const bool none = sum == 0.f;
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += f[w] * part[w][c];
    ((float*)(a.O + s * a.os + h * a.oh))[c] = none ? 0.f : x / sum;
  }
  if (threadIdx.x == 0) a.L[blockIdx.x] = none ? INFINITY : (top + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------- joining
// Block (r, h): head h of one item, item r if there are no more items than runs
// (by_item), else the one that run r ends inside of if it also begins there:
// every item of several parts has one such run.  Which parts it has follows
// from the lengths, so the blocks find that out while the kernel in front
// still runs.  D / 4 threads hold a row of o, and the block's groups of so many
// threads take the parts in turn, kAhead loads at a time.
constexpr int kJoinThreads = 256;

template <class T, int D, int kTile>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeParams a,
                                                                   int part_heads, int by_item) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes, kAhead = 4;
  __shared__ float4 os[kGroups][kLanes];
  __shared__ float2 mls[kGroups];
  __shared__ int64_t sums[kJoinThreads / 32];
  int s = 0, item = 0, block = 0, slot = 0, following = 0;
  {
    Units<kTile, kJoinThreads> units(a, sums);
    const Share share = units.share();
    int64_t base = 0;
    if (by_item) {
      s = blockIdx.x / a.items;
      item = blockIdx.x - s * a.items;
      units.find(-1, s, &base);
    } else if ((int)blockIdx.x < share.workers) {
      const int64_t x = share.first(blockIdx.x + 1) - 1;
      s = units.find(x, 0, &base);
      item = (int)((x - base) / (kItemCost + tiles_of<kTile>(rows_of(a, s))));
    }
    const int64_t tiles = tiles_of<kTile>(rows_of(a, s)), begin = base + item * (kItemCost + tiles);
    block = share.block_of(begin + kItemCost);
    if (by_item || block == (int)blockIdx.x) following = share.block_of(begin + kItemCost + tiles - 1) - block;
    // a run that holds tiles before the item has it as its second part
    slot = share.first(block) < begin ? 1 : 0;
  }
  const int head = blockIdx.y;
  int kv, heads;
  const int h = item_first_head(a, item, &kv, &heads) + head;
  const bool some = following > 0 && head < heads;
  // What comes after this kernel on its stream waits for this kernel alone, so
  // it may not end before the one in front, even if it has nothing to join:
  // block (0, 0) waits in any case.
  if (some || (blockIdx.x == 0 && blockIdx.y == 0)) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!some) return;
  const int grp = threadIdx.x / kLanes, x = threadIdx.x % kLanes;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  if (grp < kGroups) {
    for (int k0 = grp; k0 <= following; k0 += kGroups * kAhead) {
      float2 ml[kAhead];
      float4 v[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int k = k0 + e * kGroups;
        ml[e] = make_float2(-INFINITY, 0.f);
        v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k > following) continue;
        const int64_t p = (int64_t)(2 * (block + k) + (k == 0 ? slot : 0)) * part_heads + head;
        ml[e] = a.part_ml[p];
        v[e] = *reinterpret_cast<const float4*>(a.part_o + p * D + 4 * x);
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
    os[grp][x] = o;
    if (x == 0) mls[grp] = make_float2(m, l);
  }
  __syncthreads();
  if (threadIdx.x >= kLanes) return;
  m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) m = fmaxf(m, mls[k].x);
  const float base = base_of(m);
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  l = 0.f;
#pragma unroll 8
  for (int k = 0; k < kGroups; ++k) {
    const float4 v = os[k][x];
    const float w = ptx::ex2(mls[k].x - base);
    o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y), o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
    l = fmaf(w, mls[k].y, l);
  }
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  store4<T>(a.O + s * a.os + (int64_t)h * a.oh, 4 * x, o);
  if (threadIdx.x == 0) a.L[(int64_t)s * a.H + h] = none ? INFINITY : (m + log2f(l)) * kLn2;
}

// ----------------------------------------------------------------- launching
// How a problem is cut: what the workspace's size and the launch go by.
struct Cut {
  int split, item_heads, part_heads;  // items a group is cut into, heads of an item, heads of a part's slots
  int64_t most_tiles;                 // of an item
  int workers;                        // at most
};

Cut cut_of(const fa_cache& c, int H) {
  Cut k;
  const int group = H / c.H_kv;
  // up to 16 query heads share one reading of the cache; larger groups are cut
  // evenly, and read it again (from L2 where it holds an item)
  k.split = (int)ceil_div(group, 16);
  k.item_heads = (int)ceil_div(group, k.split);
  k.part_heads = k.item_heads <= 8 ? 8 : 16;
  k.most_tiles = ceil_div(cache_rows(c), 64);
  const int64_t tiles = (int64_t)c.S * c.H_kv * k.split * k.most_tiles;
  k.workers = (int)(tiles < kMaxWorkers ? tiles : kMaxWorkers);
  return k;
}

template <class T, int D, int kTile>
cudaError_t launch_join(const DecodeParams& a, int part_heads, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int by_item = (int64_t)a.S * a.items <= a.workers;
  cfg.gridDim = dim3((unsigned)(by_item ? a.S * a.items : a.workers), (unsigned)a.item_heads);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  // its blocks may be there before the kernel in front ends, and wait for that themselves
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_join_kernel<T, D, kTile>, a, part_heads, by_item);
}

// Raises a kernel's shared-memory limit, once a device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<bool>* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
  return cudaSuccess;
}

template <int D, int NH>
cudaError_t launch_mma(const Cut& k, DecodeParams a, cudaStream_t s) {
  using M = Mma<D>;
  static std::atomic<bool> ready[64];
  cudaError_t e = allow_smem((const void*)decode_mma_kernel<D, NH>, M::kSmem, ready);
  if (e != cudaSuccess) return e;
  const int resident = sm_count() * M::kBlocks;
  if (resident < 1) return cudaErrorInvalidDevice;
  if (a.workers > resident) a.workers = resident;
  decode_mma_kernel<D, NH><<<a.workers, kThreads, M::kSmem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || k.most_tiles <= 1) return e;
  return launch_join<__nv_bfloat16, D, M::kTile>(a, k.part_heads, s);
}

template <int D>
cudaError_t launch_bf16(const Cut& k, const DecodeParams& a, cudaStream_t s) {
  return k.part_heads == 8 ? launch_mma<D, 1>(k, a, s) : launch_mma<D, 2>(k, a, s);
}

template <int D>
cudaError_t launch_fp32(const Cut&, const DecodeParams& a, cudaStream_t s) {
  decode_fp32_kernel<D><<<a.S * a.H, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

// H against the cache; the strides of Q and O are checked by the entry point.
fa_status check_heads(const fa_cache* c, int32_t H) {
  const fa_status st = check_cache(c);
  if (st != FA_OK) return st;
  if (H < 1 || H % c->H_kv != 0) return FA_ERR_INVALID_ARG;
  if ((int64_t)c->S * H > (1 << 24)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_decode_workspace_bytes(const fa_cache* c, int32_t H) {
  if (fa::check_heads(c, H) != FA_OK) return 0;
  const fa::Cut k = fa::cut_of(*c, H);
  if (k.most_tiles <= 1) return 0;
  return 2 * (size_t)k.workers * k.part_heads * (sizeof(float2) + sizeof(float) * c->d);
}

fa_status fa_decode(const fa_cache* c, int32_t H, float scale, const void* Q, int64_t q_stride_s, int64_t q_stride_h,
                    const void* K_pages, const void* V_pages, const int32_t* page_table, const int32_t* lengths,
                    void* O, int64_t o_stride_s, int64_t o_stride_h, float* L, void* workspace,
                    size_t workspace_bytes, void* stream) {
  fa::NvtxRange range("fa_decode");
  const fa_status st = fa::check_heads(c, H);
  if (st != FA_OK) return st;
  const int es = fa::elem_size(c->dtype);
  if (!(scale > 0.f) || !isfinite(scale) || !fa::aligned16(Q) || !fa::aligned16(K_pages) || !fa::aligned16(V_pages) ||
      !fa::aligned16(O) || !fa::aligned4(page_table) || !fa::aligned4(lengths) || !fa::aligned4(L) ||
      !fa::good_stride(q_stride_s, c->d, es, false) || !fa::good_stride(q_stride_h, c->d, es, false) ||
      !fa::good_stride(o_stride_s, c->d, es, true) || !fa::good_stride(o_stride_h, c->d, es, true))
    return FA_ERR_INVALID_ARG;
  const size_t need = fa_decode_workspace_bytes(c, H);
  if (need > 0 && (!fa::aligned16(workspace) || workspace_bytes < need)) return FA_ERR_INVALID_ARG;
  const fa::Cut k = fa::cut_of(*c, H);
  fa::DecodeParams a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  a.Q = (const char*)Q;
  a.K = (const char*)K_pages;
  a.V = (const char*)V_pages;
  a.O = (char*)O;
  a.L = L;
  a.table = page_table;
  a.lengths = lengths;
  a.part_o = (float*)workspace;
  a.part_ml = (float2*)(a.part_o + (need > 0 ? 2 * (size_t)k.workers * k.part_heads * c->d : 0));
  a.page_rows = fa::FastDiv(c->page_rows);
  a.S = c->S;
  a.H = H;
  a.group = H / c->H_kv;
  a.split = k.split;
  a.item_heads = k.item_heads;
  a.items = c->H_kv * k.split;
  a.num_pages = c->num_pages;
  a.max_pages = c->max_pages;
  a.cap = (int)fa::cache_rows(*c);
  a.workers = k.workers;
  a.table_stride = c->table_stride;
  a.qs = q_stride_s * es;
  a.qh = q_stride_h * es;
  a.os = o_stride_s * es;
  a.oh = o_stride_h * es;
  a.pp = c->stride_page * es;
  a.ph = c->stride_h * es;
  a.pn = c->stride_n * es;
  a.scale2 = scale * fa::kLog2e;
  const cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = cudaErrorInvalidValue;
  if (c->dtype == FA_BF16) {
    switch (c->d) {
      case 32: e = fa::launch_bf16<32>(k, a, s); break;
      case 64: e = fa::launch_bf16<64>(k, a, s); break;
      case 96: e = fa::launch_bf16<96>(k, a, s); break;
      case 128: e = fa::launch_bf16<128>(k, a, s); break;
      case 256: e = fa::launch_bf16<256>(k, a, s); break;
    }
  } else {
    switch (c->d) {
      case 16: e = fa::launch_fp32<16>(k, a, s); break;
      case 32: e = fa::launch_fp32<32>(k, a, s); break;
      case 64: e = fa::launch_fp32<64>(k, a, s); break;
      case 96: e = fa::launch_fp32<96>(k, a, s); break;
      case 128: e = fa::launch_fp32<128>(k, a, s); break;
      case 256: e = fa::launch_fp32<256>(k, a, s); break;
    }
  }
  return fa::status_of(e);
}

}  // extern "C"
