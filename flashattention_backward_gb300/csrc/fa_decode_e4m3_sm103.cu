// Attention of one new token over a paged key-value cache in 8 bits on the fifth
// generation's tensor cores: the large bf16 problems of fa_decode_e4m3 with d 128
// or 256 and up to four query heads a key head.  The formulas are those of
// fa_decode_e4m3.cu, which has the others; how the work is shared out and joined is
// in fa_decode.cuh.
//
// HBM is the bound if the instructions that every byte takes are few enough.  As
// 16-bit numbers for mma.sync they are half of the time: 450 instructions for 4 KB (d 128),
// 48 % of the issue slots, and each warp waits for its own chain of them.  So the stored numbers go into tcgen05.mma
// as they are, keys and values as the operand of 128 rows:
//
//  S [128 keys, 16] = K [128, d] Q^T             K-major, under the swizzle of 128 bytes
//  O^T [d, 16] += V^T [d, 128 keys] P [128, 16]  the same rows of V, read MN-major
//
// and the other operand, queries and weights, is cut into terms of 8 bits, side by side as
// columns, of which a product has 16 at least.
//  Queries are three e4m3 numbers, x = t0 + t1 / 32 + t2 / 1024.  A head's are multiplied by the power of two
//  that takes the largest to 2^7 ... 2^8 before that: the 8 bits of a bf16 number are held exactly down to
//  2^-19 of the largest, and to 2^-27 of it below.
//  Weights are four e5m2 numbers, x = t0 + t1 / 16 + t2 / 256 + t3 / 4096, off by at most 2^-15 of the weight or, if
//  that is more, 2^-29, where the largest is 2^7 or more: 2^-36 of the largest weight.  Range counts here more than
//  bits: the sum that O is divided by has every weight in fp32, and many small ones behind one that is large may be
//  most of O.  Three e4m3 terms, 32 apart, with the largest weight at 2 lost all below 2^-20 of it: with 2^15 rows of
//  2^-17 behind a first one whose value is 0, O was off by a fifth and more.
// Sums are fp32: against 64 bits S and O were off by at most 2^-21.5 of the sum of their
// terms' absolute values, with terms of 14 binades.
//
// A kernel that uses tensor memory has one block on an SM (cudaOccupancyMax-
// ActiveBlocksPerMultiprocessor says so, and the counters), so one block has
// everything: one or two groups of warps, each with a run, a ring of tiles and
// barriers of its own.  Of a group
//   two or four warps  look up pages and copy rows and scales (cp.async: pages end anywhere)
//   one thread         issues the products, S of the next tile before O of this one
//   one warp           makes the terms of an item's queries, an item ahead
//   four warps         a thread a key: its scores from tensor memory, its weights, its row of P
// With all that in the same four warps, one after the other, a tile of d 128 took a group 2800 cycles, 930 of them
// for looking up and copying and 700 for issuing products; apart they take 1650, and two groups have one done in 1400, which
// is what HBM gives it.
//
// The maximum that weights are taken against moves only where a score passes it by 7
// (weights up to 2^7 are as exact), and so does the power of two U that the weights are in
// units of: p_j b_j / U is at most 2^8 when U is set and 2^15 ever.  So a tile takes one barrier
// and no reduction over its keys.
//
// Measured (GPU time; the share is of the 6.8 TB/s of a copy): 64 sequences of up to 8192 rows, 32 heads on 8
// of d 128, 494 MB: 82.7 to 83.8 us, 87 to 88 % (the kernels of fa_decode_e4m3.cu: 88.7).  32 of up to 7296, 8 heads of d 256,
// 462 MB: 77.3 us, 88 % (83.5); 32 heads on 8: 79.9 (85.1).

#include "fa_decode.cuh"
#include "fa_e4m3.cuh"

namespace fa {
namespace {

// HP: heads of a group, 1 or 4.
template <int D, int HP>
struct Tile8 {
  static constexpr int kRows = 128;             // keys
  // Of an item's beginning and end, in tiles, with 1, 2, 3 and 4: 64 sequences of up to 8192 rows of d 128 82.9, 83.8, 84.1,
  // 84.8 us; 32 of up to 2048 of d 256 35.0, 32.1, 31.9, 32.5.
  static constexpr int kCost = D == 256 ? 2 : 1;
  // Terms of a number; term t of head h is column t HP + h.
  static constexpr int kTermsQ = 3, kTermsP = 4;
  static constexpr int kN = 16;                 // columns of a product
  static constexpr int kPieces = D / 16;        // of 16 bytes in a row
  static constexpr int kLd = 128;               // bytes between rows, a swizzle's width; d 256 is two halves
  static constexpr int kHalves = D == 256 ? 2 : 1;
  static constexpr int kTileBytes = kHalves * kRows * kLd;       // of K, and of V
  static constexpr int kScales = 2 * kTileBytes;                 // then the rows' scales, of K and of V
  static constexpr int kStageBytes = kScales + 1024;
  static constexpr int kQHalf = kN * kLd;
  static constexpr int kQBytes = kHalves * kQHalf;
  // Two groups hide what one waits for (an item's first and last tile, the issue of products): 64 sequences of up to
  // 8192 rows, 32 heads on 8 of d 128, take 102 us with one of six tiles and 84 with two of three.  Three tiles of d 256 are
  // all there is room for.
  static constexpr int kGroups = D == 256 ? 1 : 2;
  static constexpr int kLoaders = 4 / kGroups;  // warps of a group that copy
  static constexpr int kBlocks32 = 4 / kLoaders;  // blocks of 32 rows that each of them takes
  static constexpr int kStages = 3;
  static constexpr int kThreadsAll = 32 * kGroups * (6 + kLoaders);
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kQ = kRing;              // two items' queries
  static constexpr int kGroupBytes = kQ + 2 * kQBytes;
  static constexpr int kSmem = 1024 + kGroups * kGroupBytes;
  static constexpr int kGroupCols = kN * (2 + kHalves);  // S twice, O
  static constexpr uint32_t kTmem = kGroups * kGroupCols <= 64 ? 64 : 128;
  static_assert(D == 128 || D == 256, "rows of one or two swizzles' width");
  static_assert(HP == 1 || (HP == 4 && kTermsP * HP == kN), "columns and their packing");
  static_assert(kSmem <= 232448 - 4096 && kGroups * kGroupCols <= (int)kTmem && kGroupBytes % 1024 == 0, "shared and tensor memory");
  // where the piece of 16 bytes of a row is, from the beginning of a tile or of the queries' terms (`rows` of a half)
  __device__ static __forceinline__ int place(int row, int piece, int rows = kRows) {
    return piece / 8 * (rows * kLd) + row * kLd + ((piece % 8 ^ (row & 7)) << 4);
  }
};
constexpr uint32_t kSwizzle128 = 2;   // as descriptors name it
constexpr float kStepQ = 32.f, kStepP = 16.f;  // between terms
constexpr float kMostWeight = 32768.f;  // in units of U, ever: e5m2's half step of it, 16 times itself, is below 57344
constexpr float kSetWeight = 256.f;     // and when U is set
constexpr float kMostScore = 7.f;     // above the maximum that weights are taken against

// A group's barriers.
template <class M>
struct Bars {
  uint64_t full[M::kStages], empty[M::kStages];  // a tile's rows are there; read
  uint64_t s_full[2], s_empty[2];                // its S is there; read
  uint64_t p_full[2];                            // its P is there
  // Its O is there.  Two, as a wait names its phase by parity: whoever waits for a tile's O has seen its S or that of the
  // one behind, so that the O of the tile two before is done, which the same barrier was for.
  uint64_t o_done[2];
  uint64_t q_full[2], q_empty[2];                // an item's queries are there; read
  uint64_t drained;                              // every product is done
};

// Shared-memory matrix descriptor of tcgen05: address, leading and stride byte offsets in 16 bytes, version 1, layout.
__device__ __forceinline__ uint64_t matrix(uint32_t at, uint32_t leading, uint32_t stride, uint32_t layout) {
  return (uint64_t)(at >> 4) | (uint64_t)(leading >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | 1ull << 46 |
         (uint64_t)layout << 61;
}
// the same, `bytes` further on: shared memory's addresses leave the field room
__device__ __forceinline__ uint64_t further(uint64_t m, uint32_t bytes) {
  return (m & 0xffffffff00000000ull) | (uint32_t)((uint32_t)m + (bytes >> 4));
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((int)add)
      : "memory");
}
// The first C columns of this thread's row of tensor memory (4, or 16); waits for them.
template <int C>
struct Row {
  uint32_t r[C <= 4 ? 4 : 16];
  __device__ __forceinline__ float operator[](int i) const { return __uint_as_float(r[i]); }
  __device__ __forceinline__ void load(uint32_t at) {
    if constexpr (C <= 4)
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\ttcgen05.wait::ld.sync.aligned;\n"
                   : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                   : "r"(at)
                   : "memory");
    else
      ptx::tmem_ld16(at, r);
  }
};

// Terms added up: head h of HP.
template <int HP, int kTerms, class R>
__device__ __forceinline__ float sum_terms(const R& r, int h, float step) {
  float x = r[(kTerms - 1) * HP + h];
#pragma unroll
  for (int t = kTerms - 2; t >= 0; --t) x = fmaf(x, 1.f / step, r[t * HP + h]);
  return x;
}

// Two numbers of a query, |x| <= 256, as terms: term t's in bits 0-7 and 8-15 of w[t].  fp16 holds the 8 bits
// of a bf16 number down to 2^-17, and what is left after a term exactly; the last term's steps are 2^-19.
template <int kTerms>
__device__ __forceinline__ void cut_query(float x0, float x1, uint32_t (&w)[kTerms]) {
  __half2 x = __floats2half2_rn(x0, x1);
#pragma unroll
  for (int t = 0; t < kTerms; ++t) {
    w[t] = pack_e4m3x2(x);
    if (t + 1 == kTerms) break;
    const uint32_t y = e4m3x2_lo(w[t]);
    x = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&y)), __float2half2_rn(kStepQ));
  }
}

// Two weights, 0 <= x <= kMostWeight, as terms of e5m2, as above.  What is left after the first, at most an eighth of a
// weight's power of two, goes on as a number of fp16: its 11 bits are all that three more terms hold.
template <int kTerms>
__device__ __forceinline__ void cut_weights(float x0, float x1, uint32_t (&w)[kTerms]) {
  w[0] = pack_e5m2x2(x0, x1);
  const float2 first = f16x2_to_float2(e5m2x2(w[0]));
  __half2 x = __floats2half2_rn((x0 - first.x) * kStepP, (x1 - first.y) * kStepP);
#pragma unroll
  for (int t = 1; t < kTerms; ++t) {
    w[t] = pack_e5m2x2(x);
    if (t + 1 == kTerms) break;
    const uint32_t y = e5m2x2(w[t]);
    x = __hmul2(__hsub2(x, *reinterpret_cast<const __half2*>(&y)), __float2half2_rn(kStepP));
  }
}

// Barriers of the 128 threads of a group that have keys.
__device__ __forceinline__ void group_sync(int group) { ptx::bar_sync(1 + group, kThreads); }
__device__ __forceinline__ bool group_or(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(1 + group), "n"(kThreads)
      : "memory");
  return r != 0;
}

// A place in a ring of N barriers and the parity of its use.
template <int N>
struct Turn {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) at = 0, phase ^= 1;
  }
};

// The run of a group: its number, and where it begins and ends; false if it has none.
template <class M>
__device__ __forceinline__ bool run_of_group(const E4m3Params& a, int group, Walk<M::kRows, M::kCost>* walk, int* run) {
  __shared__ int64_t sums[M::kThreadsAll / 32];
  Units<M::kRows, M::kThreadsAll, M::kCost> units(a, sums);
  const Share share = units.share();
  const int first = blockIdx.x * M::kGroups;
  *run = first + group;
  bool some = false;
#pragma unroll 1
  for (int g = 0; g < M::kGroups && first + g < share.runs(); ++g) {
    const int64_t x = share.first(first + g);
    if (g > 0) {
      __syncthreads();  // the last place found has been read
      if (a.S > M::kThreadsAll) units.restart();
    }
    int64_t base;
    const int s = units.find(x, 0, &base);
    if (g == group) {
      Place<M::kRows, M::kCost> at;
      at.set(a, s, base, x);
      walk->begin(a, at, share.first(first + g + 1));
      some = walk->some();
    }
  }
  return some;
}

// ---------------------------------------------------------------- copying
template <class M>
__device__ __forceinline__ void copy_tiles(const E4m3Params& a, Walk<M::kRows, M::kCost> walk, uint32_t ring, Bars<M>* bars, uint32_t (*seen_at)[4],
                                           int loader, const ptx::Waiter& waiter) {
  constexpr int kStages = M::kStages, NB = M::kBlocks32;
  const int lane = threadIdx.x & 31;
  // This lane's row of each block of 32: its page is asked for one tile ahead of the copies.
  int page[NB], scale[NB];
  bool in[NB];
  int64_t off[NB];
  auto look_up = [&](int t) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int j = t * M::kRows + (loader + b * M::kLoaders) * 32 + lane;
      uint32_t r;
      const uint32_t col = a.page_rows.div((uint32_t)j, &r);
      in[b] = j < walk.rows;
      page[b] = in[b] ? a.table[walk.s * a.table_stride + col] : -1;
      off[b] = walk.item * a.ph + (int64_t)r * a.pn;
      scale[b] = walk.item * a.blocks + (int)a.block_rows.div(r);
    }
  };
  const int64_t in_row = (int64_t)(lane / M::kPieces) * a.pn + lane % M::kPieces * 16;
  const bool wide = a.page_rows.d % 16 == 0;
  // Copies of the tile looked up.  Rows that are not there are filled with
  // zeros, and not read.  The pieces of a row go to neighbouring lanes, so that
  // a request takes whole lines.
  auto copy = [&](int st) {
    const uint32_t to = ring + st * M::kStageBytes;
    int64_t from_row[NB], from[NB][2];
    uint32_t seen[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int block = loader + b * M::kLoaders;
      const bool ok = in[b] && page[b] >= 0 && page[b] < a.num_pages;
      if (in[b] && !ok) report_pages(a.status);
      from_row[b] = ok ? page[b] * a.pp + off[b] : 0;
      const int64_t from_scale = ok ? page[b] * a.page_scales + scale[b] : 0;
      seen[b] = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) seen_at[st][block] = seen[b];
      cp_async4(to + M::kScales + (block * 32 + lane) * 4, a.KS + from_scale, ok);
      cp_async4(to + M::kScales + 512 + (block * 32 + lane) * 4, a.VS + from_scale, ok);
      from[b][0] = __shfl_sync(0xffffffffu, from_row[b], 0) + in_row;
      from[b][1] = __shfl_sync(0xffffffffu, from_row[b], 16) + in_row;
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int row0 = (loader + b * M::kLoaders) * 32;
      if (wide && seen[b] == 0xffffffffu) {
        // the rows are all there, 16 on a page at least: two addresses for all of them
#pragma unroll
        for (int i = 0; i < M::kPieces; ++i) {
          const uint32_t place = to + M::place(row0 + (i * 32 + lane) / M::kPieces, lane % M::kPieces);
          const int64_t x = from[b][i >= M::kPieces / 2] + i % (M::kPieces / 2) * (32 / M::kPieces) * a.pn;
          cp_async16(place, a.K + x, true);
          cp_async16(place + M::kTileBytes, a.V + x, true);
        }
      } else {
#pragma unroll
        for (int i = 0; i < M::kPieces; ++i) {
          const int row = (i * 32 + lane) / M::kPieces, piece = (i * 32 + lane) % M::kPieces;
          const int64_t x = __shfl_sync(0xffffffffu, from_row[b], row) + piece * 16;
          const bool on = (seen[b] >> row) & 1;
          const uint32_t place = to + M::place(row0 + row, piece);
          cp_async16(place, a.K + x, on);
          cp_async16(place + M::kTileBytes, a.V + x, on);
        }
      }
    }
    cp_commit();
  };
  // this warp's copies of the oldest tile that is not published are done
  Turn<kStages> done;
  auto publish = [&]() {
    ptx::fence_proxy_async_smem();  // for the tensor core
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bars->full[done.at]));
    done.next();
  };
  look_up(walk.t);
  Turn<kStages> turn;
  int n = 0;
  bool ok = true, more = true;
  while (more) {
    const int count = walk.count, t0 = walk.t;
    for (int i = 0; i < count && ok; ++i, ++n, turn.next()) {
      if (n >= kStages) ok = ptx::warp_wait(ptx::smem_addr(&bars->empty[turn.at]), turn.phase ^ 1, waiter);
      if (!ok) break;
      copy(turn.at);
      if (i + 1 < count)
        look_up(t0 + i + 1);
      else if ((more = walk.next(a)))
        look_up(0);
      if (n > 0) {  // one stays in flight: with more, what follows sees each tile that much later
        cp_wait<1>();
        publish();
      }
    }
    if (!ok) break;
  }
  cp_wait<0>();
  if (ok && n > 0) publish();  // the last
}

// --------------------------------------------------------------- products
// One thread: a warp's votes at every wait made 1650 cycles a tile.
template <class M, int D>
__device__ __forceinline__ void issue_products(const E4m3Params& a, Walk<M::kRows, M::kCost> walk, uint32_t ring, Bars<M>* bars, uint32_t tmem,
                                               const ptx::Waiter& waiter) {
  constexpr int kStages = M::kStages, kN = M::kN;
  constexpr uint32_t kShape = 1u << 4 | (uint32_t)(kN >> 3) << 17 | 8u << 24;  // fp32 sums, n columns, 128 rows
  constexpr uint32_t kWeights = 1u << 15 | 1u << 16 | 1u << 10;                // both operands MN-major, the second of e5m2
  auto bar = [&](uint64_t& b) { return ptx::smem_addr(&b); };
  auto wait = [&](uint64_t& b, uint32_t phase) { return ptx::wait_bounded(bar(b), phase, waiter, true); };
  const uint32_t tO = tmem + 2 * kN;
  const uint64_t keys = matrix(ring, 16, 8 * M::kLd, kSwizzle128), values = matrix(ring + M::kTileBytes, 0, 8 * M::kLd, kSwizzle128);
  const uint64_t queries = matrix(ring + M::kQ, 16, 8 * M::kLd, kSwizzle128);
  const uint64_t weights = matrix(ring, 128, 2048, 0);  // in the place of the keys, which are read by then
  Turn<kStages> turn, before;
  Turn<2> two, two_before, q;
  auto add_values = [&](bool adds) {
    if (!wait(bars->p_full[two_before.at], two_before.phase)) return false;
    ptx::tc_fence_after();
    const uint64_t v = further(values, before.at * M::kStageBytes);
    const uint64_t p = further(weights, before.at * M::kStageBytes);
#pragma unroll
    for (int x = 0; x < M::kHalves; ++x)
#pragma unroll
      for (int k = 0; k < M::kRows / 32; ++k)
        mma_e4m3(tO + x * kN, further(v, x * M::kRows * M::kLd + 32 * M::kLd * k), further(p, 512 * k), kShape | kWeights,
                 k > 0 || adds);
    ptx::tc_commit(bar(bars->empty[before.at]));
    ptx::tc_commit(bar(bars->o_done[two_before.at]));
    before.next();
    two_before.next();
    return true;
  };
  int n = 0;
  bool ok = true, adds = false;  // whether the tile before is not its item's first
  do {
    ok = wait(bars->q_full[q.at], q.phase);
    const uint64_t q_at = further(queries, q.at * M::kQBytes);
    q.next();
    for (int i = 0; i < walk.count && ok; ++i, ++n) {
      // this tile's S goes first, so that it is there when it is asked for, but does not keep back the O of the one before
      const bool late = n > 0 && !ptx::mbar_try_wait(bar(bars->full[turn.at]), turn.phase);
      if (late) ok = add_values(adds);
      ok = ok && wait(bars->full[turn.at], turn.phase);
      if (n >= 2) ok = ok && wait(bars->s_empty[two.at], two.phase ^ 1);
      if (!ok) break;
      ptx::tc_fence_after();
      const uint64_t k_at = further(keys, turn.at * M::kStageBytes);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t half = k / 4, in = k % 4 * 32;
        mma_e4m3(tmem + two.at * kN, further(k_at, half * M::kRows * M::kLd + in), further(q_at, half * M::kQHalf + in), kShape, k > 0);
      }
      ptx::tc_commit(bar(bars->s_full[two.at]));
      turn.next();
      two.next();
      if (n > 0 && !late) ok = add_values(adds);
      adds = i > 0;
    }
  } while (ok && walk.next(a));
  if (ok) add_values(adds);
  // No product may be in flight when tensor memory is given back, also where a wait has run out, whatever its limit was.
  ptx::tc_commit(bar(bars->drained));
  ptx::wait_bounded(bar(bars->drained), 0, {waiter.abort, waiter.status, 1000000000ull}, false);
}

// ---------------------------------------------------------------- queries
// Each item's queries as terms, an item ahead, in units of 1 / *qscales times the softmax scale.
template <class M, int D, int HP>
__device__ __forceinline__ void store_queries(const E4m3Params& a, Walk<M::kRows, M::kCost> at, uint32_t ring, Bars<M>* bars,
                                              float (*qscales)[HP], const ptx::Waiter& waiter) {
  constexpr int kUnits = D / 128;  // of 4 columns of a head, a lane
  const int lane = threadIdx.x & 31;
  for (int n = 0;; ++n) {
    const int to = n & 1;
    if (n >= 2 && !ptx::warp_wait(ptx::smem_addr(&bars->q_empty[to]), ((n >> 1) - 1) & 1, waiter)) return;
    const uint32_t sQ = ring + M::kQ + to * M::kQBytes;
    int heads;
    const int h0 = first_head(a, at.item, 0, &heads);
    uint2 y[HP][kUnits];
#pragma unroll
    for (int h = 0; h < HP; ++h)
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int u = lane + 32 * k;
        y[h][k] = make_uint2(0, 0);
        if (h < heads) y[h][k] = *reinterpret_cast<const uint2*>(a.Q + at.s * a.qs + (int64_t)(h0 + h) * a.qh + u * 8);
      }
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      float e[kUnits][4];
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        e[k][0] = ptx::bf16lo(y[h][k].x), e[k][1] = ptx::bf16hi(y[h][k].x);
        e[k][2] = ptx::bf16lo(y[h][k].y), e[k][3] = ptx::bf16hi(y[h][k].y);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t t = __float_as_uint(e[k][x]) & 0x7fffffffu;
          top = max(top, t < 0x7f800000u ? t : 0u);
        }
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const int x = max((int)(top >> 23), 8) - 7;  // 1 ... 247
      const float by = __uint_as_float((uint32_t)(254 - x) << 23);
      if (lane == 0) qscales[to][h] = __uint_as_float((uint32_t)x << 23) * a.scale2;
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const int u = lane + 32 * k;
#pragma unroll
        for (int x = 0; x < 4; ++x) e[k][x] = isfinite(e[k][x]) ? e[k][x] * by : NAN;
        uint32_t w0[M::kTermsQ], w1[M::kTermsQ];
        cut_query<M::kTermsQ>(e[k][0], e[k][1], w0);
        cut_query<M::kTermsQ>(e[k][2], e[k][3], w1);
#pragma unroll
        for (int t = 0; t < M::kTermsQ; ++t) {
          const uint32_t at4 = sQ + M::place(t * HP + h, u / 4, M::kN) + u % 4 * 4;
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(at4), "r"(__byte_perm(w0[t], w1[t], 0x5410)) : "memory");
        }
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&bars->q_full[to]));
    if (!at.next(a)) return;
  }
}

// ---------------------------------------------------------------- weights
// the largest of a warp's numbers, NaN apart
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

template <class M, int D, int HP>
__device__ __forceinline__ void weigh_tiles(const E4m3Params& a, Walk<M::kRows, M::kCost> walk, int run, int group, uint32_t ring,
                                            Bars<M>* bars, uint32_t (*seen_at)[4], float (*qscales)[HP],
                                            float (*over_warps)[kWarps][HP], uint32_t tmem, const ptx::Waiter& waiter) {
  constexpr int kStages = M::kStages, kTermsQ = M::kTermsQ, kTermsP = M::kTermsP, kN = M::kN, kHalves = M::kHalves;
  auto bar = [&](uint64_t& b) { return ptx::smem_addr(&b); };
  const int thread = threadIdx.x % kThreads, lane = thread & 31, warp = thread >> 5;
  const uint32_t my_row = tmem + ((uint32_t)(warp * 32) << 16), tO = my_row + 2 * kN;
  float m[HP], base[HP], l[HP], qscale[HP];  // all but l are the group's
  // the largest weight that a unit was set for, and kSetWeight / unit; as in fa_decode_e4m3.cu
  float largest[HP], per_unit[HP];
  Turn<kStages> turn;
  Turn<2> two, q;
  // the O of the tile before the one that it is the turn of
  auto wait_o = [&]() { ptx::warp_wait(bar(bars->o_done[two.at ^ 1]), two.at ? two.phase : two.phase ^ 1, waiter); };
  bool first = true;     // item of the run
  do {
    ptx::warp_wait(bar(bars->q_full[q.at]), q.phase, waiter);  // one that ran out stops the tile
    bool unset = true;                                         // a head has no maximum yet
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      m[h] = -INFINITY;
      base[h] = l[h] = 0.f;
      largest[h] = 0.f;
      per_unit[h] = kSetWeight / kLeastUnit;
      qscale[h] = qscales[q.at][h];
    }
    for (int i = 0; i < walk.count; ++i) {
      const int st = turn.at;
      const uint32_t tile = ring + st * M::kStageBytes;
      const bool bad = !ptx::warp_wait2(bar(bars->s_full[two.at]), two.phase, bar(bars->full[st]), turn.phase, waiter);
      ptx::tc_fence_after();
      const bool mine = seen_at[st][warp] >> lane & 1;
      const float ks = lds4(tile + M::kScales + thread * 4), vs = lds4(tile + M::kScales + 512 + thread * 4);
      float x[HP], w[HP], p[HP];
      {
        Row<kTermsQ * HP> r;
        r.load(my_row + two.at * kN);
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(bars->s_empty[two.at]));
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          // the score above the base; the two scales first, as the sum times one of them may be too large or too small
          const float y = fmaf(sum_terms<HP, kTermsQ>(r, h, kStepQ), qscale[h] * ks, -base[h]);
          x[h] = mine ? y : -INFINITY;
        }
      }
      // weights in units of U, as terms: this key's 16 columns of P
      auto store_weights = [&](const float (&w)[HP]) {
        const uint32_t to = tile + thread * 16;
        uint32_t t[kTermsP];
        if constexpr (HP == 1) {
          cut_weights<kTermsP>(w[0], 0.f, t);
          const uint32_t x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(x) : "memory");
        } else {
          uint32_t u[kTermsP];
          cut_weights<kTermsP>(w[0], w[1], t);
          cut_weights<kTermsP>(w[2], w[3], u);
          ptx::st_shared_v4(to, __byte_perm(t[0], u[0], 0x5410), __byte_perm(t[1], u[1], 0x5410),
                            __byte_perm(t[2], u[2], 0x5410), __byte_perm(t[3], u[3], 0x5410));
        }
        ptx::fence_proxy_async_smem();
      };
      bool passed = bad || unset;
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        p[h] = ptx::ex2(x[h]);
        w[h] = p[h] * vs * per_unit[h];
        passed |= x[h] > kMostScore || w[h] > kMostWeight;
      }
      store_weights(w);
      if (group_or(group, passed)) {
        // ---- a score or a weight passed its limit: the maximum and the unit move
        if (i > 0) wait_o();
        ptx::tc_fence_after();
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          x[h] += base[h];
          const float top = warp_max(x[h]);
          if (lane == 0) over_warps[0][warp][h] = top;
        }
        if (group_or(group, *waiter.abort != 0)) return;  // a wait ran out
        unset = false;
        float f[HP];
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          float top = m[h];
#pragma unroll
          for (int k = 0; k < kWarps; ++k) top = fmaxf(top, over_warps[0][k][h]);
          base[h] = base_of(top);
          const float alpha = ptx::ex2(m[h] - base[h]);
          m[h] = top;
          unset |= top == -INFINITY;
          l[h] *= alpha;
          f[h] = alpha * inverse(per_unit[h]);
          largest[h] *= alpha;
          p[h] = ptx::ex2(x[h] - base[h]);
          w[h] = p[h] * vs;
        }
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          const float top = warp_max(w[h]);
          if (lane == 0) over_warps[1][warp][h] = top;
        }
        group_sync(group);
#pragma unroll
        for (int h = 0; h < HP; ++h) {
#pragma unroll
          for (int k = 0; k < kWarps; ++k) largest[h] = fmaxf(largest[h], over_warps[1][k][h]);
          per_unit[h] = kSetWeight * inverse(unit_for(largest[h]));
          f[h] *= per_unit[h];
          w[h] *= per_unit[h];
        }
        if (i > 0) {
#pragma unroll
          for (int x = 0; x < kHalves; ++x) {
            Row<kTermsP * HP> r;
            r.load(tO + x * kN);
#pragma unroll
            for (int c = 0; c < kTermsP * HP; ++c) r.r[c] = __float_as_uint(r[c] * f[c % HP]);
            if constexpr (HP == 1)
              asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(tO + x * kN), "r"(r.r[0]),
                           "r"(r.r[1]), "r"(r.r[2]), "r"(r.r[3])
                           : "memory");
            else
              ptx::tmem_st16(tO + x * kN, r.r);
          }
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
        }
        store_weights(w);
        group_sync(group);
      }
      if (thread == 0) ptx::mbar_arrive(bar(bars->p_full[two.at]));
#pragma unroll
      for (int h = 0; h < HP; ++h) l[h] += p[h];

      turn.next();
      two.next();
    }
      // ---- the item ends here, or goes on in the next group's run
      const bool whole = walk.t == 0 && walk.count == walk.tiles;
      // the part of an item that was being read when the run began is the
      // run's first, any other its second
      const int slot = 2 * run + (first ? 0 : 1);
      first = false;
      int heads;
      const int h0 = first_head(a, walk.item, 0, &heads);
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        float sum = l[h];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) over_warps[2][warp][h] = sum;
      }
      group_sync(group);
      if (thread == 0) ptx::mbar_arrive(bar(bars->q_empty[q.at]));
      q.next();
      wait_o();  // one that ran out stops the next tile
      ptx::tc_fence_after();
      // a thread stores a column
#pragma unroll
      for (int x = 0; x < kHalves; ++x) {
        Row<kTermsP * HP> r;
        r.load(tO + x * kN);
        const int col = x * 128 + thread;
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          if (h >= heads) continue;
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) sum += over_warps[2][k][h];
          float o = sum_terms<HP, kTermsP>(r, h, kStepP) * inverse(per_unit[h]);
          if (whole) {
            const bool none = sum == 0.f;
            o = none ? 0.f : o * (1.f / sum);
            *(reinterpret_cast<__nv_bfloat16*>(a.O + walk.s * a.os + (int64_t)(h0 + h) * a.oh) + col) = __float2bfloat16(o);
            if (col == 0) a.L[(int64_t)walk.s * a.H + h0 + h] = none ? INFINITY : (m[h] + log2f(sum)) * kLn2;
          } else {
            const int64_t to = (int64_t)slot * HP + h;
            a.part_o[to * D + col] = o;
            if (col == 0) a.part_ml[to] = make_float2(m[h], sum);
          }
        }
      }
      ptx::tc_fence_before();
  } while (walk.next(a));
}

template <int D, int HP>
__global__ void __launch_bounds__(Tile8<D, HP>::kThreadsAll, 1) decode_sm103_kernel(const __grid_constant__ E4m3Params a) {
  using M = Tile8<D, HP>;
  extern __shared__ uint8_t dynamic[];
  __shared__ __align__(8) Bars<M> all_bars[M::kGroups];
  __shared__ uint32_t all_seen[M::kGroups][M::kStages][4];
  __shared__ float all_qscales[M::kGroups][2][HP];
  __shared__ float all_over_warps[M::kGroups][3][kWarps][HP];
  __shared__ uint32_t tmem_at;
  __shared__ int abort_flags[M::kGroups];
  const int warp = threadIdx.x >> 5;
  // the warps with keys come first: a warp reaches the 32 rows of tensor memory that its number says
  const bool weighs = warp < 4 * M::kGroups, issues = !weighs && warp < 5 * M::kGroups;
  const bool asks = !weighs && !issues && warp < 6 * M::kGroups;
  const int group = weighs   ? warp / 4
                    : issues ? warp - 4 * M::kGroups
                    : asks   ? warp - 5 * M::kGroups
                             : (warp - 6 * M::kGroups) / M::kLoaders;
  Bars<M>* bars = &all_bars[group];
  Walk<M::kRows, M::kCost> walk = {};
  int run;
  after_stream();
  next_may_start();  // the join
  const bool some = run_of_group<M>(a, group, &walk, &run);
  if (issues && (threadIdx.x & 31) == 0) {
    for (int i = 0; i < M::kStages; ++i) {
      ptx::mbar_init(ptx::smem_addr(&bars->full[i]), M::kLoaders);
      ptx::mbar_init(ptx::smem_addr(&bars->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_addr(&bars->s_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->s_empty[i]), kThreads);
      ptx::mbar_init(ptx::smem_addr(&bars->p_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->o_done[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->q_full[i]), 1);
      ptx::mbar_init(ptx::smem_addr(&bars->q_empty[i]), 1);
    }
    ptx::mbar_init(ptx::smem_addr(&bars->drained), 1);
    abort_flags[group] = 0;
    ptx::fence_mbar_init();
  }
  // Not before after_stream(): a block that is here before the kernel in front has ended
  // must not hold tensor memory which one of that has still to ask for.
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_addr(&tmem_at), M::kTmem);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t ring = ((ptx::smem_addr(dynamic) + 1023u) & ~1023u) + group * M::kGroupBytes;
  const uint32_t tmem = tmem_at + group * M::kGroupCols;
  const ptx::Waiter waiter{&abort_flags[group], a.status, a.wait_ns};
  if (some) {
    if (weighs) {
      weigh_tiles<M, D, HP>(a, walk, run, group, ring, bars, all_seen[group], all_qscales[group], all_over_warps[group], tmem,
                            waiter);
    } else if (issues) {
      if ((threadIdx.x & 31) == 0) issue_products<M, D>(a, walk, ring, bars, tmem, waiter);
      __syncwarp();
    } else if (asks) {
      store_queries<M, D, HP>(a, walk, ring, bars, all_qscales[group], waiter);
    } else {
      copy_tiles<M>(a, walk, ring, bars, all_seen[group], (warp - 6 * M::kGroups) % M::kLoaders, waiter);
    }
    ptx::tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_at, M::kTmem);
  }
}

template <int D, int HP>
cudaError_t launch(const Cut& k, E4m3Params a, cudaStream_t s) {
  using M = Tile8<D, HP>;
  static std::atomic<int> known[64];
  int resident = 0;
  a.cluster = 0;
  const auto kernel = decode_sm103_kernel<D, HP>;
  cudaError_t e = resident_blocks((const void*)kernel, M::kSmem, known, &resident, M::kThreadsAll);
  if (e != cudaSuccess) return e;
  const int runs = runs_of(k, resident * M::kGroups, &a);
  e = launch_early(kernel, dim3((unsigned)ceil_div(runs, M::kGroups)), M::kThreadsAll, M::kSmem, s, 1, a);
  if (e != cudaSuccess) return e;
  return launch_join<__nv_bfloat16, D, M::kRows, M::kCost>(k, a, runs, s);
}

}  // namespace

// What the table can hold decides, as the lengths are not known here.  By tiles that a group has if it is full (128 rows; 304 groups
// of d 128, 152 of d 256), 32 sequences, half full on average, the kernels of fa_decode_e4m3.cu against these, in us:
//   d 128, 1 head a key head:  32: 34.3, 35.9   48: 45.0, 45.9   64: 58.3, 57.4   96: 81.4, 77.8
//   d 128, 4 heads:            32: 34.6, 37.2   48: 45.5, 47.1   64: 58.9, 58.5   96: 85.6, 79.0
//   d 256, 1 head:             24: 29.1, 28.5   32: 35.0, 34.6   48: 47.0, 44.9   96: 83.5, 77.3
//   d 256, 4 heads:            24: 29.6, 31.4   32: 36.2, 37.3   48: 48.2, 47.4   96: 85.1, 79.9
// 8 sequences that fill it: d 128 with 1 head, 16: 33.3, 33.8, 32: 58.2, 57.0; d 256 with 4, 12: 29.1, 31.0, 16: 35.7, 36.1,
// 32: 61.8, 58.6.  d 96 gains nothing at any size, d 64 and 32 and eight heads or more lose.
bool takes_sm103(const fa_cache& c, int H) {
  const int64_t tiles = (int64_t)c.S * c.H_kv * cache_rows(c) / 128;
  return c.dtype == FA_BF16 && H / c.H_kv <= 4 && ((c.d == 128 && tiles >= 304 * 56) || (c.d == 256 && tiles >= 152 * 40));
}

Cut cut_e4m3_sm103(const fa_cache& c, int H) {
  Cut k = pieces_of(H / c.H_kv, 4);  // one: takes_sm103
  k.part_heads = k.piece_heads == 1 ? 1 : 4;
  k.cost = c.d == 256 ? Tile8<256, 4>::kCost : Tile8<128, 4>::kCost;
  k.most_tiles = ceil_div(cache_rows(c), 128);
  k.tiles = (int64_t)c.S * c.H_kv * k.most_tiles;
  k.cluster = 0;
  return k;
}

cudaError_t launch_e4m3_sm103(int d, const Cut& k, const E4m3Params& a, cudaStream_t s) {
  const bool one = k.part_heads == 1;
  switch (d) {
    case 128: return one ? launch<128, 1>(k, a, s) : launch<128, 4>(k, a, s);
    case 256: return one ? launch<256, 1>(k, a, s) : launch<256, 4>(k, a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
