// Attention of one new token over a paged key-value cache in 8 bits
// (fa_decode_e4m3): k_j and v_j are stored numbers times the scales of their
// blocks, a_j and b_j,
//   s_j = scale a_j q . k_j,  m = max_j s_j,  l = sum_j 2^(s_j - m),
//   O = sum_j 2^(s_j - m) b_j v_j / l,  L = (m + log2 l) ln 2
// with scores in units of log 2 (the scale carries log2 e).
//
// Half the bytes of a bf16 cache for the same products: a row and head are 2 d
// bytes against 4 d flops a query head.  HBM should be the bound, but the instructions
// for every byte are twice as many, so here the design is about those as
// well.  How the work is shared out and joined is in fa_decode.cuh; large problems
// with d 128 and 256 and few heads are those of fa_decode_e4m3_sm103.cu.
//
// Measured (GPU time; the share is of the 6.8 TB/s of a copy): 32 sequences of up to 2048 rows, 32 heads of d 64, 118 MB:
// 32.3 us, 54 %.  125 MB of 32 sequences and 8 key heads with 4 heads a key head: d 128 29.6 us, 62 %, d 96 (145 MB) 34.6,
// 62 %, d 32 41.0, 45 %; with 16: d 128 39.8, d 256 47.2; in fp32 with 8: d 64 31.5, d 128 31.5.  About 8 us of each are the
// start of a call, the last tiles and the join, whatever the size; the smallest call takes 3.4.  A warp's instructions for 4 KB are 450
// at d 128 and 570 at d 64, half of the issue slots: fixed latencies, on three to four warps a scheduler,
// bound the rest (16 instructions fewer a tile, without the mask, gained 1 %; a barrier fewer an item nothing).

#include "fa_decode.cuh"
#include "fa_e4m3.cuh"

namespace fa {
namespace {

// A warp takes 16 kSub rows of each tile with mma.m16n8k16 in fp16, into which
// e4m3 numbers go exactly, two at a time:
//
//  S = Q K^T     A = 16 query heads x 16 columns, B = 16 columns x 8 keys.  The
//                columns of a step are those that make a lane's share of B four
//                bytes of a key, so that a run of 16 bytes serves four steps.
//  O^T += V^T P^T  A = 16 columns x 16 keys, B = 16 keys x 8 heads: S's accumulators
//                are P^T's operand as they stand.  ldmatrix turns V round by pairs of
//                bytes: a lane gets columns 2 i and 2 i + 1 of two keys, a byte
//                permute makes the two columns' pairs, and the 16 columns of a step are
//                the even ones and then the odd ones of 16.
//
// Queries: a head's are multiplied by the power of two that takes the largest to
// 2^14 ... 2^15, so that bf16 ones are fp16 numbers exactly, down to 2^-28 of the
// largest.  fp32 ones become the sum of two, the second 2^11 times itself: it takes
// the place of a second group of 8 heads, at no more products.
//
// Weights: P b_j / U, U a power of two, as the sum of two fp16 numbers: off by at most 2^-22 of the weight or, if that is
// more, 2^-25, where the largest is 2^10 or more: 2^-35 of the largest.  So the rounding of O is the only one to fewer
// than 16 bits, as in fa_decode.  One number for bf16, 11 bits, takes 31.2 us for 32.2 (32 sequences of up to 2048 rows,
// 32 heads of d 64) and, with 16 heads a key head of d 128, 107 for 116 (64 of up to 8192), but where values cancel it
// loses bits that O has.  The maximum that weights are taken against and U are moved only when a score passes the one by 7
// or a weight 2^15, so that almost every tile does without the maximum over its lanes and without a look at the
// accumulators.
template <int D, int NH, bool kF32>
struct Mma8 {
  static constexpr int kSub = D <= 64 ? 2 : 1;
  static constexpr int kRows = 16 * kSub;       // of a tile, a warp
  static constexpr int kTile = kWarps * kRows;
  // Of an item's beginning and end, in tiles: queries to turn into fragments and a sum over the block cost as much as 256
  // rows.  With 128, 256, 384 and 512, sequences of up to some thousand rows, 8 key heads, us: d 64, 8 heads a key head
  // 31.7, 30.7, 31.6, 32.0; d 96, 4: 34.0, 34.5, 35.1, 36.1; d 128, 8: 30.6, 30.2, 31.1, 31.9; d 128, 32: 70.1, 65.5, 67.4,
  // 68.1; d 256, 16: 55.9, 47.2, 45.5, 46.9.  One tile, as for rows of 16 bits: 31.7, 35.6, 33.3, 78.4, 71.4.
  static constexpr int kCost = 256 / kTile;
  static constexpr int kRun = D % 64 == 0 ? 16 : D % 32 == 0 ? 8 : 4;  // bytes of a key that a lane reads at a time
  static constexpr int kRuns = D / (4 * kRun);
  static constexpr int kPieces = D / 16;        // of 16 bytes in a row
  // K: an access's lanes take 128 bytes of different banks: 8 rows of 16, 4 of 32 (or of 32 out
  // of 96), 2 of 64, or of rows of 128 and more, 16 more apart, every second piece of two.
  static constexpr int kPitchK = D >= 128 ? D + 16 : D;
  // V: 8 rows' pieces of 16 bytes
  static constexpr int kPitchV = D == 16 ? 16 : D + 16;
  static constexpr int kScales = kRows * (kPitchK + kPitchV);  // then the scales of K and V, and which rows are there
  static constexpr int kSeen = kScales + kRows * 8;
  static constexpr int kStageBytes = kSeen + 16;
  // Blocks an SM, and tiles in flight.  d 64 with 4 and 2 instead of 3 and 3: 33.5 -> 31.0 us (32 sequences of up to 2048
  // rows, 32 heads); d 32 with 5 blocks instead of 4 spills: 39.1 -> 43.1; d 256 with 4 tiles instead of 3, one block: 72.4
  // -> 96.7 (16 heads on one); d 128 gains nothing from 4 and 2.
  static constexpr int kBlocks = D == 16 ? 5 : D == 32 ? 4 : D == 64 ? 4 : D == 256 ? 2 : 3;
  static constexpr int kStages = D == 16 ? 5 : D == 96 ? 4 : D == 64 ? 2 : 3;
  static constexpr int kVW = D % 64 || D == 256 ? (D == 16 ? 16 : 32) : 64;  // columns of O that are exchanged at a time
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kPad = kVW + 4;          // floats of a row of the exchange buffer
  static constexpr int kSmem = kRing + kWarps * 8 * kPad * 4;
  static_assert(!kF32 || NH == 1, "fp32 queries take both groups of heads");
  static_assert(kStageBytes % 16 == 0 && kScales % 16 == 0, "copies of 16 bytes");
  // where lane q's c-th run of a key begins
  __device__ static constexpr int run_at(int c, int q) {
    return D >= 128 ? (8 * (c / 2) + 2 * q + c % 2) * 16 : (4 * c + q) * kRun;
  }
};
constexpr float kMostScore = 7.f;  // above the maximum that weights are taken against
// Of a weight when U is set, and ever: as far up as fp16 reaches, for the sake of the small ones, but for some room to grow.
// With 2^8, after which U moves less often, calls are 0 to 1 % quicker, and weights reach less far down by 2^3.
constexpr float kTopWeight = 2048.f, kMostWeight = 32768.f;

__device__ __forceinline__ void mma16816_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_trans2(uint32_t at, uint32_t& a, uint32_t& b) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(at));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 lds8(uint32_t a) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
// A warp's copies of its rows of each tile and of their scales, ahead of their use.
template <class M>
struct Loader8 {
  static constexpr int kRows = M::kRows, kStages = M::kStages;
  // rows that a warp's request takes, and whether it takes a part of 16 rows
  static constexpr int kRequest = 32 / M::kPieces;
  static constexpr bool kWhole = 32 % M::kPieces == 0 && kRequest <= 16;
  const E4m3Params& a;
  Walk<M::kTile, M::kCost> walk;  // the item that is copied next,
  int i = 0;            // the tile of it,
  bool more;            // if there is one
  const uint32_t ring;  // of this warp
  const int piece;      // of the query heads
  const bool wide;      // 16 rows are on a page
  const int64_t in_row; // of this lane's piece, from the first row of its requests
  // The row that this lane looks up in that tile: its page is asked for one
  // tile ahead of the copies that need it.
  int page = -1;
  bool in = false;
  int64_t off = 0;
  int scale = 0;  // of the page's

  __device__ __forceinline__ Loader8(const E4m3Params& p, const Walk<M::kTile, M::kCost>& w, uint32_t r, int h)
      : a(p), walk(w), more(w.some()), ring(r), piece(h), wide(kWhole && p.page_rows.d % 16 == 0),
        in_row((int64_t)((threadIdx.x & 31) / M::kPieces) * p.pn + (threadIdx.x & 31) % M::kPieces * 16) {
    if (more) look_up();
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) produce(k);
  }
  __device__ __forceinline__ void look_up() {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = (walk.t + i) * M::kTile + warp * kRows + (lane & (kRows - 1));
    uint32_t r;
    const uint32_t col = a.page_rows.div((uint32_t)j, &r);
    in = j < walk.rows;
    page = in ? a.table[walk.s * a.table_stride + col] : -1;
    off = walk.item * a.ph + (int64_t)r * a.pn;
    scale = walk.item * a.blocks + (int)a.block_rows.div(r);
    if (i == 0) {  // a new item: its queries into L1
      int heads;
      const char* row = a.Q + walk.s * a.qs + (int64_t)first_head(a, walk.item, piece, &heads) * a.qh;
      constexpr int kLines = (M::kPieces * 32 + 127) / 128;
      for (int k = lane; k < heads * kLines; k += 32) prefetch_l1(row + (k / kLines) * a.qh + (k % kLines) * 128);
    }
  }
  // Copies of the tile looked up, into stage st.  Rows that are not there are
  // filled with zeros, and not read.  The pieces of a row go to neighbouring
  // lanes, so that a request takes whole lines.
  __device__ __forceinline__ uint32_t copy(uint32_t to) {
    const int lane = threadIdx.x & 31;
    const bool ok = in && page >= 0 && page < a.num_pages;
    if (in && !ok) report_pages(a.status);
    const int64_t from_row = ok ? page * a.pp + off : 0;
    const int64_t from_scale = ok ? page * a.page_scales + scale : 0;
    const uint32_t seen = __ballot_sync(0xffffffffu, ok);
    const uint32_t scales_to = to + M::kScales;
    if constexpr (kRows == 32) {
      cp_async4(scales_to + lane * 4, a.KS + from_scale, ok);
      cp_async4(scales_to + (32 + lane) * 4, a.VS + from_scale, ok);
    } else {
      cp_async4(scales_to + lane * 4, (lane < 16 ? a.KS : a.VS) + from_scale, ok);
    }
    if (kWhole && wide && seen == 0xffffffffu) {
      // the rows are all there, and 16 of them on a page: an address for each 16
#pragma unroll
      for (int h = 0; h < kRows / 16; ++h) {
        const int64_t from = __shfl_sync(0xffffffffu, from_row, 16 * h) + in_row;
#pragma unroll
        for (int k = 0; k < 16 / kRequest; ++k) {
          const int row = 16 * h + k * kRequest;
          const uint32_t in_k = to + (row + lane / M::kPieces) * M::kPitchK + lane % M::kPieces * 16;
          const uint32_t in_v = to + kRows * M::kPitchK + (row + lane / M::kPieces) * M::kPitchV + lane % M::kPieces * 16;
          const int64_t x = from + k * kRequest * a.pn;
          cp_async16(in_k, a.K + x, true);
          cp_async16(in_v, a.V + x, true);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < kRows * M::kPieces / 32; ++k) {
        const int row = (k * 32 + lane) / M::kPieces, at = (k * 32 + lane) % M::kPieces;
        const int64_t from = __shfl_sync(0xffffffffu, from_row, row) + at * 16;
        const bool on = (seen >> row) & 1;
        cp_async16(to + row * M::kPitchK + at * 16, a.K + from, on);
        cp_async16(to + kRows * M::kPitchK + row * M::kPitchV + at * 16, a.V + from, on);
      }
    }
    return kRows == 32 ? seen : seen & 0xffffu;
  }
  __device__ __forceinline__ void produce(int st) {
    const uint32_t to = ring + st * M::kStageBytes;
    uint32_t seen = 0;
    if (more) {
      seen = copy(to);
      if (++i == walk.count) {
        i = 0;
        more = walk.next(a);
      }
      if (more) look_up();
    }
    if ((threadIdx.x & 31) == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + M::kSeen), "r"(seen) : "memory");
    cp_commit();
  }
  // Waits for the oldest tile in flight, in stage st, asks for another, and
  // returns which rows of it are there.
  __device__ __forceinline__ uint32_t next(int st) {
    cp_wait<kStages - 2>();
    __syncwarp();  // the warp's copies are all there, and its reads of the stage refilled next are done
    uint32_t seen;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(seen) : "r"(ring + st * M::kStageBytes + M::kSeen) : "memory");
    produce(st == 0 ? kStages - 1 : st - 1);
    return seen;
  }
};

// A lane's share of a head's queries as fp16 operands: columns 4 c + 0, 1 and 2, 3
// of its runs, in units of *unit.
template <class M, class T>
struct Columns {
  static constexpr int kWords = M::kRun / 4;  // steps of a run
  float x[M::kRuns][kWords][4];
  __device__ __forceinline__ void load(const char* row, int q) {
#pragma unroll
    for (int c = 0; c < M::kRuns; ++c)
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const char* p = row + (M::run_at(c, q) + 4 * w) * (int)sizeof(T);
        if constexpr (sizeof(T) == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          x[c][w][0] = ptx::bf16lo(v.x), x[c][w][1] = ptx::bf16hi(v.x);
          x[c][w][2] = ptx::bf16lo(v.y), x[c][w][3] = ptx::bf16hi(v.y);
        } else {
          const float4 v = *reinterpret_cast<const float4*>(p);
          x[c][w][0] = v.x, x[c][w][1] = v.y, x[c][w][2] = v.z, x[c][w][3] = v.w;
        }
      }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int c = 0; c < M::kRuns; ++c)
#pragma unroll
      for (int w = 0; w < kWords; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[c][w][e] = 0.f;
  }
  // Takes the head's largest value to 2^14 ... 2^15; returns what the products are to be multiplied by.  With one that is not
  // finite all become NaN: an infinity could make all scores -inf, as if there were no rows.
  __device__ __forceinline__ float normalise() {
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < M::kRuns; ++c)
#pragma unroll
      for (int w = 0; w < kWords; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[c][w][e]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = max((int)(top >> 23), 15) - 14;  // 1 ... 240
    const float by = top < 0x7f800000u ? __uint_as_float((uint32_t)(254 - e) << 23) : NAN;
#pragma unroll
    for (int c = 0; c < M::kRuns; ++c)
#pragma unroll
      for (int w = 0; w < kWords; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[c][w][i] *= by;
    return __uint_as_float((uint32_t)e << 23);
  }
};

// kAlone: a cluster an item, joined here; else a block a run.
template <int D, int NH, bool kF32, bool kAlone>
__global__ void __launch_bounds__(kThreads, Mma8<D, NH, kF32>::kBlocks)
    decode_e4m3_kernel(const __grid_constant__ E4m3Params a) {
  using M = Mma8<D, NH, kF32>;
  using T = std::conditional_t<kF32, float, __nv_bfloat16>;
  constexpr int kTile = M::kTile, kStages = M::kStages, VW = M::kVW, kSub = M::kSub, kWords = M::kRun / 4;
  constexpr int kHeads = 8 * NH;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 ml[kWarps][kHeads];
  __shared__ float units[kWarps][kHeads];
  __shared__ float2 part_ml[kHeads];  // kAlone: this block's part, with o in part_o
  float4* part_o = reinterpret_cast<float4*>(smem);  // over the ring, which is read by then
  Place<kTile, M::kCost> at;
  int64_t end;
  bool some;
  after_stream();
  if constexpr (kAlone) {
    some = share_of_item(a, &at, &end);
    if (!some && threadIdx.x < kHeads) part_ml[threadIdx.x] = make_float2(-INFINITY, kNoPart);
  } else {
    next_may_start();  // the join
    some = run_of(a, &at, &end);
    if (!some) return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int piece = (kAlone ? blockIdx.x / a.cluster : blockIdx.x) % a.split;
  const uint32_t ring = ptx::smem_addr(smem) + warp * kStages * M::kStageBytes;
  float* exchange = reinterpret_cast<float*>(smem + M::kRing);
  Walk<kTile, M::kCost> walk;
  walk.begin(a, at, end);
  Loader8<M> load(a, walk, ring, piece);

  uint32_t qf[M::kRuns][kWords][2 * (kF32 ? 2 : NH)];
  float qscale[NH];
  float acc[NH][M::kPieces][4];  // O^T, unnormalised, in units of unit / kTopWeight: columns 2 g, 2 g + 1 of 16, heads 2 q, 2 q + 1
  float m[NH], l[NH];  // of heads g, g + 8; l of this lane's keys alone
  // the largest weight that a unit was set for, and kTopWeight / unit.  Where the maximum moves the largest goes down by
  // what the weights do, not in powers of two: else a unit stays up when its row is long of no account
  float largest[NH], per_unit[NH];
  int stage = 0;
  bool first = true;             // item of the run
  if (some) do {
    {
      int heads;
      const int h0 = first_head(a, walk.item, piece, &heads);
      const char* row = a.Q + walk.s * a.qs + (int64_t)h0 * a.qh;
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        Columns<M, T> x;
        if (g + 8 * u < heads)
          x.load(row + (g + 8 * u) * a.qh, q);
        else
          x.zero();
        qscale[u] = x.normalise() * a.scale2;
#pragma unroll
        for (int c = 0; c < M::kRuns; ++c)
#pragma unroll
          for (int w = 0; w < kWords; ++w)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float x0 = x.x[c][w][2 * e], x1 = x.x[c][w][2 * e + 1];
              const uint32_t y = pack_f16x2(x0, x1);
              qf[c][w][2 * u + e] = y;
              if constexpr (kF32) {  // what is left, 2^11 times itself
                const float2 z = f16x2_to_float2(y);
                qf[c][w][2 + e] = pack_f16x2((x0 - z.x) * 2048.f, (x1 - z.y) * 2048.f);
              }
            }
        m[u] = -INFINITY;
        l[u] = 0.f;
        largest[u] = 0.f;
        per_unit[u] = kTopWeight / kLeastUnit;
#pragma unroll
        for (int p = 0; p < M::kPieces; ++p)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[u][p][x] = 0.f;
      }
    }

    for (int i = 0; i < walk.count; ++i) {
      const uint32_t seen = load.next(stage);
      if (seen) {
        const uint32_t tile = ring + stage * M::kStageBytes;
        float s[2 * kSub][4];
#pragma unroll
        for (int o = 0; o < 2 * kSub; ++o) {  // 8 keys
          s[o][0] = s[o][1] = s[o][2] = s[o][3] = 0.f;
#pragma unroll
          for (int c = 0; c < M::kRuns; ++c) {
            const uint32_t from = tile + (8 * o + g) * M::kPitchK + M::run_at(c, q);
            uint32_t k[4];
            if constexpr (M::kRun == 16) {
              const uint4 v = lds16(from);
              k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
            } else if constexpr (M::kRun == 8) {
              const float2 v = lds8(from);
              k[0] = __float_as_uint(v.x), k[1] = __float_as_uint(v.y);
            } else {
              asm volatile("ld.shared.u32 %0, [%1];" : "=r"(k[0]) : "r"(from));
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              constexpr bool kBoth = NH > 1 || kF32;
              mma16816_f16(s[o], qf[c][w][0], kBoth ? qf[c][w][kBoth ? 2 : 0] : 0u, qf[c][w][1],
                           kBoth ? qf[c][w][kBoth ? 3 : 0] : 0u, e4m3x2_lo(k[w]), e4m3x2_hi(k[w]));
            }
          }
        }
        // keys 8 o + 2 q, 8 o + 2 q + 1 of the warp's
        float2 ks[2 * kSub], vs[2 * kSub];
#pragma unroll
        for (int o = 0; o < 2 * kSub; ++o) {
          ks[o] = lds8(tile + M::kScales + (8 * o + 2 * q) * 4);
          vs[o] = lds8(tile + M::kScales + (M::kRows + 8 * o + 2 * q) * 4);
        }
        const uint32_t mine = seen >> (2 * q);
        float x[NH][2 * kSub][2], p[NH][2 * kSub][2], w[NH][2 * kSub][2];
        bool passed = false;
#pragma unroll
        for (int u = 0; u < NH; ++u) {
          const float base = base_of(m[u]);
          float top = -INFINITY, most = 0.f;
#pragma unroll
          for (int o = 0; o < 2 * kSub; ++o)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float dot = kF32 ? fmaf(s[o][2 + e], 1.f / 2048.f, s[o][e]) : s[o][2 * u + e];
              // the two scales first, as the product with one of them may be too large or too small
              const float y = dot * (qscale[u] * (e ? ks[o].y : ks[o].x));
              x[u][o][e] = mine >> (8 * o + e) & 1 ? y : -INFINITY;
              top = fmaxf(top, x[u][o][e]);
              p[u][o][e] = ptx::ex2(x[u][o][e] - base);
              w[u][o][e] = p[u][o][e] * (e ? vs[o].y : vs[o].x);
              most = fmaxf(most, w[u][o][e]);
            }
          passed |= top > m[u] + kMostScore || most * per_unit[u] > kMostWeight;
        }
        if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
          for (int u = 0; u < NH; ++u) {
            float top = m[u], most = 0.f;
#pragma unroll
            for (int o = 0; o < 2 * kSub; ++o) top = fmaxf(top, fmaxf(x[u][o][0], x[u][o][1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float base = base_of(top), alpha = ptx::ex2(m[u] - base);
            m[u] = top;
            l[u] *= alpha;
#pragma unroll
            for (int o = 0; o < 2 * kSub; ++o)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                p[u][o][e] = ptx::ex2(x[u][o][e] - base);
                w[u][o][e] = p[u][o][e] * (e ? vs[o].y : vs[o].x);
                most = fmaxf(most, w[u][o][e]);
              }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            largest[u] = fmaxf(most, alpha * largest[u]);
            const float old = alpha * inverse(per_unit[u]);
            per_unit[u] = kTopWeight * inverse(unit_for(largest[u]));
            const float f = old * per_unit[u];
            // the factors belong to heads g, the accumulators to heads 2q, 2q + 1
            const float f0 = __shfl_sync(0xffffffffu, f, 8 * q), f1 = __shfl_sync(0xffffffffu, f, 8 * q + 4);
#pragma unroll
            for (int c = 0; c < M::kPieces; ++c) {
              acc[u][c][0] *= f0, acc[u][c][2] *= f0;
              acc[u][c][1] *= f1, acc[u][c][3] *= f1;
            }
          }
        }
        uint32_t hi[NH][2 * kSub], lo[NH][2 * kSub];
#pragma unroll
        for (int u = 0; u < NH; ++u)
#pragma unroll
          for (int o = 0; o < 2 * kSub; ++o) {
            l[u] += p[u][o][0] + p[u][o][1];
            const float w0 = w[u][o][0] * per_unit[u], w1 = w[u][o][1] * per_unit[u];
            hi[u][o] = pack_f16x2(w0, w1);
            const float2 z = f16x2_to_float2(hi[u][o]);
            lo[u][o] = pack_f16x2(w0 - z.x, w1 - z.y);
          }
        // V: pieces of 8 keys x 8 pairs of columns; lane 8 n + r names row r of piece n
        const uint32_t v_at = tile + M::kRows * M::kPitchK + ((lane & 7) + (lane >> 3 & 1) * 8) * M::kPitchV + (lane >> 4) * 16;
#pragma unroll
        for (int b = 0; b < kSub; ++b)
#pragma unroll
          for (int c = 0; c < M::kPieces; c += 2) {
            constexpr int kTwo = M::kPieces > 1 ? 2 : 1;
            uint32_t r[4];
            const uint32_t from = v_at + 16 * b * M::kPitchV + c * 16;
            if constexpr (kTwo == 2)
              ldmatrix_trans(from, r[0], r[1], r[2], r[3]);
            else
              ldmatrix_trans2(from, r[0], r[1]);
#pragma unroll
            for (int i = 0; i < kTwo; ++i) {
              const uint32_t v0 = __byte_perm(r[2 * i], 0, 0x3120), v1 = __byte_perm(r[2 * i + 1], 0, 0x3120);
              const uint32_t a0 = e4m3x2_lo(v0), a1 = e4m3x2_hi(v0), a2 = e4m3x2_lo(v1), a3 = e4m3x2_hi(v1);
#pragma unroll
              for (int u = 0; u < NH; ++u) {
                mma16816_f16(acc[u][c + i], a0, a1, a2, a3, hi[u][2 * b], hi[u][2 * b + 1]);
                mma16816_f16(acc[u][c + i], a0, a1, a2, a3, lo[u][2 * b], lo[u][2 * b + 1]);
              }
            }
          }
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    {
      // ---- the item ends here, or goes on in the next block's run
      const bool whole = walk.t == 0 && walk.count == walk.tiles && !(kAlone && a.cluster > 1);
      // the part of an item that was being read when the run began is the
      // block's first, any other its second
      const int slot = (2 * (blockIdx.x / a.split) + (first ? 0 : 1)) * a.split + piece;
      first = false;
      int heads;
      const int h0 = first_head(a, walk.item, piece, &heads);
      __syncthreads();  // ml, units and the exchange buffer have been read
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if (q == 0) {
          ml[warp][g + 8 * u] = make_float2(m[u], l[u]);
          units[warp][g + 8 * u] = inverse(per_unit[u]);
        }
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        // this warp's factor of heads 2q, 2q + 1
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int head = 8 * u + 2 * q + e;
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k][head].x);
          f[e] = ptx::ex2(ml[warp][head].x - base_of(top)) * units[warp][head];
        }
#pragma unroll
        for (int c = 0; c < D / VW; ++c) {
          if (u + c > 0) __syncthreads();
          float* mine_at = exchange + (warp * 8 + 2 * q) * M::kPad + 2 * g;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < VW / 16; ++i) {
              const float* o = acc[u][c * (VW / 16) + i];
              *reinterpret_cast<float2*>(mine_at + e * M::kPad + 16 * i) = make_float2(o[e] * f[e], o[2 + e] * f[e]);
            }
          __syncthreads();
          // a thread adds up four columns of a head
#pragma unroll
          for (int k0 = 0; k0 < 2 * VW; k0 += kThreads) {
            const int k = k0 + threadIdx.x, in8 = k / (VW / 4), col = c * VW + k % (VW / 4) * 4, head = 8 * u + in8;
            if (in8 >= 8 || head >= heads) continue;
            float top = -INFINITY, sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k][head].x);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
              sum += ml[k][head].y * ptx::ex2(ml[k][head].x - base_of(top));
              const float4 y = *reinterpret_cast<const float4*>(exchange + (k * 8 + in8) * M::kPad + col - c * VW);
              o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
            }
            if (whole) {
              const bool none = sum == 0.f;
              const float inv = none ? 0.f : 1.f / sum;
              o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
              store4<T>(a.O + walk.s * a.os + (int64_t)(h0 + head) * a.oh, col, o);
              if (col == 0) a.L[(int64_t)walk.s * a.H + h0 + head] = none ? INFINITY : (top + log2f(sum)) * kLn2;
            } else if (kAlone) {
              part_o[(head * D + col) / 4] = o;
              if (col == 0) part_ml[head] = make_float2(top, sum);
            } else {
              const int64_t p = (int64_t)slot * kHeads + head;
              *reinterpret_cast<float4*>(a.part_o + p * D + col) = o;
              if (col == 0) a.part_ml[p] = make_float2(top, sum);
            }
          }
        }
      }
    }
  } while (walk.next(a));
  if (kAlone && a.cluster > 1) join_cluster<T, D>(a, part_o, part_ml);
}

template <int D, int NH, bool kF32>
cudaError_t launch(const Cut& k, const E4m3Params& a, cudaStream_t s) {
  using M = Mma8<D, NH, kF32>;
  using T = std::conditional_t<kF32, float, __nv_bfloat16>;
  static std::atomic<int> known[64], known_alone[64];
  return launch_decode<T, D, M::kTile, M::kCost>(k, a, decode_e4m3_kernel<D, NH, kF32, false>,
                                                   decode_e4m3_kernel<D, NH, kF32, true>, M::kSmem, known, known_alone, s);
}

template <int D>
cudaError_t launch_d(const fa_cache& c, const Cut& k, const E4m3Params& a, cudaStream_t s) {
  if (c.dtype == FA_FP32) return launch<D, 1, true>(k, a, s);
  if constexpr (D > 16) return k.part_heads == 8 ? launch<D, 1, false>(k, a, s) : launch<D, 2, false>(k, a, s);
  return cudaErrorInvalidValue;
}

// Clusters of 16 blocks get two tiles a block at most, of 2 to 8 six, blocks alone twelve: then the runs and the join are
// quicker.  Clusters against runs, 8 key heads and 4 heads a key head, all sequences of the table's size, us:
//   16 blocks, 3 tiles:  d 64 10.1, 10.1  d 96 9.6, 9.9    d 128 10.6, 9.8   fp32 of d 128 10.8, 10.2
//   8 blocks, 6 tiles:   d 64 11.9, 12.9  d 96 10.6, 12.2  d 128 11.5, 12.5  d 256, 4 blocks: 16.6, 18.7
//             8:         d 64 14.3, 14.5  d 96 12.2, 13.2  d 128 13.7, 14.1                   19.0, 21.0
//   1 block, 12 tiles:   d 64 17.3, 18.6  d 96 13.9, 16.1  d 128 15.4, 18.6  d 256 22.7, 27.0
// and of all sizes up to it:
//   8 blocks, 6 tiles:   d 64 11.3, 11.6  d 96 10.3, 11.0  d 128 11.0, 11.5  d 256, 4 blocks: 14.2, 14.2
//             8:         d 64 13.2, 12.1  d 96 11.3, 11.3  d 128 12.2, 11.7                   17.5, 14.7
//   1 block, 12 tiles:   d 64 13.2, 13.5  d 96 12.2, 12.8  d 128 13.5, 14.1  d 256 19.5, 21.6
constexpr ClusterTiles kTilesAlone = {2, 6, 12};

template <int D>
Cut cut_d(const fa_cache& c, int H) {
  using M = Mma8<D, 1, true>;
  return cut_tiles(pieces_of(H / c.H_kv, c.dtype == FA_BF16 ? 16 : 8), c, M::kTile, M::kBlocks, M::kCost, kTilesAlone);
}
Cut cut_mma(const fa_cache& c, int H) {
  switch (c.d) {
    case 16: return cut_d<16>(c, H);
    case 32: return cut_d<32>(c, H);
    case 64: return cut_d<64>(c, H);
    case 96: return cut_d<96>(c, H);
    case 128: return cut_d<128>(c, H);
    default: return cut_d<256>(c, H);
  }
}

// Whether the kernels of fa_decode_e4m3_sm103.cu take the problem.
bool large(const fa_cache& c, int H, const Cut& k) { return k.cluster == 0 && takes_sm103(c, H); }
Cut cut_e4m3(const fa_cache& c, int H) {
  const Cut k = cut_mma(c, H);
  return large(c, H, k) ? cut_e4m3_sm103(c, H) : k;
}


}  // namespace
}  // namespace fa

extern "C" {

size_t fa_decode_e4m3_workspace_bytes(const fa_cache* c, int32_t H) {
  // the size does not go by the scales, whose number is for the call to check
  const bool good = fa::check_pools(c, 1) == FA_OK && fa::check_heads(c, H) == FA_OK;
  return good ? fa::workspace_of(fa::cut_e4m3(*c, H), c->d) : 0;
}

fa_status fa_decode_e4m3(const fa_cache* c, int32_t block_rows, int32_t H, float scale, const void* Q,
                         int64_t q_stride_s, int64_t q_stride_h, const void* K_pages, const void* V_pages,
                         const float* K_scales, const float* V_scales, const int32_t* page_table,
                         const int32_t* lengths, void* O, int64_t o_stride_s, int64_t o_stride_h, float* L,
                         void* workspace, size_t workspace_bytes, void* stream) {
  fa::NvtxRange range("fa_decode_e4m3");
  fa_status st = fa::check_cache_e4m3(c, block_rows);
  if (st == FA_OK) st = fa::check_heads(c, H);
  if (st != FA_OK) return st;
  const fa::DecodeCall x = {c, H, scale, Q, q_stride_s, q_stride_h, K_pages, V_pages, page_table, lengths,
                            O, o_stride_s, o_stride_h, L, workspace, workspace_bytes};
  const fa::Cut k = fa::cut_e4m3(*c, H);
  const size_t need = fa::workspace_of(k, c->d);
  st = fa::check_call(x, need);
  if (st == FA_OK && (!fa::aligned4(K_scales) || !fa::aligned4(V_scales))) st = FA_ERR_INVALID_ARG;
  if (st != FA_OK) return st;
  fa::E4m3Params a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  fa::fill(x, k, need, 1, &a);
  a.KS = K_scales;
  a.VS = V_scales;
  a.block_rows = fa::FastDiv(block_rows);
  a.blocks = c->page_rows / block_rows;
  a.page_scales = (int64_t)c->H_kv * a.blocks;
  a.wait_ns = fa::wait_limit_ns();
  const cudaStream_t s = (cudaStream_t)stream;
  if (fa::large(*c, H, fa::cut_mma(*c, H))) return fa::status_of(fa::launch_e4m3_sm103(c->d, k, a, s));
  cudaError_t e = cudaErrorInvalidValue;
  switch (c->d) {
    case 16: e = fa::launch_d<16>(*c, k, a, s); break;
    case 32: e = fa::launch_d<32>(*c, k, a, s); break;
    case 64: e = fa::launch_d<64>(*c, k, a, s); break;
    case 96: e = fa::launch_d<96>(*c, k, a, s); break;
    case 128: e = fa::launch_d<128>(*c, k, a, s); break;
    case 256: e = fa::launch_d<256>(*c, k, a, s); break;
  }
  return fa::status_of(e);
}

}  // extern "C"
