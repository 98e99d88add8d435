// Attention of one new token over a paged key-value cache (fa_decode).
//
//   s_j = scale q . k_j,  m = max_j s_j,  l = sum_j 2^(s_j - m),
//   O = sum_j 2^(s_j - m) v_j / l,  L = (m + log2 l) ln 2
// with scores in units of log 2 (the scale carries log2 e).  Over disjoint
// ranges of rows with (m_i, l_i, o_i), o unnormalised, m = max m_i and the l
// and o add up with the factors 2^(m_i - m).
//
// Every row of the cache is read once for the group of query heads that share
// it, 2 d elements a row against 4 d flops a query head: with 8 heads a
// group that is 8 flops a byte in bf16, far below what the tensor cores need
// to be the limit.  HBM is, so the design is about loads: all SMs have an
// equal share of the rows, whatever the lengths, and each keeps about 100 KB
// of loads in flight.
//
// How the work is shared out and joined is in fa_decode.cuh.
//
// Measured (GPU time; the share is of the 6.8 TB/s of a copy): 64 sequences of up
// to 8192 rows, 32 heads on 8 of d 128, 987 MB: 152 to 155 us, 94 to 96 %.  4 of 8192, 16 heads
// of d 256, 537 MB: 90 to 92 us, 85 to 87 %.  32 of up to 2048, 32 heads of d 64, 235 MB: 44 to
// 45 us, 77 %; one of 32768, 8 heads of d 128, 134 MB: 28 us, 70 %: the start of a call,
// the last tiles and the join take about 8 us beside the loads.

#include "fa_decode.cuh"

namespace fa {
namespace {

// ------------------------------------------------------- bf16: tensor cores
// A warp takes 16 rows of each tile with mma.m16n8k16:
//
//  S = Q K^T     A = 16 query heads x 16 columns, B = 16 columns x 8 keys.
//                A sum may be taken in any order, so the 16 columns of a step are
//                those that make a lane's share of B a run of 16 bytes of a key,
//                two steps' worth, and the same columns of Q are A's.
//  O^T += V^T P^T  A = 16 columns x 16 keys, B = 16 keys x 8 heads: S's
//                accumulators are P^T's operand as they stand, and ldmatrix turns
//                V round.
//
// A warp copies its own 16 rows (cp.async into a ring of its own) and waits for
// them alone: no block barrier in the loop, conflict-free 16-byte
// shared-memory reads.  tcgen05 could take the keys as the 64 or 128 rows of A
// and the heads as B's columns in both products, at the price of a barrier a
// tile and of the weights' way through tensor memory, for products that are not
// the limit up to 16 heads.  Above 16 they are part of it: 32 heads a key head
// reach 42 % of a copy's rate at d 32, 53 to 64 % at d 64 to 256 (32 sequences of 8192
// rows), against 80 to 90 % with 16.
//
// P is multiplied as the sum of two bf16 numbers (p rounded, and what is left
// rounded): the second product costs nothing beside the loads, and leaves the
// rounding of the output as the only one to fewer than 16 bits.  What is left
// may be 0 or below it, which makes NaN of an infinity in V: infinite_values().
template <int D>
struct Mma {
  static constexpr int kRows = 16;             // of a tile, a warp
  static constexpr int kTile = kWarps * kRows;
  static constexpr int kVW = D % 64 ? 32 : 64; // columns of O that are exchanged at a time
  static constexpr int kPieces = D / 8;        // of 16 bytes in a row
  // 16 bytes between rows: the 8 lanes of an access's quarter then take 8
  // different groups of 4 banks, of K (2 keys x 4 pieces, 2 apart) as of V (8 keys,
  // one piece)
  static constexpr int kPitch = D * 2 + 16;
  static constexpr int kStageBytes = 2 * kRows * kPitch;  // K and V rows of a warp
  // Bytes in flight an SM: (stages - 1) of blocks x warps x 64 d.
  static constexpr int kBlocks = blocks_an_sm(true, D);
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Puts the infinities of V where its rows gave NaN, although the weights are
// none: in the sums that this thread has just stored at `dst`, heads `pitch`
// bytes apart (bf16, or fp32 where they are a part), over tiles first ... last
// of an item.  The weights are positive, so a column is infinite if its
// infinities are of one sign and it holds no NaN.  Each thread by itself, and
// never in ordinary use: 64 sequences of up to 8192 rows, 32 heads on 8 of d 128,
// take 1.9 ms with an infinity in every page, 4.0 ms with nothing else in V, and
// 0.15 ms without.
template <int D, int NH>
__device__ __noinline__ void infinite_values(const DecodeParams& a, int s, int item, int rows, int first, int last,
                                             int heads, char* dst, int64_t pitch, bool part) {
  constexpr int VW = Mma<D>::kVW, kAhead = 4;
  const int end = min(rows, (last + 1) * Mma<D>::kTile);
#pragma unroll 1
  for (int i = 0; i < NH * (D / VW); ++i)
#pragma unroll 1
    for (int k = threadIdx.x; k < 2 * VW; k += kThreads) {  // four columns of a head, as they were stored
      const int head = 8 * (i / (D / VW)) + k / (VW / 4), col = i % (D / VW) * VW + k % (VW / 4) * 4;
      if (head >= heads) continue;
      float* as_part = reinterpret_cast<float*>(dst + head * pitch) + col;
      __nv_bfloat16* as_bf16 = reinterpret_cast<__nv_bfloat16*>(dst + head * pitch) + col;
      uint32_t lost = 0;  // a bit a column: NaN here, and infinities above, below and NaN in its rows
#pragma unroll
      for (int x = 0; x < 4; ++x) lost |= isnan(part ? as_part[x] : __bfloat162float(as_bf16[x])) ? 1u << x : 0;
      if (!lost) continue;
      uint32_t above = 0, below = 0, none = 0;
#pragma unroll 1
      for (int j = first * Mma<D>::kTile; j < end; j += kAhead) {
        uint2 v[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          uint32_t r;
          const uint32_t c = a.page_rows.div((uint32_t)(j + e), &r);
          const int page = j + e < end ? a.table[s * a.table_stride + c] : -1;
          v[e] = make_uint2(0, 0);
          if (page >= 0 && page < a.num_pages)
            v[e] = *reinterpret_cast<const uint2*>(a.V + page * a.pp + item * a.ph + (int64_t)r * a.pn + 2 * col);
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t bits = (x < 2 ? v[e].x : v[e].y) >> (x % 2 * 16) & 0xffffu;
            above |= bits == 0x7f80u ? 1u << x : 0;
            below |= bits == 0xff80u ? 1u << x : 0;
            none |= (bits & 0x7fffu) > 0x7f80u ? 1u << x : 0;
          }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (!((lost & ~none & (above ^ below)) >> x & 1)) continue;
        const float inf = above >> x & 1 ? INFINITY : -INFINITY;
        if (part)
          as_part[x] = inf;
        else
          as_bf16[x] = __float2bfloat16(inf);
      }
    }
}

// kAlone: a cluster an item, joined here; else a block a run.
template <int D, int NH, bool kAlone>
__global__ void __launch_bounds__(kThreads, Mma<D>::kBlocks) decode_mma_kernel(const __grid_constant__ DecodeParams a) {
  using M = Mma<D>;
  constexpr int kTile = M::kTile, kStages = M::kStages, VW = M::kVW;
  constexpr int kHeads = 8 * NH;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 ml[kWarps][kHeads];
  __shared__ float2 part_ml[kHeads];  // kAlone: this block's part, with o in part_o
  float4* part_o = reinterpret_cast<float4*>(smem);  // over the ring, which is read by then
  Place<kTile> at;
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
  Loader<kTile, M::kRows, M::kPieces, M::kPitch, kStages> load(a, at, end, ring, piece);

  uint32_t qf[NH][D / 32][4];
  float acc[NH][D / VW][VW / 16][4];  // O^T, unnormalised
  float m[NH], l[NH];                 // of heads g, g + 8; l of this lane's keys alone
  int begin = at.t;                   // tile at which the item (or this block's part of it) began
  int stage = 0;
  bool first = true, last = !some;    // item of the run

  for (bool fresh = true; !last; fresh = false) {
    Place<kTile> next = at;
    next.next(a);
    last = next.unit >= end;
    const uint32_t seen = load.next(stage);

    if (fresh || at.t == 0) {
      int heads;
      const int h0 = first_head(a, at.item, piece, &heads);
      const char* row = a.Q + at.s * a.qs + (int64_t)h0 * a.qh;
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        const bool on = g + 8 * u < heads;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 x = on ? *reinterpret_cast<const uint4*>(row + (g + 8 * u) * a.qh + M::k_piece(c, q) * 16)
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
      // V^T's operand: four 8 x 8 pieces of V (keys 0 - 7 and 8 - 15, columns 0 - 7
      // and 8 - 15 of a step), turned round on their way; lane 8 n + r names row r of piece n
      const uint32_t v_at = ring + stage * M::kStageBytes + M::kStageBytes / 2 +
                            ((lane & 7) + (lane >> 4) * 8) * M::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int c = 0; c < D / VW; ++c) {
#pragma unroll
        for (int e = 0; e < VW / 16; ++e) {
          uint32_t a0, a1, a2, a3;
          ldmatrix_trans(v_at + (c * VW + e * 16) * 2, a0, a1, a2, a3);
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
      const bool whole = begin == 0 && at.t + 1 == at.tiles && !(kAlone && a.cluster > 1);
      // the part of an item that was being read when the run began is the
      // block's first, any other its second
      const int slot = (2 * (blockIdx.x / a.split) + (first ? 0 : 1)) * a.split + piece;
      first = false;
      int heads;
      const int h0 = first_head(a, at.item, piece, &heads);
      __syncthreads();  // ml and the exchange buffer have been read
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if (q == 0) ml[warp][g + 8 * u] = make_float2(m[u], l[u]);
      }
      __syncthreads();
      bool odd = false;  // NaN in a sum of this thread's, with weights that are none
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
#pragma unroll
        for (int c = 0; c < D / VW; ++c) {
          if (u + c > 0) __syncthreads();
          float* mine_at = exchange + (warp * 8 + 2 * q) * M::kPad + g;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < VW / 16; ++x) {
              mine_at[e * M::kPad + 16 * x] = acc[u][c][x][e] * f[e];
              mine_at[e * M::kPad + 16 * x + 8] = acc[u][c][x][2 + e] * f[e];
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
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][head].x);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              sum += ml[w][head].y * ptx::ex2(ml[w][head].x - base_of(top));
              const float4 x = *reinterpret_cast<const float4*>(exchange + (w * 8 + in8) * M::kPad + col - c * VW);
              o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
            }
            odd |= isnan((o.x + o.y) + (o.z + o.w)) && !isnan(sum);
            if (whole) {
              const bool none = sum == 0.f;
              const float inv = none ? 0.f : 1.f / sum;
              o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
              store4<__nv_bfloat16>(a.O + at.s * a.os + (int64_t)(h0 + head) * a.oh, col, o);
              if (col == 0) a.L[(int64_t)at.s * a.H + h0 + head] = none ? INFINITY : (top + log2f(sum)) * kLn2;
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
      if (odd) {
        char* dst = whole    ? a.O + at.s * a.os + h0 * a.oh
                    : kAlone ? reinterpret_cast<char*>(part_o)
                             : reinterpret_cast<char*>(a.part_o + (int64_t)slot * kHeads * D);
        infinite_values<D, NH>(a, at.s, at.item, at.rows, begin, at.t, heads, dst, whole ? a.oh : D * 4, !whole);
      }
    }
    at = next;
  }
  if (kAlone && a.cluster > 1) join_cluster<__nv_bfloat16, D>(a, part_o, part_ml);
}

template <int D, int NH>
cudaError_t launch_mma(const Cut& k, const DecodeParams& a, cudaStream_t s) {
  static std::atomic<int> known[64], known_alone[64];
  return launch_decode<__nv_bfloat16, D, Mma<D>::kTile>(k, a, decode_mma_kernel<D, NH, false>,
                                                        decode_mma_kernel<D, NH, true>, Mma<D>::kSmem, known,
                                                        known_alone, s);
}

template <int D>
cudaError_t launch_bf16(const Cut& k, const DecodeParams& a, cudaStream_t s) {
  return k.part_heads == 8 ? launch_mma<D, 1>(k, a, s) : launch_mma<D, 2>(k, a, s);
}

fa_status check(const fa_cache* c, int32_t H) {
  const fa_status st = check_cache(c);
  return st == FA_OK ? check_heads(c, H) : st;
}

}  // namespace

cudaError_t launch_decode_bf16(const fa_cache& c, const Cut& k, const DecodeParams& a, cudaStream_t s) {
  switch (c.d) {
    case 32: return launch_bf16<32>(k, a, s);
    case 64: return launch_bf16<64>(k, a, s);
    case 96: return launch_bf16<96>(k, a, s);
    case 128: return launch_bf16<128>(k, a, s);
    case 256: return launch_bf16<256>(k, a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa

extern "C" {

size_t fa_decode_workspace_bytes(const fa_cache* c, int32_t H) {
  return fa::check(c, H) == FA_OK ? fa::workspace_of(fa::cut_of(*c, H), c->d) : 0;
}

fa_status fa_decode(const fa_cache* c, int32_t H, float scale, const void* Q, int64_t q_stride_s, int64_t q_stride_h,
                    const void* K_pages, const void* V_pages, const int32_t* page_table, const int32_t* lengths,
                    void* O, int64_t o_stride_s, int64_t o_stride_h, float* L, void* workspace,
                    size_t workspace_bytes, void* stream) {
  fa::NvtxRange range("fa_decode");
  fa_status st = fa::check(c, H);
  if (st != FA_OK) return st;
  const fa::DecodeCall x = {c, H, scale, Q, q_stride_s, q_stride_h, K_pages, V_pages, page_table, lengths,
                            O, o_stride_s, o_stride_h, L, workspace, workspace_bytes};
  const fa::Cut k = fa::cut_of(*c, H);
  const size_t need = fa::workspace_of(k, c->d);
  st = fa::check_call(x, need);
  if (st != FA_OK) return st;
  fa::DecodeParams a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  fa::fill(x, k, need, fa::elem_size(c->dtype), &a);
  const cudaStream_t s = (cudaStream_t)stream;
  return fa::status_of(c->dtype == FA_BF16 ? fa::launch_decode_bf16(*c, k, a, s) : fa::launch_decode_fp32(*c, k, a, s));
}

}  // extern "C"
