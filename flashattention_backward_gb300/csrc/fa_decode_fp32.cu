// Attention of one new token over a paged key-value cache in fp32 (fa_decode
// with FA_FP32): exact fp32 arithmetic on the CUDA cores, no TF32.  The formulas
// are those of fa_decode.cu; how the work is shared out and joined is in
// fa_decode.cuh.
//
// 4 d flops a row of the cache for each of the query heads that share
// it, against 8 d bytes: 4 flops a byte with 8 heads, a third of what the FMA
// units could do while HBM sends it.  So here too the loads are what counts, but
// the operands' way through shared memory has to stay short:
//
//  scores  Lane (g, q) takes a slice of the columns of several keys (an eighth of
//          four keys with 8 heads, a quarter of two with fewer), for all heads: a
//          piece of Q from shared memory serves all its keys, a piece of K all
//          heads.  The slices are added up by halves: lanes exchange the heads
//          that the other is to have, so that lane q ends with the full scores of
//          a head or two and takes their exponentials alone.
//  output  A lane holds 4 columns (or a few times 4) of all heads, and a warp's
//          lanes take whole rows of V; the weights of a row, all heads in one or
//          two 16-byte pieces of shared memory, are the same for all of them.
//
// Measured at 32 sequences of 8192 rows, as a share of the 6.8 TB/s of a copy: 94 to
// 98 % with one query head a key head (d 32 to 256), 86 to 94 % with four, at d 16 81 and
// 79 %.  With eight, 87 % at d 64, 82 % at d 128, 76 % at d 32 and 96, 61 % at d 16, whose
// tiles are 1 KB of K for a warp, and 56 % at d 256, whose tiles have 8 rows a warp
// and whose SMs one warp a scheduler.  Above eight each piece of the heads reads the
// tile again: 29 (d 256) to 48 % (d 64) with 16.

#include "fa_decode.cuh"

namespace fa {
namespace {

template <int D, int HR>
struct Simt {
  static constexpr int kRows = D == 256 ? 8 : 16;  // of a tile, a warp
  static constexpr int kTile = kWarps * kRows;
  static constexpr int kPieces = D / 4;            // of 16 bytes in a row
  static constexpr int kPitch = D * 4 + 16;        // rows start on different banks
  static constexpr int kStageBytes = 2 * kRows * kPitch;
  static constexpr int kStages = D == 16 ? 4 : 3;
  static constexpr int kBlocks = blocks_an_sm(false, D);
  // Lanes that share a key's columns, and keys a lane has at a time: with 8
  // heads eight lanes, so that a piece of Q serves four keys
  static constexpr int kSlices = HR == 8 && kRows == 16 && kPieces % 8 == 0 ? 8 : 4;
  static constexpr int kKeys = kRows * kSlices / 32;
  // Lanes of a row of V: with 8 heads a lane has at least two pieces, so that
  // the weights of a row serve both
  static constexpr int kLanes = D == 96 ? 8 : D == 256 ? 32 : HR == 8 && D >= 32 ? kPieces / 2 : kPieces;
  static constexpr int kCols = kPieces / kLanes;   // pieces a lane holds
  static constexpr int kGroups = 32 / kLanes;      // rows of V a warp takes at a time
  static constexpr int kOwn = HR > kSlices ? HR / kSlices : 1;  // heads a lane has the scores of
  static constexpr int kChunk = HR == 1 ? 1 : D == 256 ? 2 : 4;  // heads exchanged at a time
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kQ = kRing;                             // [HR][D]
  static constexpr int kP = kQ + HR * D * 4;                   // [kWarps][kRows][HR]
  static constexpr int kExchange = kP + kWarps * kRows * HR * 4;  // [kWarps][kChunk][D]
  static constexpr int kSmem = kExchange + kWarps * kChunk * D * 4;
  static_assert(kSmem <= 232448 - 2048, "shared memory budget");
};

// s[h] += dot(q, k) of one 16-byte piece
__device__ __forceinline__ float dot4(float4 q, float4 k, float s) {
  return fmaf(q.w, k.w, fmaf(q.z, k.z, fmaf(q.y, k.y, fmaf(q.x, k.x, s))));
}

// kAlone: a cluster an item, joined here; else a block a run.
template <int D, int HR, bool kAlone>
__global__ void __launch_bounds__(kThreads, Simt<D, HR>::kBlocks)
    decode_simt_kernel(const __grid_constant__ DecodeParams a) {
  using M = Simt<D, HR>;
  constexpr int kTile = M::kTile, kStages = M::kStages, kKeys = M::kKeys, kSlices = M::kSlices;
  constexpr int kKeyStep = 32 / kSlices;  // keys side by side
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 ml[kWarps][HR];
  __shared__ __align__(16) float factors[kWarps][HR];
  __shared__ float2 part_ml[HR];  // kAlone: this block's part, with o in part_o
  float4* part_o = reinterpret_cast<float4*>(smem);  // over the ring, which is read by then
  Place<kTile> at;
  int64_t end;
  bool some;
  after_stream();
  if constexpr (kAlone) {
    some = share_of_item(a, &at, &end);
    if (!some && threadIdx.x < HR) part_ml[threadIdx.x] = make_float2(-INFINITY, kNoPart);
  } else {
    next_may_start();  // the join
    some = run_of(a, &at, &end);
    if (!some) return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / kSlices, q = lane % kSlices;
  const int piece = (kAlone ? blockIdx.x / a.cluster : blockIdx.x) % a.split;
  const uint8_t* ring = smem + warp * kStages * M::kStageBytes;
  float* qs = reinterpret_cast<float*>(smem + M::kQ);
  float* ps = reinterpret_cast<float*>(smem + M::kP) + warp * M::kRows * HR;
  float* exchange = reinterpret_cast<float*>(smem + M::kExchange);
  Loader<kTile, M::kRows, M::kPieces, M::kPitch, kStages> load(a, at, end, ptx::smem_addr(ring), piece);

  const int x0 = lane % M::kLanes, row0 = lane / M::kLanes;  // of V: first piece and row
  const int h_own = HR == 1 ? 0 : M::kOwn * q;               // first head this lane has the scores of
  float4 acc[HR][M::kCols];   // o, unnormalised, of this lane's rows
  float m[M::kOwn], l[M::kOwn];
  int begin = at.t;
  int stage = 0;
  bool first = true, last = !some;

  for (bool fresh = true; !last; fresh = false) {
    Place<kTile> next = at;
    next.next(a);
    last = next.unit >= end;
    const uint32_t seen = load.next(stage);

    if (fresh || at.t == 0) {
      int heads;
      const int h0 = first_head(a, at.item, piece, &heads);
      const char* row = a.Q + at.s * a.qs + (int64_t)h0 * a.qh;
      // the item before has been through a barrier since it read its queries
      for (int k = threadIdx.x; k < HR * M::kPieces; k += kThreads) {
        const int h = k / M::kPieces, piece = k % M::kPieces;
        reinterpret_cast<float4*>(qs)[k] =
            h < heads ? *reinterpret_cast<const float4*>(row + h * a.qh + piece * 16) : make_float4(0, 0, 0, 0);
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < M::kOwn; ++u) m[u] = -INFINITY, l[u] = 0.f;
#pragma unroll
      for (int h = 0; h < HR; ++h)
#pragma unroll
        for (int c = 0; c < M::kCols; ++c) acc[h][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      begin = at.t;
    }

    if (seen) {
      const uint8_t* ks = ring + stage * M::kStageBytes;
      float s[HR][kKeys] = {};
#pragma unroll
      for (int c = 0; c < M::kPieces / kSlices; ++c) {
        // the 8 lanes of an access's quarter take 8 different groups of banks: 8 pieces of a key, or of 2
        // keys, whose rows are a piece more than a multiple of 8 apart, 4 pieces two apart
        const int piece = kSlices == 8 ? 8 * c + q : M::kPieces == 4 ? q : 8 * (c / 2) + 2 * q + c % 2;
        float4 k[kKeys];
#pragma unroll
        for (int e = 0; e < kKeys; ++e) k[e] = *reinterpret_cast<const float4*>(ks + (g + kKeyStep * e) * M::kPitch + piece * 16);
#pragma unroll
        for (int h = 0; h < HR; ++h) {
          const float4 x = *reinterpret_cast<const float4*>(qs + h * D + piece * 4);
#pragma unroll
          for (int e = 0; e < kKeys; ++e) s[h][e] = dot4(x, k[e], s[h][e]);
        }
      }
      // the slices added up by halves: lane q keeps heads h_own ... of its keys
      float x[M::kOwn][kKeys];
#pragma unroll
      for (int e = 0; e < kKeys; ++e) {
        if constexpr (HR == 1) {
          float y = s[0][e];
#pragma unroll
          for (int o = 1; o < kSlices; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
          x[0][e] = y;
        } else {
          float part[HR];
#pragma unroll
          for (int h = 0; h < HR; ++h) part[h] = s[h][e];
#pragma unroll
          for (int o = kSlices / 2, n = HR / 2; o > 0; o >>= 1, n >>= 1)
#pragma unroll
            for (int h = 0; h < HR / 2; ++h)
              if (h < n) {
                const float give = q & o ? part[h] : part[h + n], keep = q & o ? part[h + n] : part[h];
                part[h] = keep + __shfl_xor_sync(0xffffffffu, give, o);
              }
#pragma unroll
          for (int u = 0; u < M::kOwn; ++u) x[u][e] = part[u];
        }
      }
      bool moved = false;
#pragma unroll
      for (int u = 0; u < M::kOwn; ++u) {
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < kKeys; ++e) {
          x[u][e] = (seen >> (g + kKeyStep * e)) & 1 ? x[u][e] * a.scale2 : -INFINITY;
          top = fmaxf(top, x[u][e]);
        }
#pragma unroll
        for (int o = kSlices; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float now = fmaxf(m[u], top), base = base_of(now), alpha = ptx::ex2(m[u] - base);
        moved |= now != m[u];
        m[u] = now;
        l[u] *= alpha;
#pragma unroll
        for (int e = 0; e < kKeys; ++e) {
          x[u][e] = ptx::ex2(x[u][e] - base);
          l[u] += x[u][e];
          if (HR > 1 || q == 0) ps[(g + kKeyStep * e) * HR + h_own + u] = x[u][e];
        }
        if (g == 0 && (HR > 1 || q == 0)) factors[warp][h_own + u] = alpha;
      }
      moved = __any_sync(0xffffffffu, moved);
      __syncwarp();
      if (moved) {
#pragma unroll
        for (int h = 0; h < HR; ++h) {
          const float f = factors[warp][h];
#pragma unroll
          for (int c = 0; c < M::kCols; ++c)
            acc[h][c] = make_float4(acc[h][c].x * f, acc[h][c].y * f, acc[h][c].z * f, acc[h][c].w * f);
        }
      }
      const uint8_t* vs = ks + M::kRows * M::kPitch + x0 * 16;
#pragma unroll
      for (int j = 0; j < M::kRows; j += M::kGroups) {
        float4 v[M::kCols];
#pragma unroll
        for (int c = 0; c < M::kCols; ++c)
          v[c] = *reinterpret_cast<const float4*>(vs + (j + row0) * M::kPitch + c * M::kLanes * 16);
        float p[HR];
        if constexpr (HR == 1) {
          p[0] = ps[j + row0];
        } else {
#pragma unroll
          for (int h = 0; h < HR; h += 4)
            *reinterpret_cast<float4*>(&p[h]) = *reinterpret_cast<const float4*>(ps + (j + row0) * HR + h);
        }
#pragma unroll
        for (int h = 0; h < HR; ++h)
#pragma unroll
          for (int c = 0; c < M::kCols; ++c) {
            acc[h][c].x = fmaf(p[h], v[c].x, acc[h][c].x), acc[h][c].y = fmaf(p[h], v[c].y, acc[h][c].y);
            acc[h][c].z = fmaf(p[h], v[c].z, acc[h][c].z), acc[h][c].w = fmaf(p[h], v[c].w, acc[h][c].w);
          }
      }
      __syncwarp();  // ps and factors have been read
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
      __syncthreads();  // ml, the exchange buffer and the queries have been read
#pragma unroll
      for (int u = 0; u < M::kOwn; ++u) {
#pragma unroll
        for (int o = kSlices; o < 32; o <<= 1) l[u] += __shfl_xor_sync(0xffffffffu, l[u], o);
        if (g == 0 && (HR > 1 || q == 0)) ml[warp][h_own + u] = make_float2(m[u], l[u]);
      }
      __syncthreads();
#pragma unroll
      for (int c0 = 0; c0 < HR; c0 += M::kChunk) {
        if (c0 > 0) __syncthreads();
#pragma unroll
        for (int h = 0; h < M::kChunk; ++h) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k][c0 + h].x);
          const float f = ptx::ex2(ml[warp][c0 + h].x - base_of(top));
#pragma unroll
          for (int c = 0; c < M::kCols; ++c) {
            float4 o = acc[c0 + h][c];
#pragma unroll
            for (int w = M::kLanes; w < 32; w <<= 1) {
              o.x += __shfl_xor_sync(0xffffffffu, o.x, w), o.y += __shfl_xor_sync(0xffffffffu, o.y, w);
              o.z += __shfl_xor_sync(0xffffffffu, o.z, w), o.w += __shfl_xor_sync(0xffffffffu, o.w, w);
            }
            if (row0 == 0)
              reinterpret_cast<float4*>(exchange)[(warp * M::kChunk + h) * M::kPieces + x0 + c * M::kLanes] =
                  make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
          }
        }
        __syncthreads();
        for (int k = threadIdx.x; k < M::kChunk * M::kPieces; k += kThreads) {
          const int head = c0 + k / M::kPieces, piece = k % M::kPieces;
          if (head >= heads) continue;
          float top = -INFINITY, sum = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w][head].x);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            sum += ml[w][head].y * ptx::ex2(ml[w][head].x - base_of(top));
            const float4 v = reinterpret_cast<const float4*>(exchange)[w * M::kChunk * M::kPieces + k];
            o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
          }
          const bool none = sum == 0.f;
          if (whole) {
            const float inv = none ? 0.f : 1.f / sum;
            o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            store4<float>(a.O + at.s * a.os + (int64_t)(h0 + head) * a.oh, 4 * piece, o);
            if (piece == 0) a.L[(int64_t)at.s * a.H + h0 + head] = none ? INFINITY : (top + log2f(sum)) * kLn2;
          } else if (kAlone) {
            part_o[head * M::kPieces + piece] = o;
            if (piece == 0) part_ml[head] = make_float2(top, sum);
          } else {
            const int64_t p = (int64_t)slot * HR + head;
            *reinterpret_cast<float4*>(a.part_o + p * D + 4 * piece) = o;
            if (piece == 0) a.part_ml[p] = make_float2(top, sum);
          }
        }
      }
    }
    at = next;
  }
  if (kAlone && a.cluster > 1) join_cluster<float, D>(a, part_o, part_ml);
}

template <int D, int HR>
cudaError_t launch_simt(const Cut& k, const DecodeParams& a, cudaStream_t s) {
  using M = Simt<D, HR>;
  static std::atomic<int> known[64], known_alone[64];
  return launch_decode<float, D, M::kTile>(k, a, decode_simt_kernel<D, HR, false>, decode_simt_kernel<D, HR, true>,
                                           M::kSmem, known, known_alone, s);
}

template <int D>
cudaError_t launch_fp32(const Cut& k, const DecodeParams& a, cudaStream_t s) {
  switch (k.part_heads) {
    case 1: return launch_simt<D, 1>(k, a, s);
    case 4: return launch_simt<D, 4>(k, a, s);
    default: return launch_simt<D, 8>(k, a, s);
  }
}

}  // namespace

cudaError_t launch_decode_fp32(const fa_cache& c, const Cut& k, const DecodeParams& a, cudaStream_t s) {
  switch (c.d) {
    case 16: return launch_fp32<16>(k, a, s);
    case 32: return launch_fp32<32>(k, a, s);
    case 64: return launch_fp32<64>(k, a, s);
    case 96: return launch_fp32<96>(k, a, s);
    case 128: return launch_fp32<128>(k, a, s);
    case 256: return launch_fp32<256>(k, a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fa
