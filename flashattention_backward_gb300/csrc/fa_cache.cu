// Rows of a paged key-value cache: new rows into their pages
// (fa_cache_append) and rows from page to page (fa_cache_copy_pages).  Both
// move bytes and compute nothing, so HBM is their bound: every byte is read
// once and written once.
//
// A row of one head is d elements, 64 to 1024 bytes, which 4 to 64 threads
// move as 16-byte pieces.  A thread issues the loads of four pieces of K and
// four of V before its first store, 128 bytes in flight a thread.
//
// Measured: prompts of up to 4000 rows for 4 sequences, 16 heads of d 128, 163 MB
// read and written: 27 to 28 us, 5.9 TB/s (87 % of a copy's rate; 25.7 to 27.2 us in ncu).
// 2048 pages of 16 rows, 8 heads of d 128, 268 MB: 37 to 40 us, 6.8 to 7.2 TB/s
// (ncu).  One row each for 64 sequences: 3.4 us, the launch and three dependent loads.

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fa_paged.cuh"

namespace fa {

int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // pieces of each pool a thread moves at a time
constexpr int kBlockPieces = kThreads * kUnroll;

struct AppendParams {
  const char *K, *V;
  char *KP, *VP;
  const int32_t *table, *start, *counts;
  int32_t* status;
  FastDiv row_pieces, rows, heads, page_rows;
  uint32_t total_rows;   // S * H_kv * rows
  int block_rows;        // rows a block covers
  int num_pages, max_pages;
  int64_t table_stride;
  int64_t sb, sh, sn;    // byte strides of the new rows
  int64_t pp, ph, pn;    // byte strides of the pools
};

__global__ void __launch_bounds__(kThreads) cache_append_kernel(const AppendParams a) {
  after_stream();
  int64_t from[kUnroll], to[kUnroll];
  bool on[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    uint32_t c, i, h;
    const uint32_t r = a.row_pieces.div(u * kThreads + threadIdx.x, &c);
    const uint32_t row = blockIdx.x * (uint32_t)a.block_rows + r;
    on[u] = r < (uint32_t)a.block_rows && row < a.total_rows;
    from[u] = to[u] = 0;
    if (!on[u]) continue;
    const uint32_t sh = a.rows.div(row, &i);
    const uint32_t s = a.heads.div(sh, &h);
    const int64_t start = a.start[s];
    int count = (int)a.rows.d;
    if (a.counts) {
      const int given = a.counts[s];
      if ((given < 0 || given > count) && c == 0 && i == 0 && h == 0) report_pages(a.status);
      count = min(max(given, 0), count);
    }
    on[u] = start >= 0 && (int)i < count;
    if (!on[u]) continue;
    const int64_t pos = start + i;
    const int64_t col = pos < (int64_t(1) << 31) ? (int64_t)a.page_rows.div((uint32_t)pos) : a.max_pages;
    int page = -1;
    if (col < a.max_pages) page = a.table[s * a.table_stride + col];
    if (page < 0 || page >= a.num_pages) {
      on[u] = false;
      if (c == 0) report_pages(a.status);
      continue;
    }
    from[u] = (int64_t)s * a.sb + (int64_t)h * a.sh + (int64_t)i * a.sn + c * 16;
    to[u] = page * a.pp + (int64_t)h * a.ph + (pos - col * a.page_rows.d) * a.pn + c * 16;
  }
  uint4 k[kUnroll], v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (on[u]) {
      k[u] = *reinterpret_cast<const uint4*>(a.K + from[u]);
      v[u] = *reinterpret_cast<const uint4*>(a.V + from[u]);
    }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (on[u]) {
      *reinterpret_cast<uint4*>(a.KP + to[u]) = k[u];
      *reinterpret_cast<uint4*>(a.VP + to[u]) = v[u];
    }
}

struct CopyParams {
  char *KP, *VP;
  const int32_t *moves, *count;
  int32_t* status;
  FastDiv row_pieces, page_rows;
  int max_moves, num_pages;
  int chunks;            // chunks of kBlockPieces in a page
  int pieces;            // H_kv * page_rows * pieces of a row
  int64_t pp, ph, pn;    // byte strides of the pools
  float *KS, *VS;        // kScales: [num_pages, heads, blocks]
  FastDiv blocks;
  int heads, block_rows;
};

// One block takes chunks of pages, a grid's width apart.  The rows of a triple
// do not overlap another's, so loads and stores of one iteration need no
// order; K and V pools are different buffers.  kScales: pools in 8 bits, whose
// scales move along, those of a page shared out among its chunks.
template <bool kScales>
__global__ void __launch_bounds__(kThreads) cache_copy_kernel(const CopyParams a) {
  after_stream();
  int n = a.max_moves;
  if (a.count) {
    const int given = *a.count;
    if ((given < 0 || given > n) && blockIdx.x == 0 && threadIdx.x == 0) report_pages(a.status);
    n = min(max(given, 0), n);
  }
  const int64_t total = (int64_t)n * a.chunks;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x) {
    const int m = (int)(w / a.chunks), chunk = (int)(w - (int64_t)m * a.chunks);
    const int32_t* move = a.moves + 3 * (int64_t)m;
    const int src = move[0], dst = move[1], rows = move[2];
    if (src == -1) continue;
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages || rows < 0 || rows > (int)a.page_rows.d) {
      if (threadIdx.x == 0) report_pages(a.status);
      continue;
    }
    const char *ks = a.KP + src * a.pp, *vs = a.VP + src * a.pp;
    char *kd = a.KP + dst * a.pp, *vd = a.VP + dst * a.pp;
    int64_t at[kUnroll];
    bool on[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int p = chunk * kBlockPieces + u * kThreads + threadIdx.x;
      uint32_t c, r;
      const uint32_t h = a.page_rows.div(a.row_pieces.div(p, &c), &r);
      on[u] = p < a.pieces && (int)r < rows;
      at[u] = (int64_t)h * a.ph + (int64_t)r * a.pn + c * 16;
    }
    uint4 k[kUnroll], v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (on[u]) {
        k[u] = *reinterpret_cast<const uint4*>(ks + at[u]);
        v[u] = *reinterpret_cast<const uint4*>(vs + at[u]);
      }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (on[u]) {
        *reinterpret_cast<uint4*>(kd + at[u]) = k[u];
        *reinterpret_cast<uint4*>(vd + at[u]) = v[u];
      }
    if constexpr (kScales) {
      const int held = (rows + a.block_rows - 1) / a.block_rows;  // blocks of a head that hold rows
      const int64_t all = (int64_t)a.heads * a.blocks.d, from = src * all, to = dst * all;
      for (int64_t x = (int64_t)chunk * kThreads + threadIdx.x; x < all; x += (int64_t)a.chunks * kThreads) {
        uint32_t b;
        a.blocks.div((uint32_t)x, &b);
        if ((int)b >= held) continue;
        const float k = a.KS[from + x], v = a.VS[from + x];
        a.KS[to + x] = k;
        a.VS[to + x] = v;
      }
    }
  }
}

// es: bytes of an element of the pools; block_rows > 0: pools in 8 bits.
fa_status copy_pages(const fa_cache* c, int es, int32_t block_rows, int32_t max_moves, const int32_t* moves,
                     const int32_t* count, void* K_pages, void* V_pages, float* K_scales, float* V_scales,
                     void* stream) {
  if (max_moves < 0 || !aligned16(K_pages) || !aligned16(V_pages) || (max_moves > 0 && !aligned4(moves)) ||
      (count && !aligned4(count)))
    return FA_ERR_INVALID_ARG;
  const int row_pieces = c->d * es / 16;
  const int64_t pieces = (int64_t)c->H_kv * c->page_rows * row_pieces;
  if (pieces > (int64_t(1) << 30)) return FA_ERR_UNSUPPORTED;
  if (max_moves == 0) return FA_OK;
  CopyParams a;
  a.status = device_status_word();
  const int sms = sm_count();
  if (!a.status || sms < 1) return FA_ERR_CUDA;
  a.KP = (char*)K_pages;
  a.VP = (char*)V_pages;
  a.moves = moves;
  a.count = count;
  a.row_pieces = FastDiv(row_pieces);
  a.page_rows = FastDiv(c->page_rows);
  a.max_moves = max_moves;
  a.num_pages = c->num_pages;
  a.pieces = (int)pieces;
  a.chunks = (int)ceil_div(pieces, kBlockPieces);
  a.pp = c->stride_page * es;
  a.ph = c->stride_h * es;
  a.pn = c->stride_n * es;
  a.KS = K_scales;
  a.VS = V_scales;
  a.blocks = FastDiv(block_rows > 0 ? c->page_rows / block_rows : 1);
  a.heads = c->H_kv;
  a.block_rows = block_rows;
  const int64_t work = (int64_t)max_moves * a.chunks;
  const int64_t resident = (int64_t)sms * 8;
  const dim3 grid((unsigned)(work < resident ? work : resident));
  return status_of(launch_early(block_rows > 0 ? cache_copy_kernel<true> : cache_copy_kernel<false>, grid, kThreads, 0,
                                (cudaStream_t)stream, 1, a));
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_cache_append(const fa_cache* c, int32_t rows, const void* K, const void* V, int64_t stride_s,
                          int64_t stride_h, int64_t stride_n, void* K_pages, void* V_pages, const int32_t* page_table,
                          const int32_t* start, const int32_t* counts, void* stream) {
  fa::NvtxRange range("fa_cache_append");
  const fa_status st = fa::check_cache(c);
  if (st != FA_OK) return st;
  const int es = fa::elem_size(c->dtype);
  if (rows < 1 || !fa::aligned16(K) || !fa::aligned16(V) || !fa::aligned16(K_pages) || !fa::aligned16(V_pages) ||
      !fa::aligned4(page_table) || !fa::aligned4(start) || (counts && !fa::aligned4(counts)) ||
      !fa::good_stride(stride_s, c->d, es, false) || !fa::good_stride(stride_h, c->d, es, false) ||
      !fa::good_stride(stride_n, c->d, es, false))
    return FA_ERR_INVALID_ARG;
  const int64_t total = (int64_t)c->S * c->H_kv * rows;
  if (total >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
  fa::AppendParams a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  a.K = (const char*)K;
  a.V = (const char*)V;
  a.KP = (char*)K_pages;
  a.VP = (char*)V_pages;
  a.table = page_table;
  a.start = start;
  a.counts = counts;
  const int row_pieces = c->d * es / 16;
  a.row_pieces = fa::FastDiv(row_pieces);
  a.rows = fa::FastDiv(rows);
  a.heads = fa::FastDiv(c->H_kv);
  a.page_rows = fa::FastDiv(c->page_rows);
  a.total_rows = (uint32_t)total;
  a.block_rows = fa::kBlockPieces / row_pieces;
  a.num_pages = c->num_pages;
  a.max_pages = c->max_pages;
  a.table_stride = c->table_stride;
  a.sb = stride_s * es;
  a.sh = stride_h * es;
  a.sn = stride_n * es;
  a.pp = c->stride_page * es;
  a.ph = c->stride_h * es;
  a.pn = c->stride_n * es;
  const unsigned blocks = (unsigned)fa::ceil_div(total, a.block_rows);
  return fa::status_of(fa::launch_early(fa::cache_append_kernel, dim3(blocks), fa::kThreads, 0, (cudaStream_t)stream, 1, a));
}

fa_status fa_cache_copy_pages(const fa_cache* c, int32_t max_moves, const int32_t* moves, const int32_t* count,
                              void* K_pages, void* V_pages, void* stream) {
  fa::NvtxRange range("fa_cache_copy_pages");
  const fa_status st = fa::check_cache(c);
  if (st != FA_OK) return st;
  return fa::copy_pages(c, fa::elem_size(c->dtype), 0, max_moves, moves, count, K_pages, V_pages, nullptr, nullptr, stream);
}

fa_status fa_cache_copy_pages_e4m3(const fa_cache* c, int32_t block_rows, int32_t max_moves, const int32_t* moves,
                                   const int32_t* count, void* K_pages, void* V_pages, float* K_scales,
                                   float* V_scales, void* stream) {
  fa::NvtxRange range("fa_cache_copy_pages_e4m3");
  const fa_status st = fa::check_cache_e4m3(c, block_rows);
  if (st != FA_OK) return st;
  if (!fa::aligned4(K_scales) || !fa::aligned4(V_scales) || K_pages == V_pages || K_scales == V_scales)
    return FA_ERR_INVALID_ARG;
  return fa::copy_pages(c, 1, block_rows, max_moves, moves, count, K_pages, V_pages, K_scales, V_scales, stream);
}

}  // extern "C"
