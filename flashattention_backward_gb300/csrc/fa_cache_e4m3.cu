// Rows of a paged key-value cache in 8 bits: quantised as they are written
// (fa_cache_append_e4m3) and read back (fa_cache_read_e4m3).
//
// A block is block_rows rows of one page and head that share a scale,
//   s = 2^e,  e = max(ceil(log2(t / 448)), -126),  t = max |x| over its new rows,
// and no less than the block's scale where it holds rows already.  A power of
// two, because x / s and q s are then exact, and because moving rows to a larger
// scale costs nothing but what falls below e4m3's smallest normal number; a
// number of 4 significant bits is not held better by t / 448 itself.
//
// Both kernels move bytes: HBM is their bound.

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_e4m3.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

struct AppendParams {
  const char* X[2];   // K, V
  uint8_t* pages[2];
  float* scales[2];
  const int32_t *table, *start, *counts;
  int32_t* status;
  FastDiv many, heads, page_rows, block_rows, row_units;
  int rows, num_pages, max_pages;
  int64_t table_stride;
  int64_t sb, sh, sn;  // byte strides of the new rows
  int64_t pp, ph, pn;  // of the pools
};

// 16 numbers of a row
template <class T>
__device__ __forceinline__ void load16(const char* p, float (&x)[16]) {
  const uint4* v = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T); ++i) {
    const uint4 y = v[i];
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[8 * i + 2 * e] = ptx::bf16lo(w[e]), x[8 * i + 2 * e + 1] = ptx::bf16hi(w[e]);
    } else {
      x[4 * i] = __uint_as_float(y.x), x[4 * i + 1] = __uint_as_float(y.y);
      x[4 * i + 2] = __uint_as_float(y.z), x[4 * i + 3] = __uint_as_float(y.w);
    }
  }
}

// Block of threads (x, y): the x-th touched block of a sequence and head, of K or V.
template <class T>
__global__ void __launch_bounds__(kThreads) append_e4m3_kernel(const AppendParams a) {
  after_stream();
  __shared__ uint32_t tops[kThreads / 32];
  uint32_t nth, g;
  const uint32_t s = a.heads.div(a.many.div(blockIdx.x, &nth), &g);
  const int pool = blockIdx.y;
  const bool first_of_s = nth == 0 && g == 0 && pool == 0 && threadIdx.x == 0;
  const int64_t start = a.start[s];
  int count = a.rows;
  if (a.counts) {
    const int given = a.counts[s];
    if ((given < 0 || given > count) && first_of_s) report_pages(a.status);
    count = min(max(given, 0), count);
  }
  if (start < 0) return;
  const int br = a.block_rows.d;
  const int64_t lo = ((int64_t)a.block_rows.div((uint32_t)start) + nth) * br;
  const int64_t from = max(start, lo), to = min(start + count, lo + br);
  if (from >= to) return;
  const int64_t col = lo < (int64_t(1) << 31) ? (int64_t)a.page_rows.div((uint32_t)lo) : a.max_pages;
  int page = -1;
  if (col < a.max_pages) page = a.table[s * a.table_stride + col];
  if (page < 0 || page >= a.num_pages) {
    if (threadIdx.x == 0) report_pages(a.status);
    return;
  }
  const int row0 = (int)(lo - col * a.page_rows.d);
  uint8_t* dst = a.pages[pool] + page * a.pp + g * a.ph + row0 * a.pn;
  float* scale_at = a.scales[pool] + ((int64_t)page * a.heads.d + g) * (a.page_rows.d / br) + row0 / br;
  const char* src = a.X[pool] + s * a.sb + g * a.sh + (from - start) * a.sn;

  const int units = (int)(to - from) * a.row_units.d;
  uint32_t top = 0;
  for (int u = threadIdx.x; u < units; u += kThreads) {
    uint32_t c;
    const uint32_t r = a.row_units.div(u, &c);
    float x[16];
    load16<T>(src + r * a.sn + c * 16 * sizeof(T), x);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t t = __float_as_uint(x[e]) & 0x7fffffffu;
      top = max(top, t < 0x7f800000u ? t : 0u);
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  const float old = from > lo ? *scale_at : 0.f;
  __syncthreads();  // everyone has the old scale
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = max(top, tops[w]);
  const float scale = fmaxf(scale_for(top), old), inv = inverse(scale);
  if (threadIdx.x == 0) *scale_at = scale;
  for (int u = threadIdx.x; u < units; u += kThreads) {
    uint32_t c;
    const uint32_t r = a.row_units.div(u, &c);
    float x[16];
    load16<T>(src + r * a.sn + c * 16 * sizeof(T), x);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = isfinite(x[e]) ? x[e] * inv : NAN;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_e4m3x4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
    *reinterpret_cast<uint4*>(dst + (from - lo + r) * a.pn + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (from > lo && scale > old) {
    const float by = old * inv;
    for (int u = threadIdx.x; u < (int)(from - lo) * (int)a.row_units.d; u += kThreads) {
      uint32_t c;
      const uint32_t r = a.row_units.div(u, &c);
      uint4* at = reinterpret_cast<uint4*>(dst + r * a.pn + c * 16);
      const uint4 q = *at;
      uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 x = e4m3x4_to_float4(w[e]);
        w[e] = pack_e4m3x4(x.x * by, x.y * by, x.z * by, x.w * by);
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

struct ReadParams {
  const uint8_t* pages[2];
  const float* scales[2];
  char* X[2];
  const int32_t *table, *start, *counts;
  int32_t* status;
  FastDiv row_units, rows, heads, page_rows, block_rows;
  uint32_t total_rows;  // S * H_kv * rows
  int block_of_rows;    // rows that a block of threads takes
  int num_pages, max_pages;
  int64_t table_stride;
  int64_t sb, sh, sn;   // byte strides of the rows outside
  int64_t pp, ph, pn;   // of the pools
};

template <class T>
__global__ void __launch_bounds__(kThreads) read_e4m3_kernel(const ReadParams a) {
  after_stream();
  uint32_t c, i, g;
  const uint32_t r = a.row_units.div(threadIdx.x, &c);
  const uint32_t row = blockIdx.x * (uint32_t)a.block_of_rows + r;
  if (r >= (uint32_t)a.block_of_rows || row >= a.total_rows) return;
  const uint32_t s = a.heads.div(a.rows.div(row, &i), &g);
  const bool first_of_s = c == 0 && i == 0 && g == 0;
  const int64_t start = a.start ? a.start[s] : 0;
  int count = (int)a.rows.d;
  if (a.counts) {
    const int given = a.counts[s];
    if ((given < 0 || given > count) && first_of_s) report_pages(a.status);
    count = min(max(given, 0), count);
  }
  if (start < 0 && first_of_s) report_pages(a.status);
  bool on = start >= 0 && (int)i < count;
  int64_t from = 0, scale_at = 0;
  if (on) {
    const int64_t pos = start + i;
    const int64_t col = pos < (int64_t(1) << 31) ? (int64_t)a.page_rows.div((uint32_t)pos) : a.max_pages;
    int page = -1;
    if (col < a.max_pages) page = a.table[s * a.table_stride + col];
    on = page >= 0 && page < a.num_pages;
    if (!on && c == 0) report_pages(a.status);
    if (on) {
      const int in_page = (int)(pos - col * a.page_rows.d);
      from = page * a.pp + g * a.ph + in_page * a.pn + c * 16;
      scale_at = ((int64_t)page * a.heads.d + g) * (a.page_rows.d / a.block_rows.d) + a.block_rows.div(in_page);
    }
  }
  const int64_t to = s * a.sb + g * a.sh + i * a.sn + c * 16 * (int)sizeof(T);
#pragma unroll
  for (int pool = 0; pool < 2; ++pool) {
    uint4 q = make_uint4(0, 0, 0, 0);
    float scale = 0.f;
    if (on) {
      q = *reinterpret_cast<const uint4*>(a.pages[pool] + from);
      scale = a.scales[pool][scale_at];
    }
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint4* dst = reinterpret_cast<uint4*>(a.X[pool] + to);
    float4 x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = e4m3x4_to_float4(w[e]);
      x[e] = on ? make_float4(x[e].x * scale, x[e].y * scale, x[e].z * scale, x[e].w * scale) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int e = 0; e < (int)sizeof(T); ++e) {
      if constexpr (sizeof(T) == 2)
        dst[e] = make_uint4(ptx::pack_bf16x2(x[2 * e].x, x[2 * e].y), ptx::pack_bf16x2(x[2 * e].z, x[2 * e].w),
                            ptx::pack_bf16x2(x[2 * e + 1].x, x[2 * e + 1].y), ptx::pack_bf16x2(x[2 * e + 1].z, x[2 * e + 1].w));
      else
        *reinterpret_cast<float4*>(dst + e) = x[e];
    }
  }
}

// Arguments that both calls take.
fa_status check_rows(const fa_cache* c, int32_t block_rows, int32_t rows, const void* K, const void* V, int64_t ss,
                     int64_t sh, int64_t sn, const void* KP, const void* VP, const void* KS, const void* VS,
                     const int32_t* table, const int32_t* start, const int32_t* counts, bool reads) {
  const fa_status st = check_cache_e4m3(c, block_rows);
  if (st != FA_OK) return st;
  const int es = elem_size(c->dtype);
  if (rows < 1 || !aligned16(K) || !aligned16(V) || !aligned16(KP) || !aligned16(VP) || !aligned4(KS) || !aligned4(VS) ||
      !aligned4(table) || (start ? !aligned4(start) : !reads) || (counts && !aligned4(counts)) ||
      !good_stride(ss, c->d, es, reads) || !good_stride(sh, c->d, es, reads) || !good_stride(sn, c->d, es, reads) ||
      (reads ? K == V : KP == VP || KS == VS))
    return FA_ERR_INVALID_ARG;
  return (int64_t)c->S * c->H_kv * rows < (int64_t(1) << 31) ? FA_OK : FA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace fa

extern "C" {

fa_status fa_cache_append_e4m3(const fa_cache* c, int32_t block_rows, int32_t rows, const void* K, const void* V,
                               int64_t stride_s, int64_t stride_h, int64_t stride_n, void* K_pages, void* V_pages,
                               float* K_scales, float* V_scales, const int32_t* page_table, const int32_t* start,
                               const int32_t* counts, void* stream) {
  fa::NvtxRange range("fa_cache_append_e4m3");
  const fa_status st = fa::check_rows(c, block_rows, rows, K, V, stride_s, stride_h, stride_n, K_pages, V_pages,
                                      K_scales, V_scales, page_table, start, counts, false);
  if (st != FA_OK) return st;
  const int es = fa::elem_size(c->dtype);
  fa::AppendParams a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  a.X[0] = (const char*)K, a.X[1] = (const char*)V;
  a.pages[0] = (uint8_t*)K_pages, a.pages[1] = (uint8_t*)V_pages;
  a.scales[0] = K_scales, a.scales[1] = V_scales;
  a.table = page_table;
  a.start = start;
  a.counts = counts;
  // blocks that `rows` rows can touch, whatever the start
  const int many = (int)(((int64_t)rows + block_rows - 2) / block_rows + 1);
  a.many = fa::FastDiv(many);
  a.heads = fa::FastDiv(c->H_kv);
  a.page_rows = fa::FastDiv(c->page_rows);
  a.block_rows = fa::FastDiv(block_rows);
  a.row_units = fa::FastDiv(c->d / 16);
  a.rows = rows;
  a.num_pages = c->num_pages;
  a.max_pages = c->max_pages;
  a.table_stride = c->table_stride;
  a.sb = stride_s * es;
  a.sh = stride_h * es;
  a.sn = stride_n * es;
  a.pp = c->stride_page;
  a.ph = c->stride_h;
  a.pn = c->stride_n;
  // many <= rows, so the blocks are fewer than 2^31
  const dim3 grid((unsigned)((int64_t)c->S * c->H_kv * many), 2);
  const cudaStream_t s = (cudaStream_t)stream;
  return fa::status_of(c->dtype == FA_BF16
                           ? fa::launch_early(fa::append_e4m3_kernel<__nv_bfloat16>, grid, fa::kThreads, 0, s, 1, a)
                           : fa::launch_early(fa::append_e4m3_kernel<float>, grid, fa::kThreads, 0, s, 1, a));
}

fa_status fa_cache_read_e4m3(const fa_cache* c, int32_t block_rows, int32_t rows, const void* K_pages,
                             const void* V_pages, const float* K_scales, const float* V_scales,
                             const int32_t* page_table, const int32_t* start, const int32_t* counts, void* K, void* V,
                             int64_t stride_s, int64_t stride_h, int64_t stride_n, void* stream) {
  fa::NvtxRange range("fa_cache_read_e4m3");
  const fa_status st = fa::check_rows(c, block_rows, rows, K, V, stride_s, stride_h, stride_n, K_pages, V_pages,
                                      K_scales, V_scales, page_table, start, counts, true);
  if (st != FA_OK) return st;
  const int es = fa::elem_size(c->dtype);
  fa::ReadParams a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  a.pages[0] = (const uint8_t*)K_pages, a.pages[1] = (const uint8_t*)V_pages;
  a.scales[0] = K_scales, a.scales[1] = V_scales;
  a.X[0] = (char*)K, a.X[1] = (char*)V;
  a.table = page_table;
  a.start = start;
  a.counts = counts;
  a.row_units = fa::FastDiv(c->d / 16);
  a.rows = fa::FastDiv(rows);
  a.heads = fa::FastDiv(c->H_kv);
  a.page_rows = fa::FastDiv(c->page_rows);
  a.block_rows = fa::FastDiv(block_rows);
  a.total_rows = (uint32_t)((int64_t)c->S * c->H_kv * rows);
  a.block_of_rows = fa::kThreads / (c->d / 16);
  a.num_pages = c->num_pages;
  a.max_pages = c->max_pages;
  a.table_stride = c->table_stride;
  a.sb = stride_s * es;
  a.sh = stride_h * es;
  a.sn = stride_n * es;
  a.pp = c->stride_page;
  a.ph = c->stride_h;
  a.pn = c->stride_n;
  const dim3 grid((unsigned)fa::ceil_div(a.total_rows, a.block_of_rows));
  const cudaStream_t s = (cudaStream_t)stream;
  return fa::status_of(c->dtype == FA_BF16
                           ? fa::launch_early(fa::read_e4m3_kernel<__nv_bfloat16>, grid, fa::kThreads, 0, s, 1, a)
                           : fa::launch_early(fa::read_e4m3_kernel<float>, grid, fa::kThreads, 0, s, 1, a));
}

}  // extern "C"
