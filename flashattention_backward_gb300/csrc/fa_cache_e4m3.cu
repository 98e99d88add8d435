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
// Both kernels move bytes and HBM is their bound, as long as the instructions are
// few: a thread takes 16 numbers of a row at a time, 32 or 64 bytes outside and 16 in
// the cache, and keeps what it has read in registers from the search for t to
// the rounding.
//
// Measured (GPU time; the share is of the 6.8 TB/s of a copy): prompts of up to 4000 rows for 4 sequences, 16 heads of
// d 128, blocks of 16 rows: 128 MB, 24.0 us, 79 %; with each unit read twice, from L1 the second time, and a block of
// threads a block of rows: 40.1; with the look at infinities beside the rounding of every number 30.0.  The same rows read back into bf16,
// 165 MB: 27.7 us, 88 %.  One row each for 64 sequences, 8 heads of d 128: 2.4 us, the launch and three
// dependent loads.

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_e4m3.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;
constexpr int kKeep = 4;  // units of 16 numbers that a thread keeps

struct AppendParams {
  const char* X[2];   // K, V
  uint8_t* pages[2];
  float* scales[2];
  const int32_t *table, *start, *counts;
  int32_t* status;
  FastDiv many, heads, page_rows, block_rows, row_units;
  uint32_t teams;      // S * H_kv * many
  int rows, num_pages, max_pages;
  bool wide;           // rows begin on 32 bytes
  int64_t table_stride;
  int64_t sb, sh, sn;  // byte strides of the new rows
  int64_t pp, ph, pn;  // of the pools
};

// 16 numbers of a row, as they are
template <class T>
struct Unit {
  static constexpr int kWords = 16 * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                       "=r"(w[i + 6]), "=r"(w[i + 7])
                     : "l"(p + 4 * i));
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return i % 2 ? ptx::bf16hi(w[i / 2]) : ptx::bf16lo(w[i / 2]);
  }
  // the bits of the largest |x|, NaN apart, and 0x7f800000 if one is infinite
  __device__ __forceinline__ uint32_t top() const {
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 t = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]));
#pragma unroll
      for (int i = 1; i < kWords; ++i) t = __hmax2(t, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
      const float m = fmaxf(__low2float(t), __high2float(t));
      return isnan(m) ? 0u : __float_as_uint(m);
    } else {
      float m = fabsf(at(0));
#pragma unroll
      for (int i = 1; i < 16; ++i) m = fmaxf(m, fabsf(at(i)));
      return isnan(m) ? 0u : __float_as_uint(m);
    }
  }
  // the same of the finite numbers
  __device__ __forceinline__ uint32_t finite_top() const {
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t x = __float_as_uint(at(i)) & 0x7fffffffu;
      t = max(t, x < 0x7f800000u ? x : 0u);
    }
    return t;
  }
  // times `by`, a power of two, to e4m3; kInfinite: infinities become NaN
  template <bool kInfinite = false>
  __device__ __forceinline__ uint4 quantised(float by) const {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = kInfinite && isinf(at(i)) ? NAN : at(i) * by;
    return make_uint4(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]),
                      pack_e4m3x4(x[8], x[9], x[10], x[11]), pack_e4m3x4(x[12], x[13], x[14], x[15]));
  }
};

// The largest over a team, a warp or a block.
template <int kTeam>
__device__ __forceinline__ uint32_t over_team(uint32_t x) {
  x = __reduce_max_sync(0xffffffffu, x);
  if constexpr (kTeam > 32) {
    __shared__ uint32_t tops[kThreads / 32];
    __syncthreads();  // the last call's readers are done
    if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) x = max(x, tops[w]);
  }
  return x;
}

// A team of kTeam threads, a warp or a block, takes one touched block of rows of a sequence and head, of K or V (y).
template <class T, int kTeam>
__global__ void __launch_bounds__(kThreads) append_e4m3_kernel(const AppendParams a) {
  after_stream();
  const uint32_t team = kTeam == 32 ? blockIdx.x * (kThreads / 32) + threadIdx.x / 32 : blockIdx.x;
  const int thread = threadIdx.x % kTeam;
  if (team >= a.teams) return;
  uint32_t nth, g;
  const uint32_t s = a.heads.div(a.many.div(team, &nth), &g);
  const int pool = blockIdx.y;
  const int64_t start = a.start[s];
  int count = a.rows;
  if (a.counts) {
    const int given = a.counts[s];
    if ((given < 0 || given > count) && nth == 0 && g == 0 && pool == 0 && thread == 0) report_pages(a.status);
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

  // the rows do not wait for their page
  const char* src = a.X[pool] + s * a.sb + g * a.sh + (from - start) * a.sn;
  const uint32_t units = (uint32_t)(to - from) * a.row_units.d;
  auto place = [&](uint32_t u, uint32_t* row) {
    uint32_t c;
    *row = a.row_units.div(u, &c);
    return c * 16;
  };
  Unit<T> x[kKeep];
  uint32_t row, top = 0;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const uint32_t u = k * kTeam + thread;
    if (u >= units) continue;
    const uint32_t c = place(u, &row);
    x[k].load(src + row * a.sn + c * sizeof(T), a.wide);
  }
  if (page < 0 || page >= a.num_pages) {
    if (thread == 0) report_pages(a.status);
    return;
  }
  const int row0 = (int)(lo - col * a.page_rows.d);
  uint8_t* dst = a.pages[pool] + page * a.pp + g * a.ph + row0 * a.pn;
  float* scale_at = a.scales[pool] + ((int64_t)page * a.heads.d + g) * (a.page_rows.d / br) + a.block_rows.div(row0);
  const float old = from > lo ? *scale_at : 0.f;
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (k * kTeam + thread < units) top = max(top, x[k].top());
  // a block that is too large to be kept is read twice
  for (uint32_t u = kKeep * kTeam + thread; u < units; u += kTeam) {
    Unit<T> y;
    const uint32_t c = place(u, &row);
    y.load(src + row * a.sn + c * sizeof(T), a.wide);
    top = max(top, y.top());
  }
  top = over_team<kTeam>(top);
  const bool infinite = top >= 0x7f800000u;
  if (infinite) {  // once more, without what is not finite
    top = 0;
#pragma unroll 1
    for (uint32_t u = thread; u < units; u += kTeam) {
      Unit<T> y;
      const uint32_t c = place(u, &row);
      y.load(src + row * a.sn + c * sizeof(T), a.wide);
      top = max(top, y.finite_top());
    }
    top = over_team<kTeam>(top);
  }
  const float scale = fmaxf(scale_for(top), old), inv = inverse(scale);
  // everyone of the team has read the old scale: a warp in step, a block at its barriers
  if (kTeam == 32) __syncwarp();
  if (thread == 0) *scale_at = scale;
  uint8_t* new_rows = dst + (from - lo) * a.pn;
  if (infinite) {
#pragma unroll 1
    for (uint32_t u = thread; u < units; u += kTeam) {
      Unit<T> y;
      const uint32_t c = place(u, &row);
      y.load(src + row * a.sn + c * sizeof(T), a.wide);
      *reinterpret_cast<uint4*>(new_rows + row * a.pn + c) = y.template quantised<true>(inv);
    }
  } else {
#pragma unroll
    for (int k = 0; k < kKeep; ++k) {
      const uint32_t u = k * kTeam + thread;
      if (u >= units) continue;
      const uint32_t c = place(u, &row);
      *reinterpret_cast<uint4*>(new_rows + row * a.pn + c) = x[k].quantised(inv);
    }
    for (uint32_t u = kKeep * kTeam + thread; u < units; u += kTeam) {
      Unit<T> y;
      const uint32_t c = place(u, &row);
      y.load(src + row * a.sn + c * sizeof(T), a.wide);
      *reinterpret_cast<uint4*>(new_rows + row * a.pn + c) = y.quantised(inv);
    }
  }
  if (from > lo && scale > old) {
    const float by = old * inv;
    const uint32_t before = (uint32_t)(from - lo) * a.row_units.d;
    for (uint32_t u = thread; u < before; u += kTeam) {
      const uint32_t c = place(u, &row);
      uint4* at = reinterpret_cast<uint4*>(dst + row * a.pn + c);
      const uint4 q = *at;
      uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 y = e4m3x4_to_float4(w[e]);
        w[e] = pack_e4m3x4(y.x * by, y.y * by, y.z * by, y.w * by);
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
  bool wide;            // rows outside begin on 32 bytes
  int64_t table_stride;
  int64_t sb, sh, sn;   // byte strides of the rows outside
  int64_t pp, ph, pn;   // of the pools
};

// A thread takes 16 numbers, of K and of V.
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
  const int64_t to = s * a.sb + g * a.sh + i * a.sn + c * 16 * (int)sizeof(T);
  uint4 q[2] = {};
  float scale[2] = {};  // where nothing is read: 0 times 0
  if (start >= 0 && (int)i < count) {
    const int64_t pos = start + i;
    const int64_t col = pos < (int64_t(1) << 31) ? (int64_t)a.page_rows.div((uint32_t)pos) : a.max_pages;
    int page = -1;
    if (col < a.max_pages) page = a.table[s * a.table_stride + col];
    if (page >= 0 && page < a.num_pages) {
      const int in_page = (int)(pos - col * a.page_rows.d);
      const int64_t from = page * a.pp + g * a.ph + in_page * a.pn + c * 16;
      const int64_t scale_at =
          ((int64_t)page * a.heads.d + g) * (a.page_rows.d / a.block_rows.d) + a.block_rows.div(in_page);
#pragma unroll
      for (int pool = 0; pool < 2; ++pool) {
        q[pool] = *reinterpret_cast<const uint4*>(a.pages[pool] + from);
        scale[pool] = a.scales[pool][scale_at];
      }
    } else if (c == 0) {
      report_pages(a.status);
    }
  }
#pragma unroll
  for (int pool = 0; pool < 2; ++pool) {
    const uint32_t w[4] = {q[pool].x, q[pool].y, q[pool].z, q[pool].w};
    constexpr int kWords = 16 * sizeof(T) / 4;
    uint32_t out[kWords];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float4 x = e4m3x4_to_float4(w[e]);
      const float by = scale[pool];
      x = make_float4(x.x * by, x.y * by, x.z * by, x.w * by);
      if constexpr (sizeof(T) == 2) {
        out[2 * e] = ptx::pack_bf16x2(x.x, x.y), out[2 * e + 1] = ptx::pack_bf16x2(x.z, x.w);
      } else {
        out[4 * e] = __float_as_uint(x.x), out[4 * e + 1] = __float_as_uint(x.y);
        out[4 * e + 2] = __float_as_uint(x.z), out[4 * e + 3] = __float_as_uint(x.w);
      }
    }
    char* dst = a.X[pool] + to;
    if (a.wide) {
#pragma unroll
      for (int e = 0; e < kWords; e += 8)
        ptx::st_global_v8(dst + 4 * e, out[e], out[e + 1], out[e + 2], out[e + 3], out[e + 4], out[e + 5], out[e + 6], out[e + 7]);
    } else {
#pragma unroll
      for (int e = 0; e < kWords; e += 4)
        *reinterpret_cast<uint4*>(dst + 4 * e) = make_uint4(out[e], out[e + 1], out[e + 2], out[e + 3]);
    }
  }
}

// Whether rows begin on 32 bytes.
bool on_32(const void* K, const void* V, int64_t sb, int64_t sh, int64_t sn) {
  return ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V) | (uint64_t)sb | (uint64_t)sh | (uint64_t)sn) & 31u) == 0;
}

template <class T>
cudaError_t launch_append(const AppendParams& a, int most_units, cudaStream_t s) {
  // a warp keeps kKeep * 32 units
  if (most_units <= kKeep * 32)
    return launch_early(append_e4m3_kernel<T, 32>, dim3((unsigned)ceil_div(a.teams, kThreads / 32), 2), kThreads, 0, s, 1, a);
  return launch_early(append_e4m3_kernel<T, kThreads>, dim3(a.teams, 2), kThreads, 0, s, 1, a);
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
  // a block's units are counted in 32 bits, and a loop over them ends by that
  if ((int64_t)block_rows * (c->d / 16) >= (int64_t(1) << 31)) return FA_ERR_UNSUPPORTED;
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
  a.teams = (uint32_t)((int64_t)c->S * c->H_kv * many);  // many <= rows, so fewer than 2^31
  a.wide = fa::on_32(K, V, a.sb, a.sh, a.sn);
  const int units = (rows < block_rows ? rows : block_rows) * (c->d / 16);
  const cudaStream_t s = (cudaStream_t)stream;
  return fa::status_of(c->dtype == FA_BF16 ? fa::launch_append<__nv_bfloat16>(a, units, s) : fa::launch_append<float>(a, units, s));
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
  a.wide = fa::on_32(K, V, stride_s * es, stride_h * es, stride_n * es);
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
