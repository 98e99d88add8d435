// Attention of one new token over a paged key-value cache (fa_decode).
//
//   s_j = scale q . k_j,  m = max_j s_j,  l = sum_j exp(s_j - m),
//   O = sum_j exp(s_j - m) v_j / l,  L = m + log l.
//
// One block per (sequence, query head).  Its warps take the rows of the cache
// in turn, each with a running maximum and sum of its own (a row that raises
// the maximum rescales what has been summed), and are joined at the end.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  const void *Q, *K, *V;
  void* O;
  float* L;
  const int32_t *table, *lengths;
  int32_t* status;
  FastDiv page_rows;
  int H, group, num_pages, max_pages;
  int64_t table_stride, rows;
  int64_t qs, qh, os, oh;   // element strides
  int64_t pp, ph, pn;
  float scale2;             // scale * log2(e)
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps) decode_kernel(const DecodeParams a) {
  constexpr int E = (D + 31) / 32;  // columns a lane holds: lane, lane + 32, ...
  __shared__ float part[kWarps][D], ms[kWarps], ls[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.x / a.H, h = blockIdx.x % a.H, g = h / a.group;
  int64_t n = __ldg(a.lengths + s);
  if ((n < 0 || n > a.rows) && threadIdx.x == 0) report_pages(a.status);
  n = n < 0 ? 0 : (n > a.rows ? a.rows : n);
  const T* q = (const T*)a.Q + s * a.qs + h * a.qh;
  float qv[E], o[E] = {};
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = lane + 32 * e < D ? to_f(q[lane + 32 * e]) : 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < n; j += kWarps) {
    uint32_t r;
    const uint32_t col = a.page_rows.div(j, &r);
    const int page = __ldg(a.table + s * a.table_stride + col);
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) report_pages(a.status);
      continue;
    }
    const int64_t at = page * a.pp + g * a.ph + (int64_t)r * a.pn;
    float x = 0.f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = lane + 32 * e;
      x = fmaf(c < D ? to_f(((const T*)a.K)[at + c]) : 0.f, qv[e], x);
      v[e] = c < D ? to_f(((const T*)a.V)[at + c]) : 0.f;
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= a.scale2;
    const float mn = fmaxf(m, x), mb = mn == -INFINITY ? 0.f : mn;
    const float alpha = exp2f(m - mb), p = exp2f(x - mb);
    l = l * alpha + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * alpha + p * v[e];
    m = mn;
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (lane + 32 * e < D) part[warp][lane + 32 * e] = o[e];
  if (lane == 0) ms[warp] = m, ls[warp] = l;
  __syncthreads();
  float M = -INFINITY, sum = 0.f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ms[w]);
  const float Mb = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = exp2f(ms[w] - Mb);
    sum += f[w] * ls[w];
  }
  const bool empty = sum == 0.f;
  for (int c = threadIdx.x; c < D; c += 32 * kWarps) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += f[w] * part[w][c];
    put((T*)a.O + s * a.os + h * a.oh + c, empty ? 0.f : x / sum);
  }
  if (threadIdx.x == 0) a.L[blockIdx.x] = empty ? INFINITY : (M + log2f(sum)) * kLn2;
}

template <class T>
cudaError_t launch(const fa_cache& c, const DecodeParams& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(c.S * a.H);
  switch (c.d) {
    case 16: decode_kernel<T, 16><<<grid, 32 * kWarps, 0, s>>>(a); break;
    case 32: decode_kernel<T, 32><<<grid, 32 * kWarps, 0, s>>>(a); break;
    case 64: decode_kernel<T, 64><<<grid, 32 * kWarps, 0, s>>>(a); break;
    case 96: decode_kernel<T, 96><<<grid, 32 * kWarps, 0, s>>>(a); break;
    case 128: decode_kernel<T, 128><<<grid, 32 * kWarps, 0, s>>>(a); break;
    case 256: decode_kernel<T, 256><<<grid, 32 * kWarps, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
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
  return 0;
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
  fa::DecodeParams a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  a.Q = Q;
  a.K = K_pages;
  a.V = V_pages;
  a.O = O;
  a.L = L;
  a.table = page_table;
  a.lengths = lengths;
  a.page_rows = fa::FastDiv(c->page_rows);
  a.H = H;
  a.group = H / c->H_kv;
  a.num_pages = c->num_pages;
  a.max_pages = c->max_pages;
  a.table_stride = c->table_stride;
  a.rows = fa::cache_rows(*c);
  a.qs = q_stride_s;
  a.qh = q_stride_h;
  a.os = o_stride_s;
  a.oh = o_stride_h;
  a.pp = c->stride_page;
  a.ph = c->stride_h;
  a.pn = c->stride_n;
  a.scale2 = scale * fa::kLog2e;
  const cudaStream_t s = (cudaStream_t)stream;
  return fa::status_of(c->dtype == FA_BF16 ? fa::launch<__nv_bfloat16>(*c, a, s) : fa::launch<float>(*c, a, s));
}

}  // extern "C"
