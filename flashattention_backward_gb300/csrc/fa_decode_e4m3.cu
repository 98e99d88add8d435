// Attention of one new token over a paged key-value cache in 8 bits
// (fa_decode_e4m3): k_j and v_j are stored numbers times the scales of their
// blocks,
//   s_j = scale q . k_j,  m = max_j s_j,  l = sum_j 2^(s_j - m),
//   O = sum_j 2^(s_j - m) v_j / l,  L = (m + log2 l) ln 2
// with scores in units of log 2.

#include "fa_decode.cuh"
#include "fa_e4m3.cuh"

namespace fa {
namespace {

struct SimpleParams {
  const char* Q;
  const uint8_t *K, *V;
  const float *KS, *VS;
  char* O;
  float* L;
  const int32_t *table, *lengths;
  int32_t* status;
  FastDiv page_rows, block_rows;
  int H, group, heads, d, num_pages, max_pages, cap;
  int64_t table_stride, qs, qh, os, oh, pp, ph, pn;
  float scale2;
};

// A block a sequence and query head, a warp a row, 8 columns a lane.
template <class T>
__global__ void __launch_bounds__(128) decode_simple_kernel(const SimpleParams a) {
  after_stream();
  __shared__ float ms[4], ls[4], os[4][256];
  const int s = blockIdx.x / a.H, h = blockIdx.x % a.H, g = h / a.group;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool mine = lane * 8 < a.d;
  int n = a.lengths[s];
  if ((n < 0 || n > a.cap) && threadIdx.x == 0) report_pages(a.status);
  n = min(max(n, 0), a.cap);
  float q[8], acc[8];
  for (int e = 0; e < 8; ++e) {
    const T* row = reinterpret_cast<const T*>(a.Q + s * a.qs + h * a.qh);
    q[e] = mine ? (float)row[lane * 8 + e] * a.scale2 : 0.f;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = warp; j < n; j += 4) {
    uint32_t r;
    const uint32_t col = a.page_rows.div((uint32_t)j, &r);
    const int page = a.table[s * a.table_stride + col];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) report_pages(a.status);
      continue;
    }
    const int64_t at = page * a.pp + g * a.ph + (int64_t)r * a.pn + lane * 8;
    const int64_t sc = ((int64_t)page * a.heads + g) * (a.page_rows.d / a.block_rows.d) + a.block_rows.div(r);
    uint2 k = make_uint2(0, 0), v = make_uint2(0, 0);
    if (mine) k = *reinterpret_cast<const uint2*>(a.K + at), v = *reinterpret_cast<const uint2*>(a.V + at);
    const float4 k0 = e4m3x4_to_float4(k.x), k1 = e4m3x4_to_float4(k.y);
    float x = q[0] * k0.x + q[1] * k0.y + q[2] * k0.z + q[3] * k0.w + q[4] * k1.x + q[5] * k1.y + q[6] * k1.z + q[7] * k1.w;
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= a.KS[sc];
    const float now = fmaxf(m, x), base = base_of(now), alpha = exp2f(m - base), p = exp2f(x - base), w = p * a.VS[sc];
    m = now;
    l = l * alpha + p;
    const float4 v0 = e4m3x4_to_float4(v.x), v1 = e4m3x4_to_float4(v.y);
    const float y[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    for (int e = 0; e < 8; ++e) acc[e] = acc[e] * alpha + w * y[e];
  }
  if (lane == 0) ms[warp] = m, ls[warp] = l;
  if (mine)
    for (int e = 0; e < 8; ++e) os[warp][lane * 8 + e] = acc[e];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, ms[w]);
  const float base = base_of(top);
  for (int w = 0; w < 4; ++w) sum += ls[w] * exp2f(ms[w] - base);
  const bool none = sum == 0.f;
  for (int c = threadIdx.x; c < a.d; c += 128) {
    float o = 0.f;
    for (int w = 0; w < 4; ++w) o += os[w][c] * exp2f(ms[w] - base);
    reinterpret_cast<T*>(a.O + s * a.os + h * a.oh)[c] = (T)(none ? 0.f : o / sum);
  }
  if (threadIdx.x == 0) a.L[(int64_t)s * a.H + h] = none ? INFINITY : (top + log2f(sum)) * kLn2;
}

fa_status check_heads(const fa_cache* c, int32_t block_rows, int32_t H) {
  const fa_status st = check_cache_e4m3(c, block_rows);
  if (st != FA_OK) return st;
  if (H < 1 || H % c->H_kv != 0) return FA_ERR_INVALID_ARG;
  if ((int64_t)c->S * H > (1 << 24) || H / c->H_kv > kMostHeads) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_decode_e4m3_workspace_bytes(const fa_cache* c, int32_t H) { return 0; }

fa_status fa_decode_e4m3(const fa_cache* c, int32_t block_rows, int32_t H, float scale, const void* Q,
                         int64_t q_stride_s, int64_t q_stride_h, const void* K_pages, const void* V_pages,
                         const float* K_scales, const float* V_scales, const int32_t* page_table,
                         const int32_t* lengths, void* O, int64_t o_stride_s, int64_t o_stride_h, float* L,
                         void* workspace, size_t workspace_bytes, void* stream) {
  fa::NvtxRange range("fa_decode_e4m3");
  const fa_status st = fa::check_heads(c, block_rows, H);
  if (st != FA_OK) return st;
  const int es = fa::elem_size(c->dtype);
  if (!(scale > 0.f) || !isfinite(scale * fa::kLog2e) || O == Q || !fa::aligned16(Q) || !fa::aligned16(K_pages) ||
      !fa::aligned16(V_pages) || !fa::aligned4(K_scales) || !fa::aligned4(V_scales) || !fa::aligned16(O) ||
      !fa::aligned4(page_table) || !fa::aligned4(lengths) || !fa::aligned4(L) ||
      !fa::good_stride(q_stride_s, c->d, es, false) || !fa::good_stride(q_stride_h, c->d, es, false) ||
      !fa::good_stride(o_stride_s, c->d, es, true) || !fa::good_stride(o_stride_h, c->d, es, true))
    return FA_ERR_INVALID_ARG;
  fa::SimpleParams a;
  a.status = fa::device_status_word();
  if (!a.status) return FA_ERR_CUDA;
  a.Q = (const char*)Q;
  a.K = (const uint8_t*)K_pages;
  a.V = (const uint8_t*)V_pages;
  a.KS = K_scales;
  a.VS = V_scales;
  a.O = (char*)O;
  a.L = L;
  a.table = page_table;
  a.lengths = lengths;
  a.page_rows = fa::FastDiv(c->page_rows);
  a.block_rows = fa::FastDiv(block_rows);
  a.H = H;
  a.group = H / c->H_kv;
  a.heads = c->H_kv;
  a.d = c->d;
  a.num_pages = c->num_pages;
  a.max_pages = c->max_pages;
  a.cap = (int)fa::cache_rows(*c);
  a.table_stride = c->table_stride;
  a.qs = q_stride_s * es;
  a.qh = q_stride_h * es;
  a.os = o_stride_s * es;
  a.oh = o_stride_h * es;
  a.pp = c->stride_page;
  a.ph = c->stride_h;
  a.pn = c->stride_n;
  a.scale2 = scale * fa::kLog2e;
  const dim3 grid((unsigned)(c->S * H));
  const cudaStream_t s = (cudaStream_t)stream;
  return fa::status_of(c->dtype == FA_BF16
                           ? fa::launch_early(fa::decode_simple_kernel<__nv_bfloat16>, grid, 128, 0, s, 1, a)
                           : fa::launch_early(fa::decode_simple_kernel<float>, grid, 128, 0, s, 1, a));
}

}  // extern "C"
