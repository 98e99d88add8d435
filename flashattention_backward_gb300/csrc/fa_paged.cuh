// Shared by the paged-cache translation units (fa_decode.cu, fa_cache.cu,
// fa_pages.cu): exact division by a number known at launch, host checks of a
// fa_cache, and the report of a bad page.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_internal.h"

namespace fa {

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 as one multiply-high, an addition
// and a shift: with s = ceil(log2 d) and m = floor(2^32 (2^s - d) / d) + 1,
// floor(n / d) = (mulhi(n, m) + n) >> s (the round-up method of Granlund and
// Montgomery; the sum stays below 2^32 because mulhi(n, m) <= n).
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), s(0) {
    while ((1ull << s) < div) ++s;
    m = (uint32_t)((((1ull << s) - div) << 32) / div + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
  __device__ __forceinline__ uint32_t div(uint32_t n, uint32_t* rem) const {
    const uint32_t q = div(n);
    *rem = n - q * d;
    return q;
  }
};

inline bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int elem_size(int32_t dtype) { return dtype == FA_BF16 ? 2 : 4; }
inline int64_t cache_rows(const fa_cache& c) { return (int64_t)c.page_rows * c.max_pages; }

// The table's geometry: what the page calls read.
inline fa_status check_pages(const fa_cache* c) {
  if (!c || c->num_pages < 1 || c->page_rows < 1 || c->S < 1 || c->max_pages < 1 || c->H_kv < 1 || c->reserved != 0 ||
      c->table_stride < c->max_pages)
    return FA_ERR_INVALID_ARG;
  if (c->num_pages > (1 << 30) || cache_rows(*c) > (1 << 30) || (int64_t)c->S * c->H_kv > (1 << 24))
    return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// One row-shaped operand's strides: no two rows may overlap where it is
// written, and every row starts on 16 bytes.
inline bool good_stride(int64_t stride, int d, int es, bool written) {
  return stride >= (written ? d : 0) && stride < (int64_t(1) << 48) && (stride * es) % 16 == 0;
}

// es: bytes of an element of the pools.
inline fa_status check_pools(const fa_cache* c, int es) {
  const fa_status st = check_pages(c);
  if (st != FA_OK) return st;
  if (c->dtype != FA_BF16 && c->dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  const bool known = c->d == 32 || c->d == 64 || c->d == 96 || c->d == 128 || c->d == 256;
  if (!known && !(c->d == 16 && c->dtype == FA_FP32)) return FA_ERR_UNSUPPORTED;
  if (!good_stride(c->stride_page, c->d, es, true) || !good_stride(c->stride_h, c->d, es, true) ||
      !good_stride(c->stride_n, c->d, es, true))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}
inline fa_status check_cache(const fa_cache* c) {
  return check_pools(c, c && c->dtype == FA_BF16 ? 2 : 4);
}
// Pools in 8 bits with a scale for every block_rows rows.
inline fa_status check_cache_e4m3(const fa_cache* c, int32_t block_rows) {
  const fa_status st = check_pools(c, 1);
  if (st != FA_OK) return st;
  if (block_rows < 1 || c->page_rows % block_rows != 0) return FA_ERR_INVALID_ARG;
  // a page's scales are counted in 32 bits
  return (int64_t)c->H_kv * (c->page_rows / block_rows) < (int64_t(1) << 31) ? FA_OK : FA_ERR_UNSUPPORTED;
}

inline fa_status status_of(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// SMs of the current device (looked up once per device).
int sm_count();

// Launches so that the kernel's blocks may be on the GPU before the kernel in
// front of it on the stream has ended: they wait for that themselves, with
// after_stream(), before they touch memory.  Without it a call starts 2 us
// later when calls follow one another: one sequence of 32768 rows, 8 heads of
// d 128, took 30.9 us a call and takes 28.5, one row appended to 64 sequences 5.7 and
// 3.3, five calls of a fork 25.6 and 14.4.  At least one block of every kernel has to
// wait: what comes next on the stream waits for this kernel alone.
// What work in front may have written is read with plain loads, never with
// __ldg or through const __restrict__: a load on the non-coherent path promises
// that its data does not change while the kernel runs, and these kernels run
// from before that work has ended; nor does after_stream() hold such a load back.
template <class... P, class... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, int cluster,
                                A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
__device__ __forceinline__ void after_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's blocks line up; after after_stream(), so that what was
// in front of this kernel is done for them too.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void report_pages(int32_t* status) { atomicCAS(status, 0, (int32_t)FA_ERR_PAGES); }

}  // namespace fa
