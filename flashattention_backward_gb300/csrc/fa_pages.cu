// The page calls of the paged cache: fa_pages_extend, fa_pages_fork,
// fa_pages_free and fa_pages_compact.  They work on the page table, the
// lengths and the reference counts alone (include/fa.h says what each does).
//
// Which page goes where is a prefix sum: the k-th free page, in rising order,
// goes to the k-th demand, in the order of the sequences or pairs.  So the
// result does not depend on the order in which threads run, and there is no
// free list to keep.  One thread block does it: the arrays are a few hundred
// kilobytes at most in ordinary use (4 bytes a page), and what bounds the
// calls is the latency of a handful of dependent passes, not bandwidth.

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_paged.cuh"

namespace fa {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 4;                      // pages a thread looks at per step of a scan
constexpr int kStep = kThreads * kPer;

struct Pages {
  int32_t num_pages, page_rows, S, max_pages;
  int32_t rows;          // of a sequence at most: page_rows * max_pages
  FastDiv by_page_rows;
  int64_t table_stride;
  int32_t* status;
  // pages that n rows take, 0 <= n <= rows
  __device__ __forceinline__ int pages(int n) const { return (int)by_page_rows.div((uint32_t)(n + page_rows - 1)); }
};

// Exclusive prefix sum of one number a thread over the block; *total is the
// block's sum.  sums: kWarps + 1 ints of shared memory.  Every thread calls it.
__device__ __forceinline__ int block_scan(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();  // the last call's readers of sums are done
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  if (warp == 0) {
    int s = sums[lane];  // kWarps == 32
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += z;
    }
    sums[lane] = s;
  }
  __syncthreads();
  *total = sums[kWarps - 1];
  return y - x + (warp ? sums[warp - 1] : 0);
}
static_assert(kWarps == 32, "block_scan sums one number a warp with one warp");

// Visits the pages p in [first, last) for which pick(p) holds, in rising
// order of p, as take(p, rank) with rank counting from 0, until `most` have
// been taken; returns how many there are (at least `most` when it stopped
// early).  Element p of a step is seen by lane p % 32 of warp p / 128: a
// warp's loads are whole lines at any alignment, and ballots give the rank.
template <class Pick, class Take>
__device__ __forceinline__ int rank_pages(int first, int last, int most, int* sums, Pick pick, Take take) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int done = 0;
  for (int64_t base = first; base < last && done < most; base += kStep) {
    unsigned seen[kPer];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int64_t p = base + warp * 32 * kPer + j * 32 + lane;
      seen[j] = __ballot_sync(0xffffffffu, p < last && pick((int)p));
      mine += __popc(seen[j]);
    }
    int total;
    // the scan counts a warp's pages once, on its last lane
    int rank = block_scan(lane == 31 ? mine : 0, sums, &total);
    rank = done + __shfl_sync(0xffffffffu, rank, 31);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int r = rank + __popc(seen[j] & ((1u << lane) - 1));
      if (((seen[j] >> lane) & 1) && r < most) take((int)(base + warp * 32 * kPer + j * 32 + lane), r);
      rank += __popc(seen[j]);
    }
    done += total;
  }
  return done;
}

__global__ void __launch_bounds__(kThreads, 1) pages_extend_kernel(const Pages g, int32_t* table, int32_t* lengths,
                                                                int32_t* refs, const int32_t* n_new, int32_t* start,
                                                                int32_t* scratch) {
  __shared__ int sums[kWarps];
  __shared__ unsigned long long wanted;
  int32_t* free_pages = scratch;                // [num_pages]
  __shared__ int first_of_few[kThreads];
  // [S]: pages wanted by the sequences before
  int32_t* first_of = g.S <= kThreads ? first_of_few : scratch + g.num_pages;
  if (threadIdx.x == 0) wanted = 0;
  __syncthreads();
  bool bad = false;
  int before = 0;
  for (int base = 0; base < g.S; base += kThreads) {
    const int s = base + threadIdx.x;
    int need = 0;
    if (s < g.S) {
      const int n = lengths[s], more = n_new[s];
      if (n < 0 || more < 0 || (int64_t)n + more > g.rows)
        bad = true;
      else
        need = g.pages(n + more) - g.pages(n);
    }
    // more than there are pages: the call is refused below, and the prefix
    // sums in 32 bits may then wrap without being used
    if (need) atomicAdd(&wanted, (unsigned long long)need);
    int total;
    const int rank = block_scan(need, sums, &total);
    if (s < g.S) first_of[s] = before + rank;
    before += total;
  }
  bool refused = __syncthreads_or(bad) || wanted > (unsigned long long)g.num_pages;
  const int want = refused ? 0 : (int)wanted;
  if (!refused && want > 0)
    refused = rank_pages(0, g.num_pages, want, sums, [&](int p) { return refs[p] <= 0; },
                         [&](int p, int r) { free_pages[r] = p; }) < want;
  if (refused) {
    for (int s = threadIdx.x; s < g.S; s += kThreads) start[s] = -1;
    if (threadIdx.x == 0) report_pages(g.status);
    return;
  }
  __syncthreads();  // free_pages and first_of are read across threads
  // k-th new page: of the last sequence whose first one is at or before k
  for (int k = threadIdx.x; k < want; k += kThreads) {
    int lo = 0, hi = g.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_of[mid] <= k)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int page = free_pages[k];
    table[lo * g.table_stride + g.pages(lengths[lo]) + (k - first_of[lo])] = page;
    refs[page] = 1;
  }
  __syncthreads();  // lengths above are the ones before the call
  for (int s = threadIdx.x; s < g.S; s += kThreads) {
    const int n = lengths[s];
    start[s] = n;
    lengths[s] = n + n_new[s];
  }
}

// Calls f(i, a, b, rows of a) with one warp a pair, kThreads pairs at a time:
// the indexes and lengths of a batch are loaded by a thread each and read from
// shared memory, so that a warp's pairs do not wait for one another's loads.
struct PairBatch {
  int src[kThreads], dst[kThreads], rows[kThreads];
};
template <class F>
__device__ __forceinline__ void for_pairs(int pairs, const int32_t* src, const int32_t* dst, const int32_t* lengths,
                                          PairBatch* batch, F f) {
  for (int base = 0; base < pairs; base += kThreads) {
    const int i = base + threadIdx.x;
    __syncthreads();  // the last batch has been read
    if (i < pairs) {
      batch->src[threadIdx.x] = src[i];
      batch->dst[threadIdx.x] = dst[i];
      batch->rows[threadIdx.x] = lengths[src[i]];
    }
    __syncthreads();
    const int n = min(pairs - base, kThreads);
#pragma unroll 4
    for (int k = threadIdx.x >> 5; k < n; k += kWarps) f(base + k, batch->src[k], batch->dst[k], batch->rows[k]);
  }
}

__global__ void __launch_bounds__(kThreads, 1) pages_fork_kernel(const Pages g, int pairs, const int32_t* src,
                                                              const int32_t* dst, int32_t* table, int32_t* lengths,
                                                              int32_t* refs, int32_t* moves, int32_t* scratch) {
  __shared__ int sums[kWarps];
  __shared__ PairBatch batch;
  int32_t* free_pages = scratch;             // [num_pages]
  int32_t* mark = scratch + g.num_pages;     // [S]: 1 a source, 2 a destination
  const int lane = threadIdx.x & 31;
  for (int s = threadIdx.x; s < g.S; s += kThreads) mark[s] = 0;
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= g.S || b < 0 || b >= g.S) {
      bad = true;
      continue;
    }
    const int rows = lengths[a], none = lengths[b];
    atomicOr(&mark[a], 1);
    bad |= (atomicOr(&mark[b], 2) & 2) || rows < 0 || rows > g.rows || none != 0;
  }
  bool refused = __syncthreads_or(bad);
  int tails = 0;
  if (!refused) {
    for (int s = threadIdx.x; s < g.S; s += kThreads) bad |= mark[s] == 3;
    // a source's entries are followed below: look at them before anything changes
    for_pairs(pairs, src, dst, lengths, &batch, [&](int, int a, int, int rows) {
      const int held = g.pages(rows);
      for (int c = lane; c < held; c += 32) {
        const int p = table[a * g.table_stride + c];
        bad |= p < 0 || p >= g.num_pages;
      }
    });
    for (int base = 0; base < pairs; base += kThreads) {
      const int i = base + threadIdx.x;
      int tail = 0;
      if (i < pairs) {
        uint32_t rest;
        g.by_page_rows.div((uint32_t)lengths[src[i]], &rest);
        tail = rest != 0;
      }
      int total;
      const int rank = block_scan(tail, sums, &total);
      if (i < pairs) moves[3 * (int64_t)i + 1] = tails + rank;
      tails += total;
    }
    refused = __syncthreads_or(bad);
    if (!refused && tails > 0)
      refused = rank_pages(0, g.num_pages, tails, sums, [&](int p) { return refs[p] <= 0; },
                           [&](int p, int r) { free_pages[r] = p; }) < tails;
  }
  __syncthreads();
  if (refused) {
    for (int64_t i = threadIdx.x; i < 3 * (int64_t)pairs; i += kThreads) moves[i] = -1;
    if (threadIdx.x == 0) report_pages(g.status);
    return;
  }
  // no source is a destination: nothing read here is written here
  for_pairs(pairs, src, dst, lengths, &batch, [&](int i, int a, int b, int rows) {
    uint32_t rest;
    const int full = (int)g.by_page_rows.div((uint32_t)rows, &rest);
    for (int c = lane; c < full; c += 32) {
      const int p = table[a * g.table_stride + c];
      table[b * g.table_stride + c] = p;
      atomicAdd(&refs[p], 1);
    }
    if (lane == 0) {
      int from = -1, to = -1;
      if (rest) {
        from = table[a * g.table_stride + full];
        to = free_pages[moves[3 * (int64_t)i + 1]];
        table[b * g.table_stride + full] = to;
        refs[to] = 1;  // a free page: in no table, so no other thread counts it
      }
      moves[3 * (int64_t)i] = from;
      moves[3 * (int64_t)i + 1] = to;
      moves[3 * (int64_t)i + 2] = rest ? (int)rest : -1;
      lengths[b] = rows;
    }
  });
}

// One block a listed sequence.
__global__ void __launch_bounds__(128) pages_free_kernel(const Pages g, const int32_t* list, int32_t* table,
                                                         int32_t* lengths, int32_t* refs) {
  __shared__ int rows;
  const int s = list[blockIdx.x];
  if (s < 0 || s >= g.S) {
    if (s != -1 && threadIdx.x == 0) report_pages(g.status);
    return;
  }
  // whoever comes first of a sequence listed twice takes its length; the
  // other finds it empty
  if (threadIdx.x == 0) rows = atomicExch(&lengths[s], 0);
  __syncthreads();
  bool bad = rows < 0 || rows > g.rows;
  const int held = g.pages(min(max(rows, 0), g.rows));
  for (int c = threadIdx.x; c < held; c += blockDim.x) {
    int32_t* e = &table[s * g.table_stride + c];
    const int p = *e;
    *e = -1;
    if (p < 0 || p >= g.num_pages) {
      bad = true;
    } else if (atomicSub(&refs[p], 1) <= 0) {  // more names than it was counted for
      atomicAdd(&refs[p], 1);
      bad = true;
    }
  }
  if (bad) report_pages(g.status);
}

__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const Pages g, const int32_t* refs, int32_t* refs_out,
                                                                 int32_t* moves, int32_t* n_moves, int32_t* scratch) {
  __shared__ int sums[kWarps];
  int32_t* to = scratch;                    // [num_pages]: where a page goes
  int32_t* holes = scratch + g.num_pages;   // [num_pages / 2]
  const auto used = [&](int p) { return refs[p] > 0; };
  int mine = 0, n;
  for (int p = threadIdx.x; p < g.num_pages; p += kThreads) {
    const bool live = used(p);
    to[p] = live ? p : -1;
    mine += live;
  }
  block_scan(mine, sums, &n);
  // free pages before n, rising; a page that stays keeps its count
  rank_pages(0, n, n, sums, [&](int p) { return refs[p] <= 0; }, [&](int p, int r) { holes[r] = p; });
  __syncthreads();
  if (refs_out != refs)
    for (int p = threadIdx.x; p < n; p += kThreads) refs_out[p] = refs[p];
  __syncthreads();  // the holes' zeros before the counts that move into them
  // pages in use at n or behind: as many as there are holes
  const int count = rank_pages(n, g.num_pages, g.num_pages, sums, used, [&](int p, int r) {
    const int d = holes[r];
    to[p] = d;
    moves[3 * (int64_t)r] = p;
    moves[3 * (int64_t)r + 1] = d;
    moves[3 * (int64_t)r + 2] = g.page_rows;
    refs_out[d] = refs[p];
  });
  __syncthreads();  // counts behind n are read above
  for (int p = n + threadIdx.x; p < g.num_pages; p += kThreads) refs_out[p] = 0;
  const int64_t end = 3 * (int64_t)(g.num_pages / 2);
  for (int64_t i = 3 * (int64_t)count + threadIdx.x; i < end; i += kThreads) moves[i] = -1;
  if (threadIdx.x == 0) *n_moves = count;
}

// Table entries after a compaction: one block a sequence.  An entry that
// names a page that refs calls free is damaged and becomes -1.
__global__ void __launch_bounds__(128) pages_rename_kernel(const Pages g, const int32_t* table,
                                                           const int32_t* lengths, const int32_t* to,
                                                           int32_t* table_out) {
  const int64_t row = blockIdx.x * g.table_stride;
  const int n = lengths[blockIdx.x];
  bool bad = n < 0 || n > g.rows;
  const int held = g.pages(min(max(n, 0), g.rows));
  for (int c = threadIdx.x; c < g.max_pages; c += blockDim.x) {
    int p = -1;
    if (c < held) {
      p = table[row + c];
      p = p < 0 || p >= g.num_pages ? -1 : to[p];
      bad |= p < 0;
    }
    table_out[row + c] = p;
  }
  if (bad) report_pages(g.status);
}

bool geometry(const fa_cache& c, Pages* g) {
  g->num_pages = c.num_pages;
  g->page_rows = c.page_rows;
  g->S = c.S;
  g->max_pages = c.max_pages;
  g->rows = (int32_t)cache_rows(c);
  g->by_page_rows = FastDiv(c.page_rows);
  g->table_stride = c.table_stride;
  g->status = device_status_word();
  return g->status != nullptr;
}

}  // namespace
}  // namespace fa

extern "C" {

size_t fa_pages_scratch_elems(const fa_cache* c) {
  if (fa::check_pages(c) != FA_OK) return 0;
  return (size_t)c->num_pages + (size_t)(c->num_pages > c->S ? c->num_pages : c->S);
}

fa_status fa_pages_extend(const fa_cache* c, int32_t* page_table, int32_t* lengths, int32_t* refs,
                          const int32_t* n_new, int32_t* start, int32_t* scratch, void* stream) {
  fa::NvtxRange range("fa_pages_extend");
  const fa_status st = fa::check_pages(c);
  if (st != FA_OK) return st;
  if (!fa::aligned4(page_table) || !fa::aligned4(lengths) || !fa::aligned4(refs) || !fa::aligned4(n_new) ||
      !fa::aligned4(start) || !fa::aligned4(scratch))
    return FA_ERR_INVALID_ARG;
  fa::Pages g;
  if (!fa::geometry(*c, &g)) return FA_ERR_CUDA;
  fa::pages_extend_kernel<<<1, fa::kThreads, 0, (cudaStream_t)stream>>>(g, page_table, lengths, refs, n_new, start,
                                                                        scratch);
  return fa::status_of(cudaGetLastError());
}

fa_status fa_pages_fork(const fa_cache* c, int32_t pairs, const int32_t* src, const int32_t* dst, int32_t* page_table,
                        int32_t* lengths, int32_t* refs, int32_t* moves, int32_t* scratch, void* stream) {
  fa::NvtxRange range("fa_pages_fork");
  const fa_status st = fa::check_pages(c);
  if (st != FA_OK) return st;
  if (pairs < 1 || pairs > c->S || !fa::aligned4(src) || !fa::aligned4(dst) || !fa::aligned4(page_table) ||
      !fa::aligned4(lengths) || !fa::aligned4(refs) || !fa::aligned4(moves) || !fa::aligned4(scratch))
    return FA_ERR_INVALID_ARG;
  fa::Pages g;
  if (!fa::geometry(*c, &g)) return FA_ERR_CUDA;
  fa::pages_fork_kernel<<<1, fa::kThreads, 0, (cudaStream_t)stream>>>(g, pairs, src, dst, page_table, lengths, refs,
                                                                      moves, scratch);
  return fa::status_of(cudaGetLastError());
}

fa_status fa_pages_free(const fa_cache* c, int32_t count, const int32_t* sequences, int32_t* page_table,
                        int32_t* lengths, int32_t* refs, void* stream) {
  fa::NvtxRange range("fa_pages_free");
  const fa_status st = fa::check_pages(c);
  if (st != FA_OK) return st;
  if (count < 0 || (count > 0 && !fa::aligned4(sequences)) || !fa::aligned4(page_table) || !fa::aligned4(lengths) ||
      !fa::aligned4(refs))
    return FA_ERR_INVALID_ARG;
  fa::Pages g;
  if (!fa::geometry(*c, &g)) return FA_ERR_CUDA;
  if (count == 0) return FA_OK;
  fa::pages_free_kernel<<<count, 128, 0, (cudaStream_t)stream>>>(g, sequences, page_table, lengths, refs);
  return fa::status_of(cudaGetLastError());
}

fa_status fa_pages_compact(const fa_cache* c, const int32_t* page_table, const int32_t* lengths, const int32_t* refs,
                           int32_t* table_out, int32_t* refs_out, int32_t* moves, int32_t* n_moves, int32_t* scratch,
                           void* stream) {
  fa::NvtxRange range("fa_pages_compact");
  const fa_status st = fa::check_pages(c);
  if (st != FA_OK) return st;
  if (!fa::aligned4(page_table) || !fa::aligned4(lengths) || !fa::aligned4(refs) || !fa::aligned4(table_out) ||
      !fa::aligned4(refs_out) || (c->num_pages > 1 && !fa::aligned4(moves)) || !fa::aligned4(n_moves) ||
      !fa::aligned4(scratch))
    return FA_ERR_INVALID_ARG;
  fa::Pages g;
  if (!fa::geometry(*c, &g)) return FA_ERR_CUDA;
  const cudaStream_t s = (cudaStream_t)stream;
  fa::pages_compact_kernel<<<1, fa::kThreads, 0, s>>>(g, refs, refs_out, moves, n_moves, scratch);
  fa::pages_rename_kernel<<<c->S, 128, 0, s>>>(g, page_table, lengths, scratch, table_out);
  return fa::status_of(cudaGetLastError());
}

}  // extern "C"
