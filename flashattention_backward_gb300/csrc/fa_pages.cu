// The page calls of the paged cache: fa_pages_extend, fa_pages_fork,
// fa_pages_free and fa_pages_compact.  They work on the page table, the
// lengths and the reference counts alone (include/fa.h says what each does).
//
// Which page goes where is a prefix sum: the k-th free page, in rising order,
// goes to the k-th demand, in the order of the sequences or pairs.  So the
// result does not depend on the order in which threads run, and there is no
// free list to keep.  One thread block does it (a cluster in pages_fork): the
// arrays are a few hundred kilobytes at most in ordinary use (4 bytes a page),
// and what bounds the calls is the latency of a handful of dependent passes,
// not bandwidth.
//
// Measured (ncu, cold caches, launch included): extend 9.2 to 9.5 us for 256
// sequences and a pool of 2000 pages, fork 10.4 to 11.0 us for 224 pairs of up to 63 pages,
// free 6.2 to 6.9 us for the same, compact 9.3 to 9.5 us and 8.4 to 9.1 us for 8192 pages
// and a table of 64 x 64.

#include <cooperative_groups.h>
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
// block's sum.  sums: kWarps numbers of shared memory.  Every thread calls it.
template <class T>
__device__ __forceinline__ T block_scan(T x, T* sums, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T z = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) y += z;
  }
  __syncthreads();  // the last call's readers of sums are done
  if (lane == 31) sums[warp] = y;
  __syncthreads();
  if (warp == 0) {
    T s = sums[lane];  // kWarps == 32
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T z = __shfl_up_sync(0xffffffffu, s, o);
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
                                                                   int32_t* refs, const int32_t* n_new,
                                                                   int32_t* start) {
  __shared__ int sums[kWarps];
  __shared__ unsigned long long wanted;
  __shared__ int first_of_few[kThreads];
  // [S]: pages wanted by the sequences before; many of them are kept in `start`,
  // whose values are only known at the end
  int* first_of = g.S <= kThreads ? first_of_few : start;
  after_stream();
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
  // the k-th new page belongs to the last sequence whose first one is at or before k
  const auto entry = [&](int k) -> int32_t* {
    int lo = 0, hi = g.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first_of[mid] <= k)
        lo = mid;
      else
        hi = mid - 1;
    }
    return &table[lo * g.table_stride + g.pages(lengths[lo]) + (k - first_of[lo])];
  };
  if (want > 0) {
    const int found = rank_pages(0, g.num_pages, want, sums, [&](int p) { return refs[p] <= 0; }, [&](int p, int k) {
      *entry(k) = p;
      refs[p] = 1;
    });
    if (found < want) {  // too few: give them back
      refused = true;
      __syncthreads();
      for (int k = threadIdx.x; k < found; k += kThreads) {
        int32_t* e = entry(k);
        refs[*e] = 0;
        *e = -1;
      }
    }
    __syncthreads();  // lengths and first_of above are the ones before the call
  }
  for (int s = threadIdx.x; s < g.S; s += kThreads) {
    if (refused) {
      start[s] = -1;
    } else {
      const int n = lengths[s];
      start[s] = n;
      lengths[s] = n + n_new[s];
    }
  }
  if (refused && threadIdx.x == 0) report_pages(g.status);
}

// A cluster of kForkBlocks blocks.  All of them work out the same plan (who gets
// which free page), which only reads what the call changes; then, with the
// cluster's barrier between, each looks at and copies the table rows of its
// share of the pairs.  The references are what costs: one SM sends about one
// scattered atomic a cycle, 3.7 us for 224 pairs of 32 pages; in one block the
// call took 17 us.
// marks: two bits a sequence in shared memory, whether it is a source and
// whether it is a destination.
constexpr int kForkBlocks = 8;

__global__ void __launch_bounds__(kThreads, 1)
    pages_fork_kernel(const Pages g, int pairs, const int32_t* src, const int32_t* dst, int32_t* table,
                      int32_t* lengths, int32_t* refs, int32_t* moves) {
  namespace cg = cooperative_groups;
  __shared__ int sums[kWarps];
  __shared__ int any_bad;      // of the cluster, in block 0
  extern __shared__ unsigned marks[];  // 16 sequences a word
  const cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const int first = blockIdx.x * kWarps + (threadIdx.x >> 5), step = kForkBlocks * kWarps;  // this warp's pairs
  after_stream();
  for (int w = threadIdx.x; w < (g.S + 15) / 16; w += kThreads) marks[w] = 0;
  if (threadIdx.x == 0) any_bad = 0;
  cluster.sync();
  bool bad = false;
  for (int i = threadIdx.x; i < pairs; i += kThreads) {
    const int a = src[i], b = dst[i];
    if (a < 0 || a >= g.S || b < 0 || b >= g.S) {
      bad = true;
      continue;
    }
    const int rows = lengths[a], none = lengths[b];
    atomicOr(&marks[a / 16], 1u << (a % 16 * 2));
    const unsigned is_dst = 2u << (b % 16 * 2);
    bad |= (atomicOr(&marks[b / 16], is_dst) & is_dst) || rows < 0 || rows > g.rows || none != 0;
  }
  bool refused = __syncthreads_or(bad);  // the same in all blocks
  int tails = 0;
  if (!refused) {
    for (int w = threadIdx.x; w < (g.S + 15) / 16; w += kThreads) bad |= (marks[w] & (marks[w] >> 1) & 0x55555555u) != 0;
    // a source's entries are followed below: look at them before anything changes
    for (int i = first; i < pairs; i += step) {
      const int a = src[i], held = g.pages(lengths[a]);
      for (int c = lane; c < held; c += 32) {
        const int p = table[a * g.table_stride + c];
        // nor may it name a free page, which could be handed out below
        bad |= p < 0 || p >= g.num_pages || refs[p] <= 0;
      }
    }
    if (bad) atomicOr(cluster.map_shared_rank(&any_bad, 0), 1);
    // the k-th pair with a partly filled page gets the k-th free page: until
    // then the first number of move k says which pair that is.  All blocks
    // write the same numbers.
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
      if (tail) moves[3 * (int64_t)(tails + rank)] = i;
      tails += total;
    }
    __syncthreads();
    if (tails > 0)
      refused = rank_pages(0, g.num_pages, tails, sums, [&](int p) { return refs[p] <= 0; }, [&](int p, int k) {
                  moves[3 * (int64_t)moves[3 * (int64_t)k] + 1] = p;
                }) < tails;
  }
  cluster.sync();  // every block has its plan: what it was made from may change
  refused |= *cluster.map_shared_rank(&any_bad, 0) != 0;
  cluster.sync();  // block 0's flag has been read
  if (refused) {
    if (blockIdx.x == 0) {
      for (int64_t i = threadIdx.x; i < 3 * (int64_t)pairs; i += kThreads) moves[i] = -1;
      if (threadIdx.x == 0) report_pages(g.status);
    }
    return;
  }
  // no source is a destination: nothing read here is written here
  for (int i = first; i < pairs; i += step) {
    const int a = src[i], b = dst[i], rows = lengths[a];
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
        to = moves[3 * (int64_t)i + 1];
        table[b * g.table_stride + full] = to;
        refs[to] = 1;  // a free page: in no table, so no other thread counts it
      }
      moves[3 * (int64_t)i] = from;
      moves[3 * (int64_t)i + 1] = to;
      moves[3 * (int64_t)i + 2] = rest ? (int)rest : -1;
      lengths[b] = rows;
    }
  }
}

// One block a listed sequence.
__global__ void __launch_bounds__(128) pages_free_kernel(const Pages g, const int32_t* list, int32_t* table,
                                                         int32_t* lengths, int32_t* refs) {
  __shared__ int rows;
  after_stream();
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

__global__ void __launch_bounds__(kThreads, 1) pages_compact_kernel(const Pages g, const int32_t* refs,
                                                                    int32_t* refs_out, int32_t* moves,
                                                                    int32_t* n_moves) {
  __shared__ int sums[kWarps];
  after_stream();
  next_may_start();  // pages_rename_kernel
  const auto used = [&](int p) { return refs[p] > 0; };
  int mine = 0, n;
  for (int p = threadIdx.x; p < g.num_pages; p += kThreads) mine += used(p);
  block_scan(mine, sums, &n);
  // free pages before n, rising, into the moves; at most num_pages / 2 of them
  rank_pages(0, n, n, sums, [&](int p) { return !used(p); }, [&](int p, int k) { moves[3 * (int64_t)k + 1] = p; });
  __syncthreads();
  if (refs_out != refs)  // a page that stays keeps its count
    for (int p = threadIdx.x; p < n; p += kThreads) refs_out[p] = refs[p];
  __syncthreads();
  // pages in use at n or behind: as many as there are free ones before n
  const int count = rank_pages(n, g.num_pages, g.num_pages, sums, used, [&](int p, int k) {
    moves[3 * (int64_t)k] = p;
    moves[3 * (int64_t)k + 2] = g.page_rows;
    refs_out[moves[3 * (int64_t)k + 1]] = refs[p];
  });
  __syncthreads();  // counts behind n are read above
  for (int p = n + threadIdx.x; p < g.num_pages; p += kThreads) refs_out[p] = 0;
  const int64_t end = 3 * (int64_t)(g.num_pages / 2);
  for (int64_t i = 3 * (int64_t)count + threadIdx.x; i < end; i += kThreads) moves[i] = -1;
  if (threadIdx.x == 0) *n_moves = count;
}

// Table entries after a compaction: one block a sequence.  The moves are in
// rising order of their sources and of their destinations, and the sources lie
// behind all pages that stay.  An entry that names no page in use is damaged and
// becomes -1: also one that names a destination, which was free and is in use now.
__global__ void __launch_bounds__(128) pages_rename_kernel(const Pages g, const int32_t* table,
                                                           const int32_t* lengths, const int32_t* refs_out,
                                                           const int32_t* moves, const int32_t* n_moves,
                                                           int32_t* table_out) {
  const int64_t row = blockIdx.x * g.table_stride;
  const int n = lengths[blockIdx.x];
  bool bad = n < 0 || n > g.rows;
  const int held = g.pages(min(max(n, 0), g.rows));
  // the kernel in front writes no table: entries may be read ahead of it
  int ahead = threadIdx.x < held ? table[row + threadIdx.x] : -1;
  after_stream();
  const int count = *n_moves, source0 = count > 0 ? moves[0] : g.num_pages;
  for (int c = threadIdx.x; c < g.max_pages; c += blockDim.x) {
    int p = -1;
    if (c < held) {
      p = c == (int)threadIdx.x ? ahead : table[row + c];
      if (p < 0 || p >= g.num_pages) {
        p = -1;
      } else {
        // the first move whose source (or destination, of a page before all
        // sources) is at or behind p, eight ways at a time
        const int32_t* key = moves + (p < source0);
        int lo = 0, hi = count;
        while (lo < hi) {
          const int step = (hi - lo + 7) / 8;
          int below = 0;
#pragma unroll
          for (int k = 1; k < 8; ++k) {
            const int at = lo + k * step - 1;
            if (at < hi && key[3 * (int64_t)at] < p) below = k;
          }
          if (below < 7) hi = min(hi, lo + (below + 1) * step - 1);
          lo += below * step;
        }
        if (lo < count && key[3 * (int64_t)lo] == p)
          p = p < source0 ? -1 : moves[3 * (int64_t)lo + 1];
        else if (refs_out[p] <= 0)
          p = -1;
      }
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

fa_status fa_pages_extend(const fa_cache* c, int32_t* page_table, int32_t* lengths, int32_t* refs,
                          const int32_t* n_new, int32_t* start, void* stream) {
  fa::NvtxRange range("fa_pages_extend");
  const fa_status st = fa::check_pages(c);
  if (st != FA_OK) return st;
  if (!fa::aligned4(page_table) || !fa::aligned4(lengths) || !fa::aligned4(refs) || !fa::aligned4(n_new) ||
      !fa::aligned4(start) || start == lengths || start == n_new)
    return FA_ERR_INVALID_ARG;
  fa::Pages g;
  if (!fa::geometry(*c, &g)) return FA_ERR_CUDA;
  return fa::status_of(fa::launch_early(fa::pages_extend_kernel, dim3(1), fa::kThreads, 0, (cudaStream_t)stream, 1, g,
                                        page_table, lengths, refs, n_new, start));
}

fa_status fa_pages_fork(const fa_cache* c, int32_t pairs, const int32_t* src, const int32_t* dst, int32_t* page_table,
                        int32_t* lengths, int32_t* refs, int32_t* moves, void* stream) {
  fa::NvtxRange range("fa_pages_fork");
  const fa_status st = fa::check_pages(c);
  if (st != FA_OK) return st;
  if (c->S > 65536) return FA_ERR_UNSUPPORTED;  // its marks are kept in shared memory
  if (pairs < 1 || pairs > c->S || !fa::aligned4(src) || !fa::aligned4(dst) || !fa::aligned4(page_table) ||
      !fa::aligned4(lengths) || !fa::aligned4(refs) || !fa::aligned4(moves))
    return FA_ERR_INVALID_ARG;
  fa::Pages g;
  if (!fa::geometry(*c, &g)) return FA_ERR_CUDA;
  return fa::status_of(fa::launch_early(fa::pages_fork_kernel, dim3(fa::kForkBlocks), fa::kThreads,
                                        (c->S + 15) / 16 * 4, (cudaStream_t)stream, fa::kForkBlocks, g, pairs, src, dst,
                                        page_table, lengths, refs, moves));
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
  return fa::status_of(fa::launch_early(fa::pages_free_kernel, dim3((unsigned)count), 128, 0, (cudaStream_t)stream, 1, g,
                                        sequences, page_table, lengths, refs));
}

fa_status fa_pages_compact(const fa_cache* c, const int32_t* page_table, const int32_t* lengths, const int32_t* refs,
                           int32_t* table_out, int32_t* refs_out, int32_t* moves, int32_t* n_moves, void* stream) {
  fa::NvtxRange range("fa_pages_compact");
  const fa_status st = fa::check_pages(c);
  if (st != FA_OK) return st;
  if (!fa::aligned4(page_table) || !fa::aligned4(lengths) || !fa::aligned4(refs) || !fa::aligned4(table_out) ||
      !fa::aligned4(refs_out) || (c->num_pages > 1 && !fa::aligned4(moves)) || !fa::aligned4(n_moves))
    return FA_ERR_INVALID_ARG;
  fa::Pages g;
  if (!fa::geometry(*c, &g)) return FA_ERR_CUDA;
  const cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e =
      fa::launch_early(fa::pages_compact_kernel, dim3(1), fa::kThreads, 0, s, 1, g, refs, refs_out, moves, n_moves);
  if (e != cudaSuccess) return FA_ERR_CUDA;
  return fa::status_of(fa::launch_early(fa::pages_rename_kernel, dim3((unsigned)c->S), 128, 0, s, 1, g, page_table,
                                        lengths, refs_out, moves, n_moves, table_out));
}

}  // extern "C"
