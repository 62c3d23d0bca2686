// pages.cu -- page bookkeeping of a paged cache: mapping room for new rows, forking, releasing and
// compacting.  The state is the caller's: page_table [B, max_pages] (-1: unmapped), seq_lens [B],
// refs [num_pages] = how many table entries map a page (0: free), and the pool.
//
// Free pages are taken lowest first, by list entry and then by position, so the outcome does not
// depend on the order in which blocks run: a first kernel takes a snapshot (one bit per page for
// free and for shared, free counts of 4,096-page chunks and of the words inside them, and each
// list entry's demand), and the second works from the snapshot alone -- the r-th free page is
// two binary searches -- while it changes table, lengths and refs.  Counts change by integer
// atomics, whose order does not matter.
//
// What bounds it: two launches, and the bytes of the pages that are copied (a page is in flight
// at once per CTA: 512 threads, 16 bytes each, eight deep).  Measured: compaction of a 1.1 GB pool,
// half free, 7 us of snapshot and 74 of moves (86 together with the tables' reset); 256 sequences:
// release 4 us, fork of 96 7 + 9, reserve 7 + 7.
#include <algorithm>

#include "internal.h"
#include "mla.h"
#include "sm100.cuh"

namespace mla {
namespace pages {

constexpr int kThreads = 512;
constexpr int kChunk = 4096;            // pages per snapshot chunk
constexpr int kChunkWords = kChunk / 32;
constexpr int kStatusPages = 7;         // MLA_ERR_PAGES
constexpr int kBad = -1;                // demand of an entry that is refused

struct Book {
  int32_t *table, *lens, *refs;
  uint8_t *pool;
  int page_bytes, B, max_pages, num_pages, nchunks;
  int32_t *status;
  // snapshot
  uint32_t *free_bits, *shared_bits;
  uint16_t *word_rank;   // free pages of the chunk before the word
  int32_t *chunk_free;   // free pages of the chunk
  int32_t *demand;       // pages that list entry k takes, or kBad
};

__device__ __forceinline__ bool mapped(const Book &bk, int page) { return page >= 0 && page < bk.num_pages; }

// ------------------------------------------------------------------ snapshot
__device__ void scan_chunk(const Book &bk, int chunk) {
  __shared__ int words[kChunkWords];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int w = warp; w < kChunkWords; w += kThreads / 32) {
    const long long p = (long long)chunk * kChunk + w * 32 + lane;
    const int r = p < bk.num_pages ? bk.refs[p] : 1;
    const uint32_t fr = __ballot_sync(0xffffffffu, r == 0), sh = __ballot_sync(0xffffffffu, r > 1);
    if (lane == 0) {
      words[w] = __popc(fr);
      if ((long long)chunk * kChunk + w * 32 < bk.num_pages) {
        bk.free_bits[chunk * kChunkWords + w] = fr;
        bk.shared_bits[chunk * kChunkWords + w] = sh;
      }
    }
  }
  __syncthreads();
  if (warp == 0) {
    int base = 0;
    for (int w0 = 0; w0 < kChunkWords; w0 += 32) {
      const int n = words[w0 + lane];
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if ((long long)chunk * kChunk + (w0 + lane) * 32 < bk.num_pages)
        bk.word_rank[chunk * kChunkWords + w0 + lane] = (uint16_t)(base + x - n);
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) bk.chunk_free[chunk] = base;
  }
}

// Table entries [first, end) that the rows [L, L + Q) of sequence b fall on; false if they have none.
__device__ __forceinline__ bool reserve_range(const Book &bk, int b, int Q, int &first, int &end) {
  const long long L = bk.lens[b];
  first = (int)(L / kPageTokens);
  end = (int)((L + Q - 1) / kPageTokens) + 1;
  return L >= 0 && L + Q <= (long long)bk.max_pages * kPageTokens;
}

// Pages that sequence b needs to take Q more rows: its unmapped entries, and the shared pages that
// it is about to write.
__device__ int reserve_demand(const Book &bk, int b, int Q) {
  int first, end, n = 0;
  bool ok = reserve_range(bk, b, Q, first, end);
  if (ok)
    for (int k = first + (int)threadIdx.x; k < end; k += kThreads) {
      const int page = bk.table[(long long)b * bk.max_pages + k];
      if (page < -1 || page >= bk.num_pages) ok = false;
      else n += page < 0 || bk.refs[page] > 1;
    }
  ok = __syncthreads_and(ok);
  __shared__ int total;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  n = __reduce_add_sync(0xffffffffu, n);
  if (threadIdx.x % 32 == 0 && n) atomicAdd(&total, n);
  __syncthreads();
  return ok ? total : kBad;
}

// Fork k is sound: both sequences exist, the child is empty and stands nowhere else in the list,
// the parent's full pages are mapped or unmapped (given back behind a window), its partial last page is
// mapped.  Its demand: the copy of that one.
__device__ int fork_demand(const Book &bk, const int32_t *parents, const int32_t *children, int n, int k) {
  const int par = parents[k], child = children[k];
  bool ok = par >= 0 && par < bk.B && child >= 0 && child < bk.B && par != child;
  int partial = 0;
  if (ok) {
    for (int i = threadIdx.x; i < n; i += kThreads) ok = ok && (i == k || children[i] != child) && parents[i] != child;
    const long long L = bk.lens[par];
    ok = ok && L >= 0 && L <= (long long)bk.max_pages * kPageTokens;
    partial = L % kPageTokens != 0;
    for (int e = threadIdx.x; e < bk.max_pages; e += kThreads) {
      ok = ok && bk.table[(long long)child * bk.max_pages + e] == -1;
      if ((long long)e * kPageTokens >= L) continue;
      const int page = bk.table[(long long)par * bk.max_pages + e];
      const bool full = (e + 1LL) * kPageTokens <= L;
      ok = ok && (mapped(bk, page) || (full && page == -1));
    }
  }
  return __syncthreads_and(ok) ? partial : kBad;
}

enum Op : int { kReserve = 0, kFork = 1, kCompact = 2 };

// Blocks [0, nchunks): the pages; the others: the list entries' demands.
template <int kOp>
__global__ void __launch_bounds__(kThreads) snapshot_kernel(const Book bk, const int32_t *parents,
                                                            const int32_t *children, int n, int Q) {
  grid_dep_launch();
  grid_dep_wait();
  if ((int)blockIdx.x < bk.nchunks) {
    scan_chunk(bk, blockIdx.x);
    return;
  }
  if constexpr (kOp != kCompact) {
    const int k = blockIdx.x - bk.nchunks;
    const int d = kOp == kReserve ? reserve_demand(bk, k, Q) : fork_demand(bk, parents, children, n, k);
    if (threadIdx.x == 0) bk.demand[k] = d;
  }
}

// ------------------------------------------------------------------ working from the snapshot
// Free pages before each chunk, in shared memory (nchunks + 1 entries), by the whole block.
__device__ void load_ranks(const Book &bk, int32_t *rank) {
  __shared__ int warp_sum[kThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int base = 0;
  for (int c0 = 0; c0 < bk.nchunks; c0 += kThreads) {
    const int c = c0 + (int)threadIdx.x;
    const int n = c < bk.nchunks ? bk.chunk_free[c] : 0;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = base, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      before += w < warp ? warp_sum[w] : 0;
      total += warp_sum[w];
    }
    if (c < bk.nchunks) rank[c] = before + x - n;
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) rank[bk.nchunks] = base;
  __syncthreads();
}

// Free pages below page p (p <= num_pages).
__device__ __forceinline__ int free_below(const Book &bk, const int32_t *rank, int p) {
  if (p >= bk.num_pages) return rank[bk.nchunks];
  const int w = p / 32;
  return rank[w / kChunkWords] + bk.word_rank[w] + __popc(bk.free_bits[w] & ((1u << (p % 32)) - 1u));
}

// The page with `r` pages of its kind below it: the r-th free page, or (kUsed) the r-th used one.
template <bool kUsed>
__device__ int nth_page(const Book &bk, const int32_t *rank, int r) {
  int lo = 0, hi = bk.nchunks - 1;  // the last chunk with at most r pages of the kind before it
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    const int before = kUsed ? mid * kChunk - rank[mid] : rank[mid];
    if (before <= r) lo = mid; else hi = mid - 1;
  }
  const int chunk = lo;
  r -= kUsed ? chunk * kChunk - rank[chunk] : rank[chunk];
  const int words = min(kChunkWords, (bk.num_pages - chunk * kChunk + 31) / 32);
  lo = 0, hi = words - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    const int fr = bk.word_rank[chunk * kChunkWords + mid];
    if ((kUsed ? mid * 32 - fr : fr) <= r) lo = mid; else hi = mid - 1;
  }
  const int w = chunk * kChunkWords + lo, fr = bk.word_rank[w];
  r -= kUsed ? lo * 32 - fr : fr;
  uint32_t bits = kUsed ? ~bk.free_bits[w] : bk.free_bits[w];
  for (; r > 0; --r) bits &= bits - 1;
  return w * 32 + __ffs(bits) - 1;
}

// pool[dst] = pool[src], by the whole block, eight 16-byte loads a thread in flight.
__device__ void copy_page(const Book &bk, int dst, int src) {
  const uint4 *from = reinterpret_cast<const uint4 *>(bk.pool + (long long)src * bk.page_bytes);
  uint4 *to = reinterpret_cast<uint4 *>(bk.pool + (long long)dst * bk.page_bytes);
  const int units = bk.page_bytes / 16;
  constexpr int kDeep = 8;
  for (int u0 = threadIdx.x; u0 < units; u0 += kDeep * kThreads) {
    uint4 v[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      if (u0 + i * kThreads < units) v[i] = from[u0 + i * kThreads];
#pragma unroll
    for (int i = 0; i < kDeep; ++i)
      if (u0 + i * kThreads < units) to[u0 + i * kThreads] = v[i];
  }
}

// Pages taken by list entries before k (refused ones take none), by the whole block.  In 64 bits:
// a list of 66 sequences can ask for 2^31 pages.
__device__ long long demand_before(const Book &bk, int k) {
  __shared__ unsigned long long total;
  if (threadIdx.x == 0) total = 0;
  __syncthreads();
  unsigned long long n = 0;
  for (int i = threadIdx.x; i < k; i += kThreads) n += max(bk.demand[i], 0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (threadIdx.x % 32 == 0 && n) atomicAdd(&total, n);
  __syncthreads();
  return (long long)total;
}

// True if entry k goes ahead; reports why it does not.
__device__ bool granted(const Book &bk, const int32_t *rank, int k, long long before) {
  const int d = bk.demand[k];
  const bool room = d <= 0 || before + d <= rank[bk.nchunks];
  if (threadIdx.x == 0) {
    if (d == kBad) report_status(bk.status, kStatusIndex);
    else if (!room) report_status(bk.status, kStatusPages);
  }
  return d != kBad && room;
}

// Block b: the pages of sequence b's next Q rows.
__global__ void __launch_bounds__(kThreads) reserve_kernel(const Book bk, int Q) {
  extern __shared__ int32_t rank[];
  grid_dep_launch();
  grid_dep_wait();
  const int b = blockIdx.x;
  if (bk.demand[b] == 0) return;
  load_ranks(bk, rank);
  const long long taken = demand_before(bk, b);
  if (!granted(bk, rank, b, taken)) return;
  int next = (int)taken;  // below the number of free pages
  int first, end;
  reserve_range(bk, b, Q, first, end);
  int32_t *row = bk.table + (long long)b * bk.max_pages;
  __shared__ int warp_takes[kThreads / 32];
  __shared__ int copies, copy_src[kThreads], copy_dst[kThreads];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int k0 = first; k0 < end; k0 += kThreads) {
    const int k = k0 + (int)threadIdx.x;
    const int old = k < end ? row[k] : 0;
    const bool shared = k < end && old >= 0 && (bk.shared_bits[old / 32] >> (old % 32) & 1);
    const bool take = k < end && (old < 0 || shared);
    const uint32_t m = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_takes[warp] = __popc(m);
    if (threadIdx.x == 0) copies = 0;
    __syncthreads();
    int before = next, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      before += w < warp ? warp_takes[w] : 0;
      total += warp_takes[w];
    }
    if (take) {
      const int page = nth_page<false>(bk, rank, before + __popc(m & ((1u << lane) - 1u)));
      row[k] = page;
      bk.refs[page] = 1;
      if (shared) {
        atomicSub(&bk.refs[old], 1);
        const int c = atomicAdd(&copies, 1);  // which copy is made first does not matter
        copy_src[c] = old;
        copy_dst[c] = page;
      }
    }
    __syncthreads();
    for (int c = 0; c < copies; ++c) copy_page(bk, copy_dst[c], copy_src[c]);
    next += total;
    __syncthreads();
  }
}

// Block k: fork k.
__global__ void __launch_bounds__(kThreads) fork_kernel(const Book bk, const int32_t *parents,
                                                        const int32_t *children) {
  extern __shared__ int32_t rank[];
  grid_dep_launch();
  grid_dep_wait();
  const int k = blockIdx.x;
  load_ranks(bk, rank);
  const long long before = demand_before(bk, k);
  if (!granted(bk, rank, k, before)) return;
  const int par = parents[k], child = children[k];
  const int L = bk.lens[par];
  const int full = L / kPageTokens;
  const int32_t *from = bk.table + (long long)par * bk.max_pages;
  int32_t *to = bk.table + (long long)child * bk.max_pages;
  __shared__ int fresh;
  for (int e = threadIdx.x; e < full; e += kThreads) {
    const int page = from[e];
    if (page == -1) continue;  // as the child's entry
    to[e] = page;
    atomicAdd(&bk.refs[page], 1);
  }
  if (threadIdx.x == 0) {
    bk.lens[child] = L;
    if (L % kPageTokens) {
      fresh = nth_page<false>(bk, rank, (int)before);
      to[full] = fresh;
      bk.refs[fresh] = 1;
    }
  }
  __syncthreads();
  if (L % kPageTokens) copy_page(bk, fresh, from[full]);
}

// Every mapped entry at or behind ceil(L / 64) is unmapped.
__global__ void __launch_bounds__(kThreads) release_kernel(const Book bk) {
  grid_dep_launch();
  grid_dep_wait();
  const int b = blockIdx.x;
  const long long L = bk.lens[b];
  if (L < 0 || L > (long long)bk.max_pages * kPageTokens) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report_status(bk.status, kStatusIndex);
    return;
  }
  const int first = (int)((L + kPageTokens - 1) / kPageTokens);
  for (int k = first + blockIdx.y * kThreads + (int)threadIdx.x; k < bk.max_pages; k += gridDim.y * kThreads) {
    int32_t *entry = bk.table + (long long)b * bk.max_pages + k;
    const int page = *entry;
    if (page == -1) continue;
    if (!mapped(bk, page)) {
      report_status(bk.status, kStatusIndex);
      continue;
    }
    if (atomicSub(&bk.refs[page], 1) <= 0) {  // more entries than refs: the state was not sound
      atomicAdd(&bk.refs[page], 1);
      report_status(bk.status, kStatusIndex);
    }
    *entry = -1;
  }
}

// The used pages at or above n_used move, in order, to the free pages below it; entries follow.
__global__ void __launch_bounds__(kThreads) compact_kernel(const Book bk, int32_t *n_used_out) {
  extern __shared__ int32_t rank[];
  grid_dep_launch();
  grid_dep_wait();
  load_ranks(bk, rank);
  const int n_used = bk.num_pages - rank[bk.nchunks];
  const int moves = free_below(bk, rank, n_used);
  const int kept = n_used - moves;  // used pages below n_used
  if (blockIdx.x == 0 && threadIdx.x == 0) *n_used_out = n_used;
  const long long entries = (long long)bk.B * bk.max_pages;
  const long long step = (long long)gridDim.x * kThreads;
  for (long long e = (long long)blockIdx.x * kThreads + threadIdx.x; e < entries; e += step) {
    const int page = bk.table[e];
    if (page == -1) continue;
    // outside the pool, or mapped but free: the entry stays, whatever moves to that page
    if (!mapped(bk, page) || (bk.free_bits[page / 32] >> (page % 32) & 1)) report_status(bk.status, kStatusIndex);
    else if (page >= n_used) bk.table[e] = nth_page<false>(bk, rank, page - free_below(bk, rank, page) - kept);
  }
  for (int m = blockIdx.x; m < moves; m += gridDim.x) {
    const int src = nth_page<true>(bk, rank, kept + m), dst = nth_page<false>(bk, rank, m);
    copy_page(bk, dst, src);
    if (threadIdx.x == 0) {
      bk.refs[dst] = bk.refs[src];
      bk.refs[src] = 0;
    }
  }
}

// ------------------------------------------------------------------ host
size_t align16(size_t n) { return (n + 15) & ~size_t(15); }

size_t workspace_bytes(int n, int num_pages) {
  const size_t words = ((size_t)num_pages + 31) / 32, chunks = ((size_t)num_pages + kChunk - 1) / kChunk;
  return 2 * align16(words * 4) + align16(words * 2) + align16(chunks * 4) + align16((size_t)n * 4);
}

mla_status make_book(Book &bk, void *pool, int page_bytes, int32_t *table, int32_t *lens, int32_t *refs, int B,
                     int max_pages, int num_pages, int n, void *workspace, size_t ws_bytes, int32_t *status) {
  if (table == nullptr || refs == nullptr || B < 1 || max_pages < 1 || num_pages < 1 || n < 1) return MLA_ERR_ARG;
  if ((long long)max_pages * kPageTokens >= (1LL << 31) || (long long)num_pages * kPageTokens >= (1LL << 31))
    return MLA_ERR_ARG;
  const uintptr_t at = reinterpret_cast<uintptr_t>(pool), ws = reinterpret_cast<uintptr_t>(workspace);
  bk = {table, lens, refs, reinterpret_cast<uint8_t *>(pool), page_bytes, B, max_pages, num_pages,
        (num_pages + kChunk - 1) / kChunk, status, nullptr, nullptr, nullptr, nullptr, nullptr};
  if (pool == nullptr) return MLA_OK;  // release: no pages are touched
  if (page_bytes < 16 || page_bytes % 16 != 0 || (at & 15u) != 0) return MLA_ERR_UNSUPPORTED;
  if (workspace == nullptr || ws_bytes < workspace_bytes(n, num_pages) || (ws & 15u) != 0) return MLA_ERR_WORKSPACE;
  const size_t words = ((size_t)num_pages + 31) / 32;
  uint8_t *w = reinterpret_cast<uint8_t *>(workspace);
  bk.free_bits = reinterpret_cast<uint32_t *>(w);
  w += align16(words * 4);
  bk.shared_bits = reinterpret_cast<uint32_t *>(w);
  w += align16(words * 4);
  bk.word_rank = reinterpret_cast<uint16_t *>(w);
  w += align16(words * 2);
  bk.chunk_free = reinterpret_cast<int32_t *>(w);
  w += align16((size_t)bk.nchunks * 4);
  bk.demand = reinterpret_cast<int32_t *>(w);
  return MLA_OK;
}

size_t rank_bytes(const Book &bk) { return ((size_t)bk.nchunks + 1) * sizeof(int32_t); }  // at most 32 KB

}  // namespace pages
}  // namespace mla

extern "C" {

size_t mla_pages_workspace_bytes(int n, int num_pages) {
  if (n < 1 || num_pages < 1 || (long long)num_pages * mla::kPageTokens >= (1LL << 31)) return 0;
  return mla::pages::workspace_bytes(n, num_pages);
}

mla_status mla_pages_reserve(void *pool, int page_bytes, int32_t *page_table, const int32_t *seq_lens, int32_t *refs,
                             int B, int Q, int max_pages, int num_pages, void *workspace, size_t ws_bytes,
                             int32_t *status, void *stream) {
  using namespace mla;
  using namespace mla::pages;
  if (pool == nullptr || seq_lens == nullptr || Q < 1) return MLA_ERR_ARG;
  Book bk;
  if (mla_status s = make_book(bk, pool, page_bytes, page_table, const_cast<int32_t *>(seq_lens), refs, B, max_pages,
                               num_pages, B, workspace, ws_bytes, status);
      s != MLA_OK)
    return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_chained(snapshot_kernel<kReserve>, dim3(bk.nchunks + B), dim3(kThreads), 0, st, bk,
                                 (const int32_t *)nullptr, (const int32_t *)nullptr, B, Q);
  if (e == cudaSuccess) e = launch_chained(reserve_kernel, dim3(B), dim3(kThreads), rank_bytes(bk), st, bk, Q);
  return record_cuda_error(e);
}

mla_status mla_pages_fork(void *pool, int page_bytes, int32_t *page_table, int32_t *seq_lens, int32_t *refs,
                          const int32_t *parents, const int32_t *children, int n, int B, int max_pages, int num_pages,
                          void *workspace, size_t ws_bytes, int32_t *status, void *stream) {
  using namespace mla;
  using namespace mla::pages;
  if (pool == nullptr || seq_lens == nullptr || parents == nullptr || children == nullptr) return MLA_ERR_ARG;
  Book bk;
  if (mla_status s = make_book(bk, pool, page_bytes, page_table, seq_lens, refs, B, max_pages, num_pages, n, workspace,
                               ws_bytes, status);
      s != MLA_OK)
    return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_chained(snapshot_kernel<kFork>, dim3(bk.nchunks + n), dim3(kThreads), 0, st, bk, parents,
                                 children, n, 0);
  if (e == cudaSuccess)
    e = launch_chained(fork_kernel, dim3(n), dim3(kThreads), rank_bytes(bk), st, bk, parents, children);
  return record_cuda_error(e);
}

mla_status mla_pages_release(int32_t *page_table, const int32_t *seq_lens, int32_t *refs, int B, int max_pages,
                             int num_pages, int32_t *status, void *stream) {
  using namespace mla;
  using namespace mla::pages;
  if (seq_lens == nullptr) return MLA_ERR_ARG;
  Book bk;
  if (mla_status s = make_book(bk, nullptr, 0, page_table, const_cast<int32_t *>(seq_lens), refs, B, max_pages,
                               num_pages, B, nullptr, 0, status);
      s != MLA_OK)
    return s;
  const int splits = std::min(64, (max_pages + kThreads - 1) / kThreads);
  return record_cuda_error(launch_chained(release_kernel, dim3(B, splits), dim3(kThreads), 0,
                                          reinterpret_cast<cudaStream_t>(stream), bk));
}

mla_status mla_pages_compact(void *pool, int page_bytes, int32_t *page_table, int32_t *refs, int B, int max_pages,
                             int num_pages, int32_t *n_used, void *workspace, size_t ws_bytes, int32_t *status,
                             void *stream) {
  using namespace mla;
  using namespace mla::pages;
  if (pool == nullptr || n_used == nullptr) return MLA_ERR_ARG;
  Book bk;
  if (mla_status s = make_book(bk, pool, page_bytes, page_table, nullptr, refs, B, max_pages, num_pages, 1, workspace,
                               ws_bytes, status);
      s != MLA_OK)
    return s;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_chained(snapshot_kernel<kCompact>, dim3(bk.nchunks), dim3(kThreads), 0, st, bk,
                                 (const int32_t *)nullptr, (const int32_t *)nullptr, 0, 0);
  const int grid = std::min(num_pages, 4 * device_sm_count());
  if (e == cudaSuccess) e = launch_chained(compact_kernel, dim3(grid), dim3(kThreads), rank_bytes(bk), st, bk, n_used);
  return record_cuda_error(e);
}

}  // extern "C"
