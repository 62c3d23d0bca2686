// window_attend.cu -- split-L latent attention with a sliding window and sinks (window.cuh) over a
// contiguous or paged bf16 cache: scores q~.c_j, softmax over the rows that a query sees, value
// sum in latent space.
//
// The pipeline is attend.cu's (64-row tiles, a ring of 2.25 tiles in shared memory filled by TMA,
// scores and value products on tcgen05 from two issuing warps, eight softmax warps, lazy rescale
// of O in tensor memory).  It is a kernel of its own because the window's bookkeeping, as a
// template parameter of that kernel, changed the code generated for the other modes and cost a
// verify step 1.5%.  What differs:
//  - a sequence's tile list holds only the tiles of its sinks and of its queries' windows, so the
//    work is split evenly over what has to be read; a query walks those of them that it sees;
//  - rows that a query does not see are masked in the softmax, and zeroed in the landed slot,
//    whatever they hold;
//  - the list's ranges allow for what beginning a sequence costs, and the merge has a form for few
//    sequences with many partials (lists.cuh);
//  - l sums the unrounded weights, so lse is exact to fp32.  The value product takes them rounded to
//    bf16: against 64 bits o is off by 0.0018 to 0.0022 of its norm (windows of two rows or more),
//    where rounding the result alone costs 0.0017.
//
// What bounds it: as attend.cu, the recycling of ring slots, 3,000 cycles a tile (0.87 of the
// measured copy peak for distinct rows); around that, for windows of some thousand rows, 20 us of
// start-up, partial stores and combine.  Six queries of 16 sequences keep the tensor pipe 45% busy, the
// issue slots 21% and DRAM 10%, at about 3,200 cycles a tile.  Measured with the merge: 32 x (4,096 +
// 64) of 8,192 rows 41.7 us; 16 x 6 queries, window 4,095 + 5, 89-91 us.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "lists.cuh"
#include "window_attend.h"
#include "sm100.cuh"
#include "split.cuh"
#include "window.cuh"

namespace mla {
namespace windowed {

constexpr int kTile = 64;                       // cache rows per tile (MMA M of the score GEMM)
constexpr int kRows = 64;                       // query rows per CTA = heads (MMA N)
constexpr int kSlotQuarters = kLatent / 128;    // a tile is 4 ring slots of 128 latent values
constexpr int kSlots = 9;                       // ring slots (2.25 tiles)
constexpr int kAtomBytes = kTile * 128;         // 8 KB: 64 rows x 64 latent, 128-byte swizzle
constexpr int kSlotBytes = 2 * kAtomBytes;      // 16 KB: 64 rows x 128 latent
constexpr int kQtChunks = kLatent / 64;
constexpr int kQtChunkBytes = kRows * 64 * 2;   // 8 KB: 64 heads x 64 latent
constexpr int kPBytes = kTile * kRows * 2;      // 8 KB: P^T, 64 rows x 64 heads (bf16)
constexpr int kThreads = 352;  // producer, score MMA, 8 softmax warps, value MMA
constexpr int kSoftmaxWarps = 8;
constexpr float kTau = 8.0f;  // lazy rescale: the running max is raised only when a score
                              // exceeds it by more than 2^8 (probabilities stay <= 256)
// The running max before any score.  Finite, since -inf marks an empty partial: one that has seen
// only NaN scores, which the max passes over, or -Inf is not empty.
constexpr float kLowest = -FLT_MAX;

constexpr int kOffC = 0;
constexpr int kOffQt = kOffC + kSlots * kSlotBytes;
constexpr int kOffP = kOffQt + kQtChunks * kQtChunkBytes;
constexpr int kOffRed = kOffP + 2 * kPBytes;     // [4][64] floats
constexpr int kOffMUsed = kOffRed + 4 * 64 * 4;  // [64] floats
constexpr int kOffAlpha = kOffMUsed + 64 * 4;    // [64] floats
constexpr int kOffBar = kOffAlpha + 64 * 4;
// barriers
constexpr int kBarCFull = 0, kBarCEmpty = kSlots, kBarQFull = 2 * kSlots, kBarQEmpty = kBarQFull + 1,
              kBarSFull = kBarQEmpty + 1, kBarSEmpty = kBarSFull + 2, kBarPFull = kBarSEmpty + 2,
              kBarPEmpty = kBarPFull + 2, kBarOFull = kBarPEmpty + 2, kBarOEmpty = kBarOFull + 1,
              kBarDrain = kBarOEmpty + 1, kNumBars = kBarDrain + 1;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kOffRange = kOffMisc + 16;
constexpr int kSmemUsed = kOffRange + (int)sizeof(lists::Range);
constexpr int kSmemBytes = kSmemUsed + 1024;  // slack for 1024-byte alignment of the base
static_assert(kSmemBytes <= 232448, "shared memory budget");
static_assert(kPageTokens == kTile, "a paged tile is exactly one page");

// TMEM columns: two score buffers (M = 64 accumulators: lanes 0-15 of each 32-lane
// quadrant hold tile rows 16q..16q+15), then O^T as four 128-lane blocks of 64 columns.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0;
constexpr uint32_t kTmemO = 256;

// ------------------------------------------------------------------ sequences and tiles

using SeqTiles = window::SeqTiles<kTile>;
using QueryTiles = window::QueryTiles<kTile>;
template <bool kPaged>
struct Seqs {  // for lists.cuh
  static constexpr int kStart = 3;
  static __device__ __forceinline__ int cap(const WindowParams &p) {
    return kPaged ? p.max_pages * kPageTokens : p.Lmax;
  }
  static __device__ __forceinline__ int length(const WindowParams &p, int b) {
    return min(max(p.seq_lens ? p.seq_lens[b] : p.Lmax, 0), cap(p));
  }
  static __device__ __forceinline__ int tiles(const WindowParams &p, int L) {
    return SeqTiles(L, p.Q, p.window, p.sinks).count;
  }
  static __device__ __forceinline__ bool bad_length(const WindowParams &p, int b) {
    return p.seq_lens && (p.seq_lens[b] < 0 || p.seq_lens[b] > cap(p));
  }
};
using lists::Range;

// A segment: the piece of sequence s in a CTA's range.  lo, hi and the loops' t count list tiles, of
// which next() skips those that the query does not see; tile(t) is the tile of the sequence.
struct Seg {
  int s;
  int lo, hi;
  bool empty;  // the query sees no tile of it; its partial is written as empty
  QueryTiles q;
  __device__ __forceinline__ int next(int t) const { return q.seek(t + 1); }
  __device__ __forceinline__ int tile(int t) const { return q.seq.tile(t); }
};

// Walks the segments of a contiguous range [t, t_end) of the tile list for query iq.
template <bool kPaged>
struct SegIter {
  long long t, t_end, base;
  int s, L, start, iq;
  __device__ SegIter(const Range &r, int iq_)
      : t(r.t0), t_end(r.t1), base(r.base), s(r.s), L(r.L), start(r.start), iq(iq_) {}
  __device__ bool next(const WindowParams &p, Seg &sg) {
    if (t >= t_end) return false;
    int n = lists::places<Seqs<kPaged>>(p, L, start);
    while (base + n <= t) {
      base += n;
      L = Seqs<kPaged>::length(p, ++s);
      n = lists::places<Seqs<kPaged>>(p, L, start);
    }
    const int end = (int)min(t_end - base, (long long)n);
    sg.s = s;
    sg.q = QueryTiles(L, p.Q, iq, p.window, p.sinks);
    sg.lo = sg.q.seek(max((int)(t - base) - start, 0));
    sg.hi = min(max(end - start, 0), sg.q.e);
    sg.empty = sg.hi <= sg.lo;
    t = base + end;
    return true;
  }
};

struct PartialOrder {  // partials are stored latent by latent
  static __device__ __forceinline__ int latent(int idx) { return idx; }
  // The first of four values of thread t (of 32) in quarter `part` of the latents.
  static __device__ __forceinline__ int unit(int part, int t) { return 128 * part + 4 * t; }
};

// ------------------------------------------------------------------ shared state
struct Shared {
  uint8_t *base;
  uint64_t *bar;
  float *red, *m_used, *alpha;
  uint32_t *tmem_slot;
  volatile int *abort_flag;
  __device__ uint8_t *slot(int r) const { return base + kOffC + r * kSlotBytes; }
  __device__ uint8_t *qt(int c) const { return base + kOffQt + c * kQtChunkBytes; }
  __device__ uint8_t *pbuf(int i) const { return base + kOffP + i * kPBytes; }
};

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, const Shared &sh, int32_t *status) {
  const bool ok = mbar_wait(bar, parity, sh.abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}

// Ring slot k (k = 4 * tile + quarter, counted over the CTA's tiles): position and use.
__device__ __forceinline__ uint32_t ring_pos(uint32_t k) { return k % kSlots; }
__device__ __forceinline__ uint32_t ring_use(uint32_t k) { return k / kSlots; }

// ------------------------------------------------------------------ producer (warp 0, one lane)
// Issues the loads; counts the q~ loads and the ring-slot loads it issued (for the drain).
template <bool kPaged>
__device__ void producer_loads(const WindowParams &p, const Shared &sh, const CUtensorMap *tm_cache,
                               const CUtensorMap *tm_qt, int iq, const Range &range,
                               uint32_t &q_use, uint32_t &slots_issued) {
  uint64_t *bar = sh.bar;
  uint32_t tile_k = 0;
  SegIter<kPaged> it(range, iq);
  Seg sg;
  while (it.next(p, sg)) {
    if (sg.empty) continue;
    if (!mbar_wait(&bar[kBarQEmpty], (q_use & 1) ^ 1, sh.abort_flag, p.status)) return;
    mbar_arrive_expect_tx(&bar[kBarQFull], kQtChunks * kQtChunkBytes);
    tma_load_3d(sh.qt(0), tm_qt, &bar[kBarQFull], 0, (sg.s * p.Q + iq) * kRows, 0);  // all 8 chunks in one copy
    ++q_use;
    for (int t = sg.lo; t < sg.hi; t = sg.next(t), ++tile_k) {
      const int tile = sg.tile(t);
      long long row;
      if constexpr (kPaged) {
        int page = p.page_table[(long long)sg.s * p.max_pages + tile];
        if (page < 0 || page >= p.num_pages) {
          report_status(p.status, kStatusIndex);
          page = 0;
        }
        row = (long long)page * kPageTokens;
      } else {
        row = (long long)sg.s * p.Lmax + tile * kTile;
      }
      for (int qq = 0; qq < kSlotQuarters; ++qq) {
        const uint32_t k = tile_k * kSlotQuarters + qq;
        const uint32_t rp = ring_pos(k);
        if (!mbar_wait(&bar[kBarCEmpty + rp], (ring_use(k) & 1) ^ 1, sh.abort_flag, p.status)) return;
        mbar_arrive_expect_tx(&bar[kBarCFull + rp], kSlotBytes);
        // one copy per slot: a 3-D box {64 latent, 64 rows, 2 chunks} lands as the slot's two atoms
        tma_load_3d(sh.slot(rp), tm_cache, &bar[kBarCFull + rp], 0, (int)row, 2 * qq);
        slots_issued = k + 1;
      }
    }
  }
}
// The producer role: the loads, then (also after an abort) a wait until every copy it
// issued has landed.
template <bool kPaged>
__device__ void producer_role(const WindowParams &p, const Shared &sh, const CUtensorMap *tm_cache,
                              const CUtensorMap *tm_qt, int iq, const Range &range) {
  uint32_t q_use = 0, slots_issued = 0;
  producer_loads<kPaged>(p, sh, tm_cache, tm_qt, iq, range, q_use, slots_issued);
  bool ok = drain_ring(&sh.bar[kBarQFull], 1, q_use);
  ok = drain_ring(&sh.bar[kBarCFull], kSlots, slots_issued) && ok;
  if (!ok) report_status(p.status, kStatusTimeout);
}

// ------------------------------------------------------------------ MMA issuer (warp 1)
// Rows that the query does not see (past the end, before its window) may hold any bits: zero them
// in the landed slot so that a masked (zero) probability never meets a NaN or Inf in the value
// product.
__device__ __forceinline__ void prepare_slot(const Seg &sg, int tile, uint32_t sbase, int lane) {
  if (!sg.q.every_row(tile * kTile, kTile)) {
    for (int idx = lane; idx < 2 * kTile * 8; idx += 32) {
      const int at = idx / (kTile * 8), r = idx / 8 % kTile;
      if (!sg.q.row(tile * kTile + r)) st_shared_v4(sbase + at * kAtomBytes + r * 128 + (idx % 8) * 16, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  __syncwarp();
}

// Two warps feed the tensor pipe with independent streams, each with plain blocking waits:
// warp 1 issues the score GEMM of every tile, ring slot by ring slot as slots land, and
// warp 10 issues the value GEMM of every tile as soon as its probabilities are ready (which
// releases its ring slots).  MMAs of different threads are unordered, and the two streams
// touch disjoint TMEM columns, so the pipe simply interleaves them.  Loop state and MMA
// operands are warp-uniform; one elected lane issues.
template <bool kPaged>
__device__ void score_mma_role(const WindowParams &p, const Shared &sh, uint32_t tmem, int iq, const Range &range,
                               int lane) {
  uint64_t *bar = sh.bar;
  constexpr uint32_t idesc_s = idesc_bf16_f32(kTile, kRows, false, false);
  const uint32_t c_base = smem_u32(sh.slot(0));
  const uint32_t qt_base = smem_u32(sh.qt(0));
  uint32_t ns = 0, q_use = 0;
  SegIter<kPaged> it(range, iq);
  Seg sg;
  while (it.next(p, sg)) {
    if (sg.empty) continue;
    if (!wait_warp(&bar[kBarQFull], q_use & 1, sh, p.status)) return;
    ++q_use;
    for (int t = sg.lo; t < sg.hi; t = sg.next(t), ++ns) {
      if (!wait_warp(&bar[kBarSEmpty + (ns & 1)], ((ns >> 1) & 1) ^ 1, sh, p.status)) return;
      const uint32_t d = tmem + kTmemS + (ns & 1) * kRows;
#pragma unroll
      for (uint32_t sq = 0; sq < kSlotQuarters; ++sq) {
        // S^T[tile rows, heads] = C_tile * Q~^T; this slot holds K = 128 latent (8 steps)
        const uint32_t k = ns * kSlotQuarters + sq;
        if (!wait_warp(&bar[kBarCFull + ring_pos(k)], ring_use(k) & 1, sh, p.status)) return;
        const uint32_t sbase = c_base + ring_pos(k) * kSlotBytes;
        prepare_slot(sg, sg.tile(t), sbase, lane);
        tc_fence_after();
        const uint64_t a0 = sw128_desc(sbase, 16, 1024);
        const uint64_t b0 = sw128_desc(qt_base + 2 * sq * kQtChunkBytes, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // K step of 16 latent: 32 bytes inside a 128-byte swizzle row; the second four
            // steps are in the slot's second atom (A) and the next q~ chunk (B)
            const uint32_t ao = ((kk >> 2) * kAtomBytes + (kk & 3) * 32) >> 4;
            const uint32_t bo = ((kk >> 2) * kQtChunkBytes + (kk & 3) * 32) >> 4;
            umma_bf16(d, a0 + ao, b0 + bo, idesc_s, (sq != 0 || kk != 0) ? 1u : 0u);
          }
        }
        __syncwarp();
      }
      if (elect_one()) {
        umma_commit(&bar[kBarSFull + (ns & 1)]);
        if (sg.next(t) >= sg.hi) umma_commit(&bar[kBarQEmpty]);
      }
      __syncwarp();
    }
  }
}

template <bool kPaged>
__device__ void value_mma_role(const WindowParams &p, const Shared &sh, uint32_t tmem, int iq, const Range &range) {
  uint64_t *bar = sh.bar;
  constexpr uint32_t idesc_o = idesc_bf16_f32(128, kRows, true, true);
  const uint32_t c_base = smem_u32(sh.slot(0));
  const uint32_t p_base = smem_u32(sh.pbuf(0));
  uint32_t no = 0, o_use = 0;
  SegIter<kPaged> it(range, iq);
  Seg sg;
  while (it.next(p, sg)) {
    if (sg.empty) continue;
    if (!wait_warp(&bar[kBarOEmpty], (o_use & 1) ^ 1, sh, p.status)) return;
    for (int t = sg.lo; t < sg.hi; t = sg.next(t), ++no) {
      if (!wait_warp(&bar[kBarPFull + (no & 1)], (no >> 1) & 1, sh, p.status)) return;
      tc_fence_after();
      // O^T[latent, heads] += C_tile^T * P^T, four 128-lane latent blocks, K = 64 rows.
      // A = C_tile^T: latent (M) along the 128-byte rows, 64-wide atoms LBO apart; cache
      // rows (K) in 8-row groups.  B = P^T: heads (N) along the 128-byte rows, rows (K) in
      // 8-row groups.  A K step of 16 rows advances both by 2 KB (128 in descriptor units).
      const uint64_t b0 = sw128_desc(p_base + (no & 1) * kPBytes, kPBytes, 1024);
      uint64_t a0[kSlotQuarters];
      uint32_t rp[kSlotQuarters];
#pragma unroll
      for (int mb = 0; mb < kSlotQuarters; ++mb) {
        rp[mb] = ring_pos(no * kSlotQuarters + mb);
        a0[mb] = sw128_desc(c_base + rp[mb] * kSlotBytes, kAtomBytes, 1024);
      }
      const uint32_t acc0 = (t > sg.lo) ? 1u : 0u;
      if (elect_one()) {
#pragma unroll
        for (int mb = 0; mb < kSlotQuarters; ++mb) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            umma_bf16(tmem + kTmemO + mb * kRows, a0[mb] + kk * 128, b0 + kk * 128, idesc_o, kk > 0 ? 1u : acc0);
          umma_commit(&bar[kBarCEmpty + rp[mb]]);
        }
        umma_commit(&bar[kBarPEmpty + (no & 1)]);
        if (sg.next(t) >= sg.hi) umma_commit(&bar[kBarOFull]);
      }
      __syncwarp();
    }
    ++o_use;
  }
}

// ------------------------------------------------------------------ softmax + epilogue (warps 2-9)
// Two warpgroups; warpgroup wg owns head columns [32 wg, 32 wg + 32) of S^T and O^T.  Warp
// quadrant wq holds tile rows 16 wq .. 16 wq + 15 (the M = 64 accumulator layout); thread t
// owns rows 16 wq + t/4 and 16 wq + t/4 + 8 and the 8 head columns 8j + 2(t%4) + {0,1}.
// The running max per column lives in shared memory and in registers.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool kPaged>
__device__ void softmax_role(const WindowParams &p, const Shared &sh, uint32_t tmem, int g, int iq,
                             const Range &range, int warp, int lane) {
  uint64_t *bar = sh.bar;
  const int wg = (warp - 2) >> 2;              // warpgroup: head columns [32 wg, 32 wg + 32)
  const int wq = warp & 3;                     // TMEM lane quadrant of this warp
  const int tid = ((warp - 2) & 3) * 32 + lane;  // 0..127 within the warpgroup
  const int r0 = wq * 16 + (lane >> 2);        // tile rows r0 and r0 + 8 owned by this thread
  const int cq = lane & 3;                     // column pair within each 8-column block
  const uint32_t bar_id = 1 + wg;
  const int col0 = wg * 32;
  const uint32_t t_lane = tmem + ((uint32_t)(wq * 32) << 16);
  const uint32_t p_off = (uint32_t)r0 * 128 + cq * 4;
  float *red = sh.red;          // [4 quadrants][64 columns]
  float *m_used = sh.m_used;    // [64]
  float *alpha = sh.alpha;      // [64]
  uint32_t n = 0, o_use = 0;    // tiles seen by this CTA, segments finished
  if (tid < 32) m_used[col0 + tid] = kLowest;
  named_bar_sync(bar_id, 128);
  SegIter<kPaged> it(range, iq);
  Seg sg;
  while (it.next(p, sg)) {
    if (sg.empty) {
      // no visible tile: an empty partial (weight zero in the merge)
      if (tid < 32) {
        const long long slot = split::partial_slot(p, kModePaged, g, sg.s, iq);
        p.part_m[slot * kRows + col0 + tid] = -INFINITY;
        p.part_l[slot * kRows + col0 + tid] = 0.f;
      }
      continue;
    }
    float l_part[8], m_reg[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      l_part[c] = 0.f;
      m_reg[c] = kLowest;
    }
    for (int t = sg.lo; t < sg.hi; t = sg.next(t), ++n) {
      const uint32_t sb = n & 1;
      mbar_wait(&bar[kBarSFull + sb], (n >> 1) & 1, sh.abort_flag, p.status);
      tc_fence_after();
      const int j0 = sg.tile(t) * kTile + r0;
      const bool v0 = sg.q.row(j0), v1 = sg.q.row(j0 + 8);
      float s2[16];
      {
        uint32_t r[16];
        tmem_ld16x256_x4(t_lane + kTmemS + sb * kRows + col0, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s2[4 * j + 0] = v0 ? __uint_as_float(r[4 * j + 0]) * p.scale_log2 : -INFINITY;
          s2[4 * j + 1] = v0 ? __uint_as_float(r[4 * j + 1]) * p.scale_log2 : -INFINITY;
          s2[4 * j + 2] = v1 ? __uint_as_float(r[4 * j + 2]) * p.scale_log2 : -INFINITY;
          s2[4 * j + 3] = v1 ? __uint_as_float(r[4 * j + 3]) * p.scale_log2 : -INFINITY;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kBarSEmpty + sb]);
      // column h = 2j + e of this thread (j: 8-column block, e: pair member)
      bool flag = false;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          flag |= fmaxf(s2[4 * j + e], s2[4 * j + 2 + e]) > m_reg[2 * j + e] + kTau;
      const bool any = named_bar_or(bar_id, 128, flag);
      if (any) {
        // new running max for this warpgroup's 32 columns
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s2[4 * j + e], s2[4 * j + 2 + e]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            if (lane < 4) red[wq * kRows + col0 + 8 * j + 2 * cq + e] = mx;
          }
        named_bar_sync(bar_id, 128);
        if (tid < 32) {
          const int c = col0 + tid;
          const float mt = fmaxf(fmaxf(red[c], red[kRows + c]), fmaxf(red[2 * kRows + c], red[3 * kRows + c]));
          const float mo = m_used[c];
          const float mn = fmaxf(mo, mt);
          alpha[c] = fast_exp2(mo - mn);
          m_used[c] = mn;
        }
        named_bar_sync(bar_id, 128);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = col0 + 8 * j + 2 * cq + e;
            l_part[2 * j + e] *= alpha[c];
            m_reg[2 * j + e] = m_used[c];
          }
      }
      // probabilities, rounded to bf16 for the value product.
      // They are computed into registers first: the wait for this P buffer (the value
      // product of tile n-2) then overlaps the exponentials instead of preceding them.
      uint32_t pw[8];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // h = 0: row r0, h = 1: row r0 + 8
          const float x0 = s2[4 * j + 2 * h], x1 = s2[4 * j + 2 * h + 1];
          const float p0 = (x0 == -INFINITY) ? 0.f : fast_exp2(x0 - m_reg[2 * j]);
          const float p1 = (x1 == -INFINITY) ? 0.f : fast_exp2(x1 - m_reg[2 * j + 1]);
          const uint32_t w = pack_bf16x2(p0, p1);
          // the sum takes the weights unrounded: lse is exact to fp32, and o's error the same (2^-9
          // a weight) either way
          l_part[2 * j] += p0;
          l_part[2 * j + 1] += p1;
          pw[2 * j + h] = w;
        }
      // this P buffer is free (the value product of tile n-2 has finished)
      mbar_wait(&bar[kBarPEmpty + sb], ((n >> 1) & 1) ^ 1, sh.abort_flag, p.status);
      if (any && t > sg.lo) {
        // running max moved: once the value product of tile n-1 has finished, rescale this
        // warpgroup's O^T columns in TMEM
        mbar_wait(&bar[kBarPEmpty + (sb ^ 1)], ((n - 1) >> 1) & 1, sh.abort_flag, p.status);
        tc_fence_after();
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          uint32_t r[32];
          const uint32_t addr = t_lane + kTmemO + mb * kRows + col0;
          tmem_ld32(addr, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * alpha[col0 + j]);
          tmem_st32(addr, r);
        }
        tmem_st_wait();
      }
      const uint32_t pb = smem_u32(sh.pbuf(sb)) + p_off;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t sw = (uint32_t)(((wg * 4 + j) ^ (r0 & 7)) << 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) st_shared_b32(pb + h * 8 * 128 + sw, pw[2 * j + h]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[kBarPFull + sb]);
    }
    // ---- epilogue: l column sums, partial O, (m, l) -> workspace
    mbar_wait(&bar[kBarOFull], o_use & 1, sh.abort_flag, p.status);
    tc_fence_after();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l_part[2 * j + e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (lane < 4) red[wq * kRows + col0 + 8 * j + 2 * cq + e] = v;
      }
    named_bar_sync(bar_id, 128);
    const long long slot = split::partial_slot(p, kModePaged, g, sg.s, iq);
    if (tid < 32) {
      const int c = col0 + tid;
      p.part_m[slot * kRows + c] = m_used[c];
      p.part_l[slot * kRows + c] = red[c] + red[kRows + c] + red[2 * kRows + c] + red[3 * kRows + c];
    }
    float *po = p.part_o + slot * kRows * kLatent;
#pragma unroll 1
    for (int mb = 0; mb < 4; ++mb) {
      uint32_t r[32];
      tmem_ld32(t_lane + kTmemO + mb * kRows + col0, r);
      tmem_ld_wait();
      const int lat = mb * 128 + wq * 32 + lane;
#pragma unroll
      for (int j = 0; j < 32; ++j) po[(col0 + j) * kLatent + lat] = __uint_as_float(r[j]);
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[kBarOEmpty]);
    ++o_use;
    named_bar_sync(bar_id, 128);
    if (tid < 32) m_used[col0 + tid] = kLowest;
    named_bar_sync(bar_id, 128);
  }
}

// ------------------------------------------------------------------ kernel
template <bool kPaged>
// Bounds for 384 threads: eleven warps put three on some SM sub-partitions, whose 16K registers then
// cap a thread at 168, and the bound of 352 threads would let the compiler give it 184, with which no
// launch would succeed.  Both forms use 156 with either bound.
__global__ void __launch_bounds__(384, 1)
    attend_window_kernel(const __grid_constant__ CUtensorMap tm_cache, const __grid_constant__ CUtensorMap tm_qt,
                         const WindowParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Shared sh;
  sh.base = base;
  sh.bar = reinterpret_cast<uint64_t *>(base + kOffBar);
  sh.red = reinterpret_cast<float *>(base + kOffRed);
  sh.m_used = reinterpret_cast<float *>(base + kOffMUsed);
  sh.alpha = reinterpret_cast<float *>(base + kOffAlpha);
  sh.tmem_slot = reinterpret_cast<uint32_t *>(base + kOffMisc);
  sh.abort_flag = reinterpret_cast<volatile int *>(base + kOffMisc + 4);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = blockIdx.x / p.group_size;
  const int iq = blockIdx.x % p.group_size;

  if (threadIdx.x == 0) {
    for (int c = 0; c < kSlots; ++c) {
      mbar_init(&sh.bar[kBarCFull + c], 1);
      mbar_init(&sh.bar[kBarCEmpty + c], 1);
    }
    mbar_init(&sh.bar[kBarQFull], 1);
    mbar_init(&sh.bar[kBarQEmpty], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.bar[kBarSFull + i], 1);
      mbar_init(&sh.bar[kBarSEmpty + i], kSoftmaxWarps);
      mbar_init(&sh.bar[kBarPFull + i], kSoftmaxWarps);
      mbar_init(&sh.bar[kBarPEmpty + i], 1);
    }
    mbar_init(&sh.bar[kBarOFull], 1);
    mbar_init(&sh.bar[kBarOEmpty], kSoftmaxWarps);
    mbar_init(&sh.bar[kBarDrain], 2);
    *sh.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(sh.tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  grid_dep_launch();
  grid_dep_wait();  // inputs (q~, lengths, tables, cache) may come from the previous kernel
  Range *range = reinterpret_cast<Range *>(base + kOffRange);
  if (warp == 0) {
    // This warp initialised the barriers and finds the CTA's range: it starts loading at once.  Not on
    // barrier 0: with nothing to load it may be at the block's last barrier before the others
    // are at this one.
    const Range r = lists::find_range<Seqs<kPaged>>(p, g, lane);
    if (lane == 0) {
      *range = r;
      prefetch_tensormap(&tm_qt);
      prefetch_tensormap(&tm_cache);
    }
    __syncwarp();
    asm volatile("bar.arrive 4, %0;" ::"n"(kThreads) : "memory");
    if (lane == 0) producer_role<kPaged>(p, sh, &tm_cache, &tm_qt, iq, r);
  } else {
    tc_fence_before();
    asm volatile("bar.sync 4, %0;" ::"n"(kThreads) : "memory");
    tc_fence_after();
  }
  const uint32_t tmem = *sh.tmem_slot;
  const Range r = *range;

  if (warp == 0) {
    // done above
  } else if (warp == 1) {
    score_mma_role<kPaged>(p, sh, tmem, iq, r, lane);
  } else if (warp == 10) {
    if (blockIdx.x == 0) lists::write_partial_table<Seqs<kPaged>>(p, lane);  // needed last: there is time
    value_mma_role<kPaged>(p, sh, tmem, iq, r);
  } else {
    softmax_role<kPaged>(p, sh, tmem, g, iq, r, warp, lane);
  }

  __syncwarp();
  // After an abort, the MMAs issued by the two MMA warps (lane 0 of each) must finish
  // before TMEM is released: each commits to the drain barrier, warp 1 waits for both.
  // (The producer has already waited for its copies.)
  if (warp == 10 && *sh.abort_flag) {
    if (lane == 0) umma_commit(&sh.bar[kBarDrain]);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (*sh.abort_flag) {
      if (lane == 0) {
        umma_commit(&sh.bar[kBarDrain]);
        if (!mbar_wait_drain(&sh.bar[kBarDrain], 0)) report_status(p.status, kStatusTimeout);
      }
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace windowed

template <bool kPaged>
static cudaError_t launch_window(const CUtensorMap &tm_cache, const CUtensorMap &tm_qt, const WindowParams &p,
                                 cudaStream_t stream) {
  static std::atomic<int> configured_device{-1};
  const cudaError_t e0 =
      set_smem_limit_once(windowed::attend_window_kernel<kPaged>, windowed::kSmemBytes, configured_device);
  if (e0 != cudaSuccess) return e0;
  if (cudaError_t e = launch_chained(windowed::attend_window_kernel<kPaged>, dim3(p.groups * p.group_size),
                                     dim3(windowed::kThreads), windowed::kSmemBytes, stream, tm_cache, tm_qt, p);
      e != cudaSuccess)
    return e;
  return lists::launch_combine<windowed::Seqs<kPaged>, windowed::PartialOrder>(p, 1.f, stream);
}

cudaError_t launch_attend_window(bool paged, const CUtensorMap &tm_cache, const CUtensorMap &tm_qt,
                                 const WindowParams &p, cudaStream_t stream) {
  return paged ? launch_window<true>(tm_cache, tm_qt, p, stream) : launch_window<false>(tm_cache, tm_qt, p, stream);
}

}  // namespace mla
