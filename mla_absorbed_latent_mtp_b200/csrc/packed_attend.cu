// packed_attend.cu -- split-L latent attention over the 4-bit paged cache (packed.cuh):
//   s_j = scale q~ . c_j,  a = softmax over the rows a query sees (window.cuh),  o = sum_j a_j c_j.
//
// Work decomposition: as attend.cu (a list of the tiles of all sequences, split into equal
// ranges over CTA groups of one CTA per query of a verify window; partials in the workspace;
// a combine kernel), with tiles of 128 rows, two pages.
//
// What bounds it.  A tile is 36 KB of cache but 16.8 MFLOP per query, 2,048 cycles of the
// tensor core at N = 64: bytes cost at most half of that, so the kernel has to keep the MMAs
// fed.  An MMA that reads both operands from shared memory takes 48.5 cycles (M = 128, N = 64,
// measured back to back), with its A operand in tensor memory 32.4, the full rate; and 4-bit
// codes cannot be an operand as they are, since each row has its own scales.  So the cache
// operand is unpacked into TENSOR memory, twice, by register, and shared memory holds only the
// packed rows, q~ and P.  Measured: 5,300 cycles a tile, 2.6 times the MMAs' own; the rest is the
// unpacking, the softmax and the hand-overs between them (3,070 instructions a tile and scheduler),
// the spills of the roles that 96 registers are too few for among them (524 bytes of stores and 500
// of loads in the kernel; 1.15 of 30.0 million instructions executed for 32 x 8,192 rows).
// With the merge 32 x 8,192 rows take 67 us (bf16 rows, attend.cu: 65), 16 sequences of 1.05 M rows
// in all 193 us at 1,965 MHz (216 at the 1,755 MHz that the power cap leaves in a long run), 16 x 6
// queries with a window of 8,191 rows and 64 sinks 145 us (150 at 1,890 MHz).
//   S^T[rows, heads]    = C (A: 128 rows on the lanes, 64 latents a chunk) * Q~^T (smem)
//   O^T[latent, heads] += C^T (A: 128 latents on the lanes, 16 rows a chunk, x 4) * P^T (smem)
// Both unpackings read the same packed words.  For C a thread owns a row.  For C^T a thread
// reads the eight bytes of one scale group (16 latents) of four rows, interleaves the nibbles
// of two rows so that one conversion yields the pair (row, row + 1) of a latent, and stores
// its 4 x 4 block by a 16x256b tensor-memory store; which latent lands on which lane is free,
// since O^T's lanes only have to be read back the same way (PartialOrder).
//
// Operands are fp16: code * scale is exact there.  q~ (bf16) is converted once per segment with
// a power of two per head that puts the head's largest value in [2^14, 2^15): exact unless a
// value is 2^-31 of the largest or less.  P is p * 2^7 in fp16, p = 2^(score - running max) <= 2^8
// under the lazy rescale, so at most 2^15.  From p = 2^-21 down it is rounded by at most 2^-32 (fp16's
// subnormal range) instead of 2^-11 of itself, and below 2^-32 to zero, while the head's largest p is
// at least 1.  The row sums stay in fp32 of the unrounded p.
//
// Per CTA 19 warps (five on a scheduler: 96 registers a thread): 0 TMA loads, 1 score MMAs, 2 value
// MMAs, 3-10 softmax (two groups of four warps, 32 heads each; they also convert q~ and write
// the partials), 11-14 unpack C, 15-18 unpack C^T.
#include <math.h>

#include <algorithm>

#include "internal.h"
#include "lists.cuh"
#include "packed.cuh"
#include "packed_attend.h"
#include "sm100.cuh"
#include "split.cuh"
#include "window.cuh"

namespace mla {
namespace packed {

constexpr int kTile = 128;                      // rows per tile: two pages
constexpr int kRawSlots = 3;
constexpr int kHalfBytes = kTile * 128;                     // 16 KB: 128 rows of 128 code bytes, 128-byte swizzle
constexpr int kPageScaleBytes = kPageTokens * kScaleBytes;  // 2 KB
constexpr int kRawCodeBytes = 2 * kHalfBytes;
constexpr int kRawBytes = kRawCodeBytes + 2 * kPageScaleBytes;  // 36 KB
constexpr int kQChunkBytes = kHeads * 128;      // 8 KB: 64 heads x 64 latents
constexpr int kPBytes = kTile * 128;            // 16 KB: 128 rows x 64 heads
constexpr int kChunks = 8;                      // chunks per tile, of C and of C^T
constexpr int kStage = 3;                       // operand chunks in tensor memory, each 32 columns
constexpr int kThreads = 608;
constexpr int kSoftmaxWarps = 8;
constexpr float kTau = 8.f;                     // the running max is raised when a score exceeds it by this
constexpr float kShift = 7.f;                   // P is stored as 2^7 p

constexpr int kOffQ = kRawSlots * kRawBytes;
constexpr int kOffP = kOffQ + 8 * kQChunkBytes;
constexpr int kOffRed = kOffP + 2 * kPBytes;    // [4][64] floats
constexpr int kOffM = kOffRed + 4 * 64 * 4;     // [64] floats: kShift less the running max (log2 units)
constexpr int kOffAlpha = kOffM + 64 * 4;
constexpr int kOffRise = kOffAlpha + 64 * 4;
constexpr int kOffCs = kOffRise + 64 * 4;      // [64] floats: score factor of each head
constexpr int kOffBar = kOffCs + 64 * 4;
constexpr int kBarRawFull = 0, kBarRawEmpty = kBarRawFull + kRawSlots, kBarSAFull = kBarRawEmpty + kRawSlots,
              kBarSAEmpty = kBarSAFull + kStage, kBarVAFull = kBarSAEmpty + kStage,
              kBarVAEmpty = kBarVAFull + kStage, kBarQFull = kBarVAEmpty + kStage, kBarSFull = kBarQFull + 1,
              kBarSEmpty = kBarSFull + 1, kBarPFull = kBarSEmpty + 1, kBarPEmpty = kBarPFull + 2,
              kBarOFull = kBarPEmpty + 2, kBarOEmpty = kBarOFull + 1, kBarDrain = kBarOEmpty + 1,
              kNumBars = kBarDrain + 1;
constexpr int kOffMisc = kOffBar + kNumBars * 8;
constexpr int kOffRange = kOffMisc + 16;
constexpr int kSmemBytes = kOffRange + (int)sizeof(lists::Range) + 1024;  // slack for 1024-byte alignment of the base
static_assert(kSmemBytes <= 232448, "shared memory budget");

// Tensor memory columns.
constexpr uint32_t kTmemS = 0, kTmemSA = 64, kTmemVA = kTmemSA + 32 * kStage, kTmemO = 256, kTmemCols = 512;
static_assert(kTmemVA + 32 * kStage <= kTmemO, "tensor memory budget");

using SeqTiles = window::SeqTiles<kTile>;
using QueryTiles = window::QueryTiles<kTile>;

// Lane L of block mb of O^T holds latent 16 (8 (L / 32) + L % 8) + 4 mb + (L % 32) / 8; a
// partial is stored in (block, lane) order.
struct PartialOrder {
  static __device__ __forceinline__ int latent(int idx) {
    const int mb = idx / 128, L = idx % 128;
    return kGroup * (8 * (L / 32) + L % 8) + 4 * mb + L % 32 / 8;
  }
  // Stored place of the first of four values of thread t (of 32) in quarter `part` of the latents.
  static __device__ __forceinline__ int unit(int part, int t) { return 128 * (t / 8) + 32 * part + 4 * (t % 8); }
};

// Instruction descriptor, kind::f16 with fp16 A and B and fp32 D.
constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Tensor-memory store of a 16-lane half quadrant, 32 columns: thread t stores, for column block
// j of 8, lane base + t/4 in r[4j], r[4j+1] (columns 8j + 2(t%4) and +1) and lane base + t/4 + 8
// in r[4j+2], r[4j+3].
__device__ __forceinline__ void tmem_st16x256_x4(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of floats in one instruction: d = a b + c, d += a.
__device__ __forceinline__ void fma_f32x2(float &d0, float &d1, float a0, float a1, float b0, float b1, float c0,
                                          float c1) {
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add_f32x2(float &d0, float &d1, float a0, float a1) {
  asm("{\n\t.reg .b64 a, d;\n\tmov.b64 d, {%0, %1};\n\tmov.b64 a, {%2, %3};\n\tadd.rn.f32x2 d, d, a;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "+f"(d0), "+f"(d1)
      : "f"(a0), "f"(a1));
}

// ------------------------------------------------------------------ the tile list
struct Seqs {  // for lists.cuh
  static constexpr int kStart = 3;
  static __device__ __forceinline__ int length(const AttendPackedParams &p, int b) {
    return min(max(p.seq_lens[b], 0), p.max_pages * kPageTokens);
  }
  static __device__ __forceinline__ int tiles(const AttendPackedParams &p, int L) {
    return SeqTiles(L, p.Q, p.window, p.sinks).count;
  }
  static __device__ __forceinline__ bool bad_length(const AttendPackedParams &p, int b) {
    return p.seq_lens[b] < 0 || p.seq_lens[b] > p.max_pages * kPageTokens;
  }
};
using lists::Range;

// Walks the segments (the pieces of sequences) of the list range [t, t_end).  A segment's tiles
// for this CTA's query are n = first(), then next(n), below hi; none: its partial is empty.
struct Segment {
  int b, lo, hi;
  QueryTiles q;
  __device__ __forceinline__ int first() const { return q.seek(lo); }
  __device__ __forceinline__ int next(int n) const { return q.seek(n + 1); }
  __device__ __forceinline__ int count() const {
    return max(min(hi, q.a) - lo, 0) + max(hi - max(lo, q.b), 0);
  }
};
struct SegIter {
  long long t, t_end, base;
  int s, L, start, iq;
  __device__ SegIter(const Range &r, int iq_)
      : t(r.t0), t_end(r.t1), base(r.base), s(r.s), L(r.L), start(r.start), iq(iq_) {}
  __device__ bool next(const AttendPackedParams &p, Segment &sg) {
    if (t >= t_end) return false;
    int n = lists::places<Seqs>(p, L, start);
    while (base + n <= t) {
      base += n;
      L = Seqs::length(p, ++s);
      n = lists::places<Seqs>(p, L, start);
    }
    sg.b = s;
    sg.q = QueryTiles(L, p.Q, iq, p.window, p.sinks);
    sg.lo = max((int)(t - base) - start, 0);
    const int end = (int)min(t_end - base, (long long)n);
    sg.hi = min(max(end - start, 0), sg.q.e);
    t = base + end;
    return true;
  }
};

// ------------------------------------------------------------------ shared state
struct Shared {
  uint8_t *base;
  uint64_t *bar;
  float *red, *m, *alpha, *rise, *cs;
  const Range *range;
  uint32_t *tmem_slot;
  volatile int *abort_flag;
};

// Barriers are addressed by their shared-memory address and index.  A wait is one probe on the
// fast path; what follows a failed probe is out of line, since the roles' code competes for the
// instruction cache.  After an abort (a wait that expired anywhere in the CTA) every wait
// returns at once and the roles run to their end on whatever they find: shared memory and
// tensor memory stay theirs, no copy or MMA is issued any more, and *status says so.
struct Bars {
  uint32_t addr;
  volatile int *abort_flag;
  int32_t *status;
  __device__ __forceinline__ uint32_t operator[](uint32_t i) const { return addr + 8 * i; }
};
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *status) {
  const long long t0 = clock64();
  while (true) {
    if (*abort_flag) return false;
    if (mbar_try_wait_sleep(bar, parity, 1000000u)) return true;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort_flag = 1;
      report_status(status, kStatusTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(const Bars &bar, uint32_t i, uint32_t parity) {
  if (mbar_test_wait(bar[i], parity)) return true;
  return wait_slow(bar[i], parity, bar.abort_flag, bar.status);
}
// The same for a converged warp: true if it completed for every lane.
__device__ __forceinline__ bool wait_warp(const Bars &bar, uint32_t i, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(bar, i, parity));
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}

// A ring position: slot and phase.
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void step(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      phase ^= 1;
    }
  }
};

// ------------------------------------------------------------------ loads (warp 0)
// The warp reads the page ids of 16 tiles at a time, lane 0 issues the copies.  A page without a
// visible row is not loaded (it need not be mapped).
__device__ void producer_role(const AttendPackedParams &p, const Shared &sh, const CUtensorMap *tm_codes,
                              const CUtensorMap *tm_scales, int iq, int lane) {
  const Bars bar{smem_u32(sh.bar), sh.abort_flag, p.status};
  Ring raw;
  uint32_t issued = 0;
  SegIter it(*sh.range, iq);
  Segment sg;
  while (it.next(p, sg)) {
    const int32_t *table = p.page_table + (long long)sg.b * p.max_pages;
    const int count = sg.count();
    int n = sg.first();
    for (int k0 = 0; k0 < count; k0 += 16) {
      // lane: page lane % 2 of the tile lane / 2 further on (past tile a the list goes on at b)
      int ahead = n + lane / 2;
      if (n < sg.q.a && ahead >= sg.q.a) ahead += sg.q.b - sg.q.a;
      int id = -1;  // not loaded
      if (k0 + lane / 2 < count) {
        const int pg = sg.q.seq.tile(ahead) * (kTile / kPageTokens) + lane % 2;
        if (sg.q.any_row(pg * kPageTokens, kPageTokens)) {
          id = table[pg];
          if (id < 0 || id >= p.num_pages) {
            report_status(p.status, kStatusIndex);
            id = 0;
          }
        }
      }
      for (int k = 0; k < 16 && k0 + k < count; ++k, n = sg.next(n)) {
        const int page[2] = {__shfl_sync(0xffffffffu, id, 2 * k), __shfl_sync(0xffffffffu, id, 2 * k + 1)};
        if (!wait_warp(bar, kBarRawEmpty + raw.slot, raw.phase ^ 1)) goto done;
        if (lane == 0) {
          uint8_t *dst = sh.base + raw.slot * kRawBytes;
          uint64_t *full = &sh.bar[kBarRawFull + raw.slot];
          mbar_arrive_expect_tx(full, ((page[0] >= 0) + (page[1] >= 0)) * kPageBytes);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (page[h] < 0) continue;
            const int row = page[h] * kPageTokens;
            tma_load_3d(dst + h * (kHalfBytes / 2), tm_codes, full, 0, row, 0);
            tma_load_3d(dst + kHalfBytes + h * (kHalfBytes / 2), tm_codes, full, 0, row, 1);
            tma_load_2d(dst + kRawCodeBytes + h * kPageScaleBytes, tm_scales, full, 0, row);
          }
        }
        __syncwarp();
        raw.step(kRawSlots);
        ++issued;
      }
    }
  }
done:
  if (lane == 0 && !drain_ring(&sh.bar[kBarRawFull], kRawSlots, issued)) report_status(p.status, kStatusTimeout);
}

// ------------------------------------------------------------------ MMA issuers (warps 1 and 2)
__device__ void score_mma_role(const AttendPackedParams &p, const Shared &sh, uint32_t tmem, int iq) {
  const Bars bar{smem_u32(sh.bar), sh.abort_flag, p.status};
  constexpr uint32_t idesc = idesc_f16_f32(kTile, kHeads, false);
  const uint64_t b0 = sw128_desc(smem_u32(sh.base + kOffQ), 16, 1024);
  Ring st;
  uint32_t tiles = 0, segs = 0;
  SegIter it(*sh.range, iq);
  Segment sg;
  while (it.next(p, sg)) {
    const int count = sg.count();
    if (count == 0) continue;
    if (!wait_warp(bar, kBarQFull, segs & 1)) return;
    ++segs;
    for (int k = 0; k < count; ++k, ++tiles) {
      if (!wait_warp(bar, kBarSEmpty, (tiles & 1) ^ 1)) return;
#pragma unroll 1
      for (uint32_t ch = 0; ch < kChunks; ++ch) {
        if (!wait_warp(bar, kBarSAFull + st.slot, st.phase)) return;
        tc_fence_after();
        const uint32_t a = tmem + kTmemSA + st.slot * 32;
        const uint64_t b = b0 + ch * (kQChunkBytes / 16);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16_tmem_a(tmem + kTmemS, a + kk * 8, b + kk * 2, idesc, (ch != 0 || kk != 0) ? 1u : 0u);
          umma_commit(&sh.bar[kBarSAEmpty + st.slot]);
          if (ch == kChunks - 1) umma_commit(&sh.bar[kBarSFull]);
        }
        __syncwarp();
        st.step(kStage);
      }
    }
  }
}

__device__ void value_mma_role(const AttendPackedParams &p, const Shared &sh, uint32_t tmem, int iq) {
  const Bars bar{smem_u32(sh.bar), sh.abort_flag, p.status};
  constexpr uint32_t idesc = idesc_f16_f32(128, kHeads, true);
  const uint64_t b0 = sw128_desc(smem_u32(sh.base + kOffP), kPBytes, 1024);
  Ring st;
  uint32_t tiles = 0, segs = 0;
  SegIter it(*sh.range, iq);
  Segment sg;
  while (it.next(p, sg)) {
    const int count = sg.count();
    if (count == 0) continue;
    if (!wait_warp(bar, kBarOEmpty, (segs & 1) ^ 1)) return;
    ++segs;
    for (int k = 0; k < count; ++k, ++tiles) {
      if (!wait_warp(bar, kBarPFull + (tiles & 1), (tiles >> 1) & 1)) return;
#pragma unroll 1
      for (uint32_t ks = 0; ks < kChunks; ++ks) {
        if (!wait_warp(bar, kBarVAFull + st.slot, st.phase)) return;
        tc_fence_after();
        const uint32_t a = tmem + kTmemVA + st.slot * 32;
        const uint64_t b = b0 + (tiles & 1) * (kPBytes / 16) + ks * (16 * 128 / 16);
        const uint32_t acc = (k == 0 && ks == 0) ? 0u : 1u;
        if (elect_one()) {
#pragma unroll
          for (int mb = 0; mb < 4; ++mb)
            umma_bf16_tmem_a(tmem + kTmemO + mb * kHeads, a + mb * 8, b, idesc, acc);
          umma_commit(&sh.bar[kBarVAEmpty + st.slot]);
          if (ks == kChunks - 1) {
            umma_commit(&sh.bar[kBarPEmpty + (tiles & 1)]);
            if (k == count - 1) umma_commit(&sh.bar[kBarOFull]);
          }
        }
        __syncwarp();
        st.step(kStage);
      }
    }
  }
}

// ------------------------------------------------------------------ unpack C (warps 11-14)
// Both unpackers read the next chunk's words from shared memory before they convert this one's
// (the last chunk reads the first again, to no use).  The chunk loops are unrolled by two: with
// five kinds of warps on a scheduler, fully unrolled bodies missed the instruction cache (32 x
// 8,192 rows: 117 us with all eight chunks unrolled, 78 rolled when that was tried; 16 ragged
// sequences later 218 us rolled, 211 by two).
struct Stager {
  Bars bar;
  uint32_t full, empty;  // barrier indexes of slot 0
  Ring st;
  // The slot, once the MMAs that read its last chunk are done.
  __device__ __forceinline__ uint32_t acquire() {
    wait(bar, empty + st.slot, st.phase ^ 1);
    __syncwarp();
    tc_fence_after();
    return st.slot;
  }
  __device__ __forceinline__ void hand_over(int lane) {
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive(bar[full + st.slot]);
    st.step(kStage);
  }
};

// Thread = row.  A chunk is 64 latents: 32 bytes of codes, four scales, 32 columns.
__device__ void unpack_rows_role(const AttendPackedParams &p, const Shared &sh, uint32_t tmem, int iq, int wq,
                                 int lane) {
  const Bars bar{smem_u32(sh.bar), sh.abort_flag, p.status};
  const int row = wq * 32 + lane;
  const uint32_t raw0 = smem_u32(sh.base);
  const uint32_t code_off = row * 128 + ((row & 7) << 4);
  const uint32_t t_dst = tmem + ((uint32_t)(wq * 32) << 16) + kTmemSA;
  Ring raw;
  Stager out{bar, kBarSAFull, kBarSAEmpty, Ring()};
  SegIter it(*sh.range, iq);
  Segment sg;
  while (it.next(p, sg)) {
    for (int n = sg.first(); n < sg.hi; n = sg.next(n)) {
      wait(bar, kBarRawFull + raw.slot, raw.phase);
      __syncwarp();
      const uint32_t base = raw0 + raw.slot * kRawBytes;
      uint4 w0, w1;
      uint32_t sc;
      auto load = [&](int ch) {
        const uint32_t at = (base + code_off + (ch >> 2) * kHalfBytes) ^ ((ch & 3) << 5);
        w0 = ld_shared_v4(at);
        w1 = ld_shared_v4(at ^ 16);
        sc = ld_shared_u32(base + kRawCodeBytes + row * kScaleBytes + 4 * ch);
      };
      load(0);
#pragma unroll 2
      for (int ch = 0; ch < kChunks; ++ch) {
        const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
        const uint32_t s01 = e4m3x2_to_f16x2(sc & 0xFFFFu), s23 = e4m3x2_to_f16x2(sc >> 16);
        load((ch + 1) % kChunks);
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // words 2g, 2g + 1 share group g's scale
          const uint32_t s = prmt(i < 4 ? s01 : s23, 0, (i & 2) ? 0x3232u : 0x1010u);
          uint32_t v[4];
          e2m1x8_to_f16x2(w[i], v);
#pragma unroll
          for (int k = 0; k < 4; ++k) r[4 * i + k] = mul_f16x2(v[k], s);
        }
        tmem_st32(t_dst + out.acquire() * 32, r);
        out.hand_over(lane);
      }
      if (lane == 0) arrive(bar[kBarRawEmpty + raw.slot]);
      raw.step(kRawSlots);
    }
  }
}

// ------------------------------------------------------------------ unpack C^T (warps 15-18)
// A chunk is 16 rows, the K step of four MMAs.  Thread (warp wq, g = lane / 4, c = lane % 4)
// owns scale group 8 wq + g of rows 2c, 2c + 1, 2c + 8, 2c + 9 of the chunk, which are K
// indexes 4c .. 4c + 3: with the rows two apart over c, a half warp's eight-byte loads hit
// every bank once under the 128-byte swizzle.  (P's rows are stored in the same K order.)
// Rows the query does not see get the scale zero, so that whatever they hold (a NaN scale, or
// a page that was not loaded) meets their zero probability as a zero.
__device__ __forceinline__ int k_of_row(int r) {  // K index of tile row r
  return (r & ~15) | ((r & 6) << 1) | ((r & 8) >> 2) | (r & 1);
}

__device__ void unpack_latents_role(const AttendPackedParams &p, const Shared &sh, uint32_t tmem, int iq, int wq,
                                    int lane) {
  const Bars bar{smem_u32(sh.bar), sh.abort_flag, p.status};
  const int g = lane >> 2, c = lane & 3;
  const int group = 8 * wq + g;
  // the group's eight bytes in a row: half, 16-byte unit, which eight of it; the thread's rows of
  // a chunk are 2c + b + 8h, whose unit is the same for both h
  const uint32_t unit = 4 * (wq & 1) + (g >> 1);
  const uint32_t off0 = (wq >> 1) * kHalfBytes + (g & 1) * 8 + (2 * c) * 128;
  const uint32_t row_off[2] = {off0 + ((unit ^ (2 * c)) << 4), off0 + 128 + ((unit ^ (2 * c + 1)) << 4)};
  const uint32_t scale_off = kRawCodeBytes + (2 * c) * kScaleBytes + group;
  const uint32_t raw0 = smem_u32(sh.base);
  const uint32_t t_dst = tmem + ((uint32_t)(wq * 32) << 16) + kTmemVA;
  Ring raw;
  Stager out{bar, kBarVAFull, kBarVAEmpty, Ring()};
  SegIter it(*sh.range, iq);
  Segment sg;
  while (it.next(p, sg)) {
    for (int n = sg.first(); n < sg.hi; n = sg.next(n)) {
      wait(bar, kBarRawFull + raw.slot, raw.phase);
      __syncwarp();
      const uint32_t base = raw0 + raw.slot * kRawBytes;
      const int j0 = sg.q.seq.tile(n) * kTile;
      const bool whole = sg.q.every_row(j0, kTile);
      uint2 w[4];
      uint32_t s[4];
      auto load = [&](int ks) {
        const uint32_t rows = base + ks * (16 * 128);
        const uint32_t sp = base + scale_off + ks * 16 * kScaleBytes;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // row 2c + k % 2 + 8 (k / 2)
          w[k] = ld_shared_v2(rows + row_off[k & 1] + (k >> 1) * (8 * 128));
          s[k] = ld_shared_u8(sp + ((k & 1) + 8 * (k >> 1)) * kScaleBytes);
        }
      };
      load(0);
#pragma unroll 2
      for (int ks = 0; ks < kChunks; ++ks) {
        if (!whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!sg.q.row(j0 + 16 * ks + 2 * c + (k & 1) + 8 * (k >> 1))) s[k] = 0;
        }
        // r[upper 16 lanes][4 * block + 2 * upper 8 lanes + column]
        uint32_t r[2][16];
        const uint32_t sp[2] = {e4m3x2_to_f16x2(prmt(s[0], s[1], 0x0040u)), e4m3x2_to_f16x2(prmt(s[2], s[3], 0x0040u))};
        const uint2 v[4] = {w[0], w[1], w[2], w[3]};
        load((ks + 1) % kChunks);
#pragma unroll
        for (int col = 0; col < 2; ++col) {  // rows 2 col, 2 col + 1 of this thread's four
#pragma unroll
          for (int word = 0; word < 2; ++word) {
            const uint32_t x = word ? v[2 * col].y : v[2 * col].x, y = word ? v[2 * col + 1].y : v[2 * col + 1].x;
            const uint32_t even = (x & 0x0F0F0F0Fu) | ((y << 4) & 0xF0F0F0F0u);
            const uint32_t odd = ((x >> 4) & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
            uint32_t ve[4], vo[4];
            e2m1x8_to_f16x2(even, ve);
            e2m1x8_to_f16x2(odd, vo);
            // latent 8 word + 2i (even) or + 1 (odd) of the group: block mb = latent / 4,
            // lane g + 8 (latent % 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int mb = 2 * word + (i >> 1), slot = 2 * (i & 1);  // slot: latent % 4 of the even one
              r[slot >> 1][4 * mb + col] = mul_f16x2(ve[i], sp[col]);
              r[slot >> 1][4 * mb + 2 + col] = mul_f16x2(vo[i], sp[col]);
            }
          }
        }
        const uint32_t dst = t_dst + out.acquire() * 32;
        tmem_st16x256_x4(dst, r[0]);
        tmem_st16x256_x4(dst + (16u << 16), r[1]);
        out.hand_over(lane);
      }
      if (lane == 0) arrive(bar[kBarRawEmpty + raw.slot]);
      raw.step(kRawSlots);
    }
  }
}

// ------------------------------------------------------------------ softmax (warps 3-10)
// q~ of this segment's query as fp16, K-major with 128-byte swizzle, and the factor that turns
// an MMA result into a score in log2 units.  Warp w converts heads 8w .. 8w + 7, four at a time.
__device__ __forceinline__ void convert_query(const AttendPackedParams &p, const Shared &sh, int b, int iq, int w,
                                              int lane) {
  const uint16_t *q = p.q_tilde + ((long long)b * p.Q + iq) * kHeads * kLatent;
  const uint32_t dst = smem_u32(sh.base + kOffQ);
#pragma unroll 1
  for (int h4 = 0; h4 < 8; h4 += 4) {
    uint4 v[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        v[i][u] = *reinterpret_cast<const uint4 *>(q + (8 * w + h4 + i) * kLatent + u * 256 + lane * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = 8 * w + h4 + i;
      uint32_t mx = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t x[4] = {v[i][u].x, v[i][u].y, v[i][u].z, v[i][u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = max(mx, max(x[k] & 0x7FFFu, (x[k] >> 16) & 0x7FFFu));
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      const int e = (int)(mx >> 7);  // the largest value lies in [2^(e - 127), 2^(e - 126))
      // factor 2^(141 - e) brings it to [2^14, 2^15); a head with an Inf or NaN is left as it is
      const int f = e == 255 ? 0 : min(141 - e, 126);
      const float up = __uint_as_float((uint32_t)(127 + f) << 23);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t x[4] = {v[i][u].x, v[i][u].y, v[i][u].z, v[i][u].w};
        uint32_t y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = pack_f16x2(bf16lo_to_f32(x[k]) * up, bf16hi_to_f32(x[k]) * up);
        const uint32_t chunk = 4 * u + (lane >> 3);
        st_shared_v4(dst + chunk * kQChunkBytes + h * 128 + (((lane & 7) ^ (h & 7)) << 4), y[0], y[1], y[2], y[3]);
      }
      if (lane == 0) sh.cs[h] = p.score_factor * __uint_as_float((uint32_t)(127 - f) << 23);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.bar[kBarQFull]);
}

// Sums each of 32 per-lane columns over the warp: lane l gets column l.
__device__ __forceinline__ float sum_columns(float (&v)[32], int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

__device__ void softmax_role(const AttendPackedParams &p, const Shared &sh, uint32_t tmem, int grp, int iq, int warp,
                             int lane) {
  const Bars bar{smem_u32(sh.bar), sh.abort_flag, p.status};
  const int w = warp - 3, wg = w >> 2, wq = warp & 3;
  const int tid = wq * 32 + lane;    // within the warpgroup
  const int row = wq * 32 + lane;    // tile row = tensor-memory lane
  const int col0 = wg * 32;          // heads [col0, col0 + 32), which this group's warps convert too
  const uint32_t bar_id = 1 + wg;
  const uint32_t t_lane = tmem + ((uint32_t)(wq * 32) << 16);
  const int krow = k_of_row(row);
  const uint32_t p_dst = smem_u32(sh.base + kOffP) + krow * 128;
  const float4 *cs4 = reinterpret_cast<const float4 *>(sh.cs + col0);
  const float4 *m4 = reinterpret_cast<const float4 *>(sh.m + col0);
  uint32_t tiles = 0, segs = 0;
  SegIter it(*sh.range, iq);
  Segment sg;
  long long slot = -1;  // of the partial whose O^T is still to be stored
  while (true) {
    // The next segment with tiles for this query; the partials of those without are empty.
    bool more;
    while ((more = it.next(p, sg)) && sg.first() >= sg.hi) {
      if (tid < 32) {
        const long long row = split::partial_slot(p, kModePaged, grp, sg.b, iq) * kHeads + col0 + tid;
        p.part_m[row] = -INFINITY;
        p.part_l[row] = 0.f;
      }
    }
    // The last segment's scores are done: this one's q~ takes the place of that one's before its
    // O^T is stored, so that the first scores are computed meanwhile (256 x 500 rows: 80.0 us with
    // the store first, 74.9 so; 32 x 8,192: 69.7, 69.2; against it 16 ragged sequences, 214 and 217,
    // and 16 x 6 queries, window 8,191 + 64, 149 and 152: the code has 524 bytes of spill stores
    // instead of 460).
    if (more) convert_query(p, sh, sg.b, iq, w, lane);
    if (slot >= 0) {
      wait(bar, kBarOFull, segs & 1);
      __syncwarp();
      tc_fence_after();
      float *po = p.part_o + slot * kHeads * kLatent;
#pragma unroll 1
      for (int mb = 0; mb < 4; ++mb) {
        uint32_t o[32];
        tmem_ld32(t_lane + kTmemO + mb * kHeads + col0, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) po[(col0 + j) * kLatent + mb * 128 + row] = __uint_as_float(o[j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(bar[kBarOEmpty]);
      ++segs;
    }
    if (!more) break;
    slot = split::partial_slot(p, kModePaged, grp, sg.b, iq);
    if (tid < 32) sh.m[col0 + tid] = 0.f;
    named_bar_sync(bar_id, 128);  // this warpgroup's heads have their factors, and m = 0
    float l_part[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) l_part[j] = 0.f;
    bool first = true;
    for (int n = sg.first(); n < sg.hi; n = sg.next(n), ++tiles) {
      const uint32_t pb = tiles & 1;
      const int j0 = sg.q.seq.tile(n) * kTile;
      wait(bar, kBarSFull, tiles & 1);
      __syncwarp();
      tc_fence_after();
      float x[32];  // score - m, in log2 units
      {
        uint32_t s[32];
        tmem_ld32(t_lane + kTmemS + col0, s);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive(bar[kBarSEmpty]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 c4 = cs4[j], mm = m4[j];
          fma_f32x2(x[4 * j], x[4 * j + 1], __uint_as_float(s[4 * j]), __uint_as_float(s[4 * j + 1]), c4.x, c4.y, mm.x,
                    mm.y);
          fma_f32x2(x[4 * j + 2], x[4 * j + 3], __uint_as_float(s[4 * j + 2]), __uint_as_float(s[4 * j + 3]), c4.z,
                    c4.w, mm.z, mm.w);
        }
      }
      if (!sg.q.every_row(j0, kTile)) {
        const bool vis = sg.q.row(j0 + row);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = vis ? x[j] : -INFINITY;
      }
      float top = fmaxf(x[0], x[1]);
#pragma unroll
      for (int j = 2; j < 32; j += 2) top = fmaxf(fmaxf(top, x[j]), x[j + 1]);  // three-operand maxima
      const bool raise = named_bar_or(bar_id, 128, first || top > kTau + kShift);
      if (raise) {
        int mine = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int i = __float_as_int(fmaxf(x[j], -INFINITY));  // a NaN does not count
          const int best = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7FFFFFFF));  // ordered as the floats
          if (lane == j) mine = best ^ ((best >> 31) & 0x7FFFFFFF);
        }
        sh.red[wq * kHeads + col0 + lane] = __int_as_float(mine);
        named_bar_sync(bar_id, 128);
        if (tid < 32) {
          const int h = col0 + tid;
          const float mt =
              fmaxf(fmaxf(sh.red[h], sh.red[kHeads + h]), fmaxf(sh.red[2 * kHeads + h], sh.red[3 * kHeads + h]));
          float d = mt - kShift;  // how far m rises (the first tile sets it)
          if (mt == -INFINITY || (!first && d < 0.f)) d = 0.f;
          sh.rise[h] = d;
          sh.alpha[h] = exp2_approx(-d);
          sh.m[h] -= d;
        }
        named_bar_sync(bar_id, 128);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          x[j] -= sh.rise[col0 + j];
          if (!first) l_part[j] *= sh.alpha[col0 + j];
        }
      }
      uint32_t pw[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float p0 = exp2_approx(x[2 * j]), p1 = exp2_approx(x[2 * j + 1]);
        add_f32x2(l_part[2 * j], l_part[2 * j + 1], p0, p1);
        pw[j] = pack_f16x2(p0, p1);
      }
      // this P buffer is free (the value MMAs of two tiles ago are done)
      wait(bar, kBarPEmpty + pb, ((tiles >> 1) & 1) ^ 1);
      if (raise && !first) {
        // the running max moved: once the last tile's value MMAs are done, rescale O^T
        wait(bar, kBarPEmpty + (pb ^ 1), ((tiles - 1) >> 1) & 1);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {
          uint32_t o[32];
          const uint32_t addr = t_lane + kTmemO + mb * kHeads + col0;
          tmem_ld32(addr, o);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sh.alpha[col0 + j]);
          tmem_st32(addr, o);
        }
        tmem_st_wait();
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        st_shared_v4(p_dst + pb * kPBytes + (((4 * wg + u) ^ (krow & 7)) << 4), pw[4 * u], pw[4 * u + 1], pw[4 * u + 2],
                     pw[4 * u + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(bar[kBarPFull + pb]);
      first = false;
    }
    // ---- m and l of the partial; O^T follows
    sh.red[wq * kHeads + col0 + lane] = sum_columns(l_part, lane);
    named_bar_sync(bar_id, 128);  // and every warp of the group is done with the factors
    if (tid < 32) {
      const int h = col0 + tid;
      p.part_m[slot * kHeads + h] = -sh.m[h];
      p.part_l[slot * kHeads + h] = sh.red[h] + sh.red[kHeads + h] + sh.red[2 * kHeads + h] + sh.red[3 * kHeads + h];
    }
  }
}

// ------------------------------------------------------------------ kernel
__global__ void __launch_bounds__(kThreads, 1)
    attend_packed_kernel(const __grid_constant__ CUtensorMap tm_codes, const __grid_constant__ CUtensorMap tm_scales,
                         const AttendPackedParams p) {
  extern __shared__ uint8_t smem_raw[];
  Shared sh;
  sh.base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  sh.bar = reinterpret_cast<uint64_t *>(sh.base + kOffBar);
  sh.red = reinterpret_cast<float *>(sh.base + kOffRed);
  sh.m = reinterpret_cast<float *>(sh.base + kOffM);
  sh.alpha = reinterpret_cast<float *>(sh.base + kOffAlpha);
  sh.rise = reinterpret_cast<float *>(sh.base + kOffRise);
  sh.cs = reinterpret_cast<float *>(sh.base + kOffCs);
  Range *range = reinterpret_cast<Range *>(sh.base + kOffRange);
  sh.range = range;
  sh.tmem_slot = reinterpret_cast<uint32_t *>(sh.base + kOffMisc);
  sh.abort_flag = reinterpret_cast<volatile int *>(sh.base + kOffMisc + 4);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = blockIdx.x / p.group_size, iq = blockIdx.x % p.group_size;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRawSlots; ++i) {
      mbar_init(&sh.bar[kBarRawFull + i], 1);
      mbar_init(&sh.bar[kBarRawEmpty + i], 8);
    }
    for (int i = 0; i < kStage; ++i) {
      mbar_init(&sh.bar[kBarSAFull + i], 4);
      mbar_init(&sh.bar[kBarSAEmpty + i], 1);
      mbar_init(&sh.bar[kBarVAFull + i], 4);
      mbar_init(&sh.bar[kBarVAEmpty + i], 1);
    }
    mbar_init(&sh.bar[kBarQFull], kSoftmaxWarps);
    mbar_init(&sh.bar[kBarSFull], 1);
    mbar_init(&sh.bar[kBarSEmpty], kSoftmaxWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.bar[kBarPFull + i], kSoftmaxWarps);
      mbar_init(&sh.bar[kBarPEmpty + i], 1);
    }
    mbar_init(&sh.bar[kBarOFull], 1);
    mbar_init(&sh.bar[kBarOEmpty], kSoftmaxWarps);
    mbar_init(&sh.bar[kBarDrain], 2);
    *sh.abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_codes);
    prefetch_tensormap(&tm_scales);
  }
  if (warp == 1) {
    tmem_alloc(sh.tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  grid_dep_launch();
  grid_dep_wait();  // everything below may come from the previous kernel
  if (warp == 0) {
    // This warp initialised the barriers and finds the range: it starts loading at once.  Not on
    // barrier 0: with nothing to load it may be at the block's last barrier before the others
    // are at this one.
    const Range r = lists::find_range<Seqs>(p, g, lane);
    if (lane == 0) *range = r;
    __syncwarp();
    asm volatile("bar.arrive 4, %0;" ::"n"(kThreads) : "memory");
    producer_role(p, sh, &tm_codes, &tm_scales, iq, lane);
  } else {
    tc_fence_before();
    asm volatile("bar.sync 4, %0;" ::"n"(kThreads) : "memory");
    tc_fence_after();
  }
  const uint32_t tmem = *sh.tmem_slot;

  if (warp == 0) {
    // done above
  } else if (warp == 1) {
    score_mma_role(p, sh, tmem, iq);
  } else if (warp == 2) {
    value_mma_role(p, sh, tmem, iq);
  } else if (warp < 11) {
    softmax_role(p, sh, tmem, g, iq, warp, lane);
  } else if (warp < 15) {
    unpack_rows_role(p, sh, tmem, iq, warp & 3, lane);
  } else {
    if (blockIdx.x == 0 && warp == 15) lists::write_partial_table<Seqs>(p, lane);  // C^T is needed last: there is time
    unpack_latents_role(p, sh, tmem, iq, warp & 3, lane);
  }

  __syncwarp();
  // After an abort the MMAs already issued must finish before tensor memory is released.
  if (warp == 2 && *sh.abort_flag) {
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

}  // namespace packed

cudaError_t launch_attend_packed(const CUtensorMap &tm_codes, const CUtensorMap &tm_scales, const AttendPackedParams &p,
                                 cudaStream_t stream) {
  static std::atomic<int> configured_device{-1};
  if (cudaError_t e = set_smem_limit_once(packed::attend_packed_kernel, packed::kSmemBytes, configured_device);
      e != cudaSuccess)
    return e;
  if (cudaError_t e = launch_chained(packed::attend_packed_kernel, dim3(p.groups * p.group_size),
                                     dim3(packed::kThreads), packed::kSmemBytes, stream, tm_codes, tm_scales, p);
      e != cudaSuccess)
    return e;
  return lists::launch_combine<packed::Seqs, packed::PartialOrder>(p, p.unit, stream);
}

}  // namespace mla
