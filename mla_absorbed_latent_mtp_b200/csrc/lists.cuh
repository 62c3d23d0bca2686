// lists.cuh -- the tile list of a windowed or packed attention: which range of it a CTA group takes,
// where the partials are, and the kernels that merge them.
//
// The list holds, sequence after sequence, the tiles that its queries may see (window.cuh), and G
// groups take equal ranges of it.  `Seqs` gives a kernel's lengths and tile counts:
//   length(p, b)      rows of sequence b, clamped to the cache;  bad_length(p, b): it was clamped
//   tiles(p, L)       list tiles of a sequence of L rows
#pragma once

#include <math.h>

#include <algorithm>

#include "internal.h"
#include "sm100.cuh"
#include "split.cuh"

namespace mla {
namespace lists {

// A CTA group's range of the list, and the sequence that holds its first tile.
struct Range {
  long long t0, t1, base;  // base: first tile of sequence s
  int s, L, start;         // its length, and the list's start places per sequence
};

// Places of a sequence in the list: its tiles, and before them `start` places without work, which
// stand for what a CTA pays when it begins another sequence (an empty pipeline, q~, the last
// one's partial), so that ranges of equal length are equal in time: Seqs::kStart, fewer where a
// CTA has hardly any tiles, and none where it has at most one.  (4-bit rows, tiles of 128, kStart 3:
// 32 x 8,192 rows 75.2 us without, 67.9 with; 32 x 1,024: 35.9 without, 25.6 with one place, 28.9
// with three; 32 x 512: 22.9 without, 25.7 with three.  bf16 windows, tiles of 64: 32 x (4,096 + 64)
// 43.5 us without, 41.7 / 42.7 / 42.8 with 3 / 5 / 8; 16 x 6 queries, window 4,095: 93.9, 89.5 / 88.9 / 92.5.)
template <class Seqs>
__device__ __forceinline__ int start_places(long long tiles, int seqs, int G) {
  return tiles <= G ? 0 : (tiles >= 2LL * G && tiles >= 8LL * seqs) ? Seqs::kStart : 1;
}
template <class Seqs, class P>
__device__ __forceinline__ int places(const P &p, int L, int start) {
  const int n = Seqs::tiles(p, L);
  return n > 0 ? n + start : 0;
}

__device__ __forceinline__ int warp_scan(int x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The list's length and its start places, by one warp.
template <class Seqs, class P>
__device__ long long list_length(const P &p, int lane, int &start) {
  long long tiles = 0;
  int seqs = 0;
  for (int s0 = 0; s0 < p.B; s0 += 32) {
    const int n = s0 + lane < p.B ? Seqs::tiles(p, Seqs::length(p, s0 + lane)) : 0;
    tiles += __reduce_add_sync(0xffffffffu, n);
    seqs += __popc(__ballot_sync(0xffffffffu, n > 0));
  }
  start = start_places<Seqs>(tiles, seqs, p.groups);
  return tiles + (long long)start * seqs;
}

// floor(g T / G), in 32 bits where the list allows it.
__device__ __forceinline__ long long group_start(int g, long long T, int G) {
  if (T >= (1LL << 31)) return split::group_start(g, T, G);
  const uint32_t q = (uint32_t)T / (uint32_t)G, r = (uint32_t)T % (uint32_t)G;
  return (long long)g * q + (uint32_t)g * r / (uint32_t)G;  // G is at most the number of SMs
}

// By one warp, with scans in steps of 32 sequences (a walk from the first sequence cost the last
// CTAs of a 32-sequence step a microsecond).
template <class Seqs, class P>
__device__ Range find_range(const P &p, int g, int lane) {
  Range r = {0, 0, 0, 0, 0, 0};
  const long long T = list_length<Seqs>(p, lane, r.start);
  r.t0 = group_start(g, T, p.groups);
  r.t1 = group_start(g + 1, T, p.groups);
  if (r.t0 >= r.t1) return r;
  for (int s0 = 0; s0 < p.B; s0 += 32) {
    const int L = s0 + lane < p.B ? Seqs::length(p, s0 + lane) : 0;
    const int n = s0 + lane < p.B ? places<Seqs>(p, L, r.start) : 0;
    const int x = warp_scan(n, lane);
    const uint32_t behind = __ballot_sync(0xffffffffu, r.base + x > r.t0);  // the range starts before their end
    if (behind) {
      const int l = __ffs(behind) - 1;
      r.s = s0 + l;
      r.L = __shfl_sync(0xffffffffu, L, l);
      r.base += __shfl_sync(0xffffffffu, x - n, l);
      break;
    }
    r.base += __shfl_sync(0xffffffffu, x, 31);
  }
  return r;
}

// Where each sequence's partials are, for the combine: with at least as many places as groups they
// are those of `count` consecutive groups, seq_ts = count << 32 | first group; with fewer every
// place is a group of its own, seq_ts = -1 - first place, seq_nt places of T (written as the last
// sequence's end).
template <class Seqs, class P>
__device__ void write_partial_table(const P &p, int lane) {
  int start;
  const long long T = list_length<Seqs>(p, lane, start);
  const long long G = p.groups;
  long long base = 0;
  for (int s0 = 0; s0 < p.B; s0 += 32) {
    const int s = s0 + lane;
    const int n = s < p.B ? places<Seqs>(p, Seqs::length(p, s), start) : 0;
    const int x = warp_scan(n, lane);
    if (s < p.B) {
      const long long ts = base + x - n;
      p.seq_nt[s] = n;
      if (T < G) {
        p.seq_ts[s] = -1 - ts;
      } else if (n == 0) {
        p.seq_ts[s] = 0;
      } else {
        const long long first = split::group_of(ts, T, G), last = split::group_of(ts + n - 1, T, G);
        p.seq_ts[s] = (last - first + 1) << 32 | first;
      }
    }
    base += __shfl_sync(0xffffffffu, x, 31);
  }
}

// ------------------------------------------------------------------ combine
// Merges the partials of a query row: with M the largest running max and w_k = 2^(m_k - M),
// o = unit * sum w_k O_k / sum w_k l_k and lse = (M + log2 sum w_k l_k) ln 2.  Thread t of 128 loads
// values 4t .. 4t + 3 of a partial, in the order that the attend kernel found convenient; the row
// goes through shared memory to its latents' places, Order::latent.
//
// Only an empty partial (m = -inf, O never written) is left out.  One whose weight is zero in fp32
// still counts: a NaN or an Inf in its sums reaches the result, as 0 x NaN does in the formula.
constexpr float kEmpty = -1.f;  // in place of the weight of an empty partial

// The places of sequence b's partials, from write_partial_table.
struct Partials {
  int count, first, ts, T;
  template <class P>
  __device__ __forceinline__ Partials(const P &p, int b) : first(0), ts(-1), T(0) {
    const long long place = p.seq_ts[b];
    if (place < 0) {  // fewer places than groups
      count = p.seq_nt[b];
      ts = (int)(-1 - place);
      T = (int)(-1 - p.seq_ts[p.B - 1]) + p.seq_nt[p.B - 1];
    } else {
      count = (int)(place >> 32);
      first = (int)place;
    }
  }
  template <class P>
  __device__ __forceinline__ long long slot(const P &p, int k, int b, int i) const {
    const int g = ts >= 0 ? ((ts + k + 1) * p.groups - 1) / T : first + k;
    return split::partial_slot(p, kModePaged, g, b, i);
  }
};

template <class Seqs, class P>
__device__ __forceinline__ void report_length(const P &p, int b) {
  if (Seqs::bad_length(p, b)) report_status(p.status, kStatusIndex);
}

template <class Order>
__device__ __forceinline__ void row_to_shared(uint16_t *row, const float4 &o, float inv, int at) {
  const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
  for (int e = 0; e < 4; ++e) row[Order::latent(at + e)] = (uint16_t)(pack_bf16x2(v[e], 0.f) & 0xFFFFu);
}
template <class P>
__device__ __forceinline__ void write_row(const P &p, long long at, const uint16_t *row, float M,
                                          float den, int t) {
  reinterpret_cast<uint2 *>(p.o_latent + at * kLatent)[t] = reinterpret_cast<const uint2 *>(row)[t];
  if (p.lse != nullptr && t == 0)
    p.lse[at] = M == -INFINITY ? -INFINITY : (M + log2f(den)) * 0.69314718055994530942f;
}

// Many query rows, few partials each: a block takes some heads of a row and merges online, some
// partials at a time, all their loads in flight at once: two heads and three partials, or, with at
// least as many sequences as groups (where most rows have one or two partials, and blocks come in
// waves), four heads and one (4-bit rows, 148 x 100: the call 30.5 us with two heads, 28.9 with
// four, 33.8 with eight; but 32 x 1,024: 25.6 with two, 28.9 with four).
template <int kH, int kChunk, class Seqs, class Order, class P>
__global__ void __launch_bounds__(128, 8) combine_few_kernel(const P p, float unit) {
  grid_dep_launch();
  grid_dep_wait();
  const int v = blockIdx.x, b = v / p.Q, i = v % p.Q, t = threadIdx.x;
  const int h0 = blockIdx.y * kH;
  __shared__ __align__(16) uint16_t row[kH][kLatent];
  const Partials pt(p, b);
  if (t == 0 && blockIdx.y == 0 && i == 0) report_length<Seqs>(p, b);
  float M[kH], den[kH];
  float4 acc[kH];
#pragma unroll
  for (int hh = 0; hh < kH; ++hh) {
    M[hh] = -INFINITY;
    den[hh] = 0.f;
    acc[hh] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int k0 = 0; k0 < pt.count; k0 += kChunk) {
    float mk[kH][kChunk], lk[kH][kChunk];
    float4 ok[kH][kChunk];
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      const bool live = k0 + j < pt.count;
      const long long slot = live ? pt.slot(p, k0 + j, b, i) : 0;
#pragma unroll
      for (int hh = 0; hh < kH; ++hh) {
        const long long r = slot * kHeads + h0 + hh;
        mk[hh][j] = live ? p.part_m[r] : -INFINITY;
        lk[hh][j] = live ? p.part_l[r] : 0.f;
        ok[hh][j] = live ? *reinterpret_cast<const float4 *>(p.part_o + r * kLatent + 4 * t)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
#pragma unroll
    for (int hh = 0; hh < kH; ++hh) {
      float mx = M[hh];
#pragma unroll
      for (int j = 0; j < kChunk; ++j) mx = fmaxf(mx, mk[hh][j]);
      if (mx == -INFINITY) continue;
      const float a = exp2f(M[hh] - mx);  // 0 when M was -inf
      den[hh] *= a;
      acc[hh].x *= a;
      acc[hh].y *= a;
      acc[hh].z *= a;
      acc[hh].w *= a;
#pragma unroll
      for (int j = 0; j < kChunk; ++j) {
        if (mk[hh][j] == -INFINITY) continue;  // empty
        const float w = exp2f(mk[hh][j] - mx);
        den[hh] += w * lk[hh][j];
        acc[hh].x += w * ok[hh][j].x;
        acc[hh].y += w * ok[hh][j].y;
        acc[hh].z += w * ok[hh][j].z;
        acc[hh].w += w * ok[hh][j].w;
      }
      M[hh] = mx;
    }
  }
#pragma unroll
  for (int hh = 0; hh < kH; ++hh)
    row_to_shared<Order>(row[hh], acc[hh], M[hh] == -INFINITY ? 0.f : unit / den[hh], 4 * t);
  __syncthreads();
#pragma unroll
  for (int hh = 0; hh < kH; ++hh) write_row(p, (long long)v * kHeads + h0 + hh, row[hh], M[hh], den[hh], t);
}

// Few sequences, many partials each: a block takes one head of a row; eight slices of 128 threads
// take every eighth partial, all of a thread's loads independent, and are added up in order (1 x
// 8,192 rows, 64 partials: the call 66.6 us with the kernel above, 23.9 with this one; 4 x 8,192
// rows: 48.3 and 26.1).
constexpr int kSlices = 8;
constexpr int kMaxPartials = 256;  // per sequence: at most one per CTA group
template <class Seqs, class Order, class P>
__global__ void __launch_bounds__(128 * kSlices) combine_many_kernel(const P p, float unit) {
  grid_dep_launch();
  grid_dep_wait();
  const int v = blockIdx.x, b = v / p.Q, i = v % p.Q, h = blockIdx.y;
  const int t = threadIdx.x % 128, slice = threadIdx.x / 128, lane = threadIdx.x % 32;
  __shared__ long long slots[kMaxPartials];
  __shared__ float weight[kMaxPartials];
  __shared__ float4 sum[kSlices][128];
  __shared__ __align__(16) uint16_t row[kLatent];
  __shared__ float total, top;
  const Partials pt(p, b);
  if (threadIdx.x == 0 && h == 0 && i == 0) report_length<Seqs>(p, b);
  if (threadIdx.x < 32) {
    float M = -INFINITY, den = 0.f;
    for (int k = lane; k < pt.count; k += 32) {
      slots[k] = pt.slot(p, k, b, i);
      weight[k] = p.part_m[slots[k] * kHeads + h];
      M = fmaxf(M, weight[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int k = lane; k < pt.count; k += 32) {
      const float w = weight[k] == -INFINITY ? kEmpty : exp2f(weight[k] - M);
      weight[k] = w;
      if (w != kEmpty) den += w * p.part_l[slots[k] * kHeads + h];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane == 0) {
      total = den;
      top = M;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = slice; k < pt.count; k += kSlices) {
    const float w = weight[k];
    const float *at = p.part_o + (slots[k] * kHeads + h) * kLatent + 4 * t;
    const float4 o = w != kEmpty ? *reinterpret_cast<const float4 *>(at) : make_float4(0.f, 0.f, 0.f, 0.f);
    acc.x += w * o.x;
    acc.y += w * o.y;
    acc.z += w * o.z;
    acc.w += w * o.w;
  }
  sum[slice][t] = acc;
  __syncthreads();
  if (slice == 0) {
    for (int s = 1; s < kSlices; ++s) {
      const float4 o = sum[s][t];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
    }
    row_to_shared<Order>(row, acc, top == -INFINITY ? 0.f : unit / total, 4 * t);
  }
  __syncthreads();
  if (slice == 0) write_row(p, (long long)v * kHeads + h, row, top, total, t);
}

// A single query row: its 64 heads alone are too few blocks to read the partials at speed, so four
// blocks take a quarter of a head's latents each, a warp per slice; the weights' loads are in flight
// at once, and the first partials' before the weights are known.  (1 x 18,944 rows, 148 partials:
// the call 28.9 us with the kernel above, 22.9 with this one; with two rows that one is as fast,
// and with four this one's registers cost more than its blocks give: 26.0 us against 30.0.)
constexpr int kRowParts = 4, kRowThreads = 512;
template <class Seqs, class Order, class P>
__global__ void __launch_bounds__(kRowThreads) combine_row_kernel(const P p, float unit) {
  constexpr int kLanes = 128 / kRowParts, kSlices = kRowThreads / kLanes, kAhead = 4;
  grid_dep_launch();
  grid_dep_wait();
  const int b = 0, i = 0, h = blockIdx.x, part = blockIdx.y;
  const int t = threadIdx.x % kLanes, slice = threadIdx.x / kLanes, lane = threadIdx.x % 32;
  __shared__ float weight[kMaxPartials];
  __shared__ float4 sum[kSlices][kLanes];
  __shared__ __align__(16) uint16_t row[kLatent];
  __shared__ float total, top;
  const Partials pt(p, b);
  const int at = Order::unit(part, t);  // the first of this thread's four stored values
  float4 first[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int k = slice + j * kSlices;
    first[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < pt.count)
      first[j] = *reinterpret_cast<const float4 *>(p.part_o + (pt.slot(p, k, b, i) * kHeads + h) * kLatent + at);
  }
  if (threadIdx.x == 0 && h == 0 && part == 0) report_length<Seqs>(p, b);
  if (threadIdx.x < 32) {
    float m[kMaxPartials / 32], l[kMaxPartials / 32], M = -INFINITY, den = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxPartials / 32; ++j) {
      const int k = lane + 32 * j;
      m[j] = -INFINITY;
      l[j] = 0.f;
      if (k < pt.count) {
        const long long r = pt.slot(p, k, b, i) * kHeads + h;
        m[j] = p.part_m[r];
        l[j] = p.part_l[r];
      }
      M = fmaxf(M, m[j]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int j = 0; j < kMaxPartials / 32; ++j) {
      const int k = lane + 32 * j;
      const float w = m[j] == -INFINITY ? kEmpty : exp2f(m[j] - M);
      if (k < pt.count) weight[k] = w;
      if (w != kEmpty) den += w * l[j];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    if (lane == 0) {
      total = den;
      top = M;
    }
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float w, const float4 &o) {
    if (w == kEmpty) return;
    acc.x += w * o.x;
    acc.y += w * o.y;
    acc.z += w * o.z;
    acc.w += w * o.w;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int k = slice + j * kSlices;
    if (k < pt.count) add(weight[k], first[j]);
  }
#pragma unroll 4
  for (int k = slice + kAhead * kSlices; k < pt.count; k += kSlices)
    add(weight[k], *reinterpret_cast<const float4 *>(p.part_o + (pt.slot(p, k, b, i) * kHeads + h) * kLatent + at));
  sum[slice][t] = acc;
  __syncthreads();
  if (slice == 0) {
    for (int s = 1; s < kSlices; ++s) {
      const float4 o = sum[s][t];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
    }
    row_to_shared<Order>(row, acc, top == -INFINITY ? 0.f : unit / total, at);
  }
  __syncthreads();
  if (slice == 0) write_row(p, h, row, top, total, part * kLanes + t);  // the part's latents are adjacent
}

template <class Seqs, class Order, class P>
cudaError_t launch_combine(const P &p, float unit, cudaStream_t stream) {
  const int rows = p.B * p.Q;
  if (rows == 1)
    return launch_chained(combine_row_kernel<Seqs, Order, P>, dim3(kHeads, kRowParts), dim3(kRowThreads), 0, stream, p,
                          unit);
  if (p.B <= p.groups / 16)  // sixteen partials a sequence or more
    return launch_chained(combine_many_kernel<Seqs, Order, P>, dim3(rows, kHeads), dim3(128 * kSlices), 0, stream, p,
                          unit);
  if (p.B >= p.groups)  // two partials a sequence or fewer, on average
    return launch_chained(combine_few_kernel<4, 1, Seqs, Order, P>, dim3(rows, kHeads / 4), dim3(128), 0, stream, p,
                          unit);
  return launch_chained(combine_few_kernel<2, 3, Seqs, Order, P>, dim3(rows, kHeads / 2), dim3(128), 0, stream, p,
                        unit);
}

}  // namespace lists
}  // namespace mla
