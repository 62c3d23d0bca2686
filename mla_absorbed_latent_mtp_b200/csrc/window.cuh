// window.cuh -- which tiles and rows of a cache a query sees under the causal mask, a sliding
// window and sinks: query i of a sequence of L rows and Q queries sits at t = L - Q + i and
// sees the rows j <= t with t - j < window or j < sinks (window 0: every j <= t).
//
// A sequence's tile list holds the tiles that any of its Q queries may see: the tiles of the
// sinks, then those from the first query's window start to the end.  With the tiles of the
// list numbered n = 0, 1, ..., a query sees the n of two runs, [0, a) and [b, e).
#pragma once

#include <cuda_runtime.h>

namespace mla {
namespace window {

// A sequence's tile list: tile(n) = n below ns, then w0 + n - ns; `count` tiles.
template <int kRows>
struct SeqTiles {
  int ns, w0, count;
  __device__ __forceinline__ SeqTiles() : ns(0), w0(0), count(0) {}
  __device__ __forceinline__ SeqTiles(int L, int Q, int window, int sinks) {
    const int nt = (L + kRows - 1) / kRows;
    ns = w0 = 0;
    if (window > 0) {
      const long long lo = (long long)L - Q - window + 1;  // the first query's window start
      w0 = lo > 0 ? (int)(lo / kRows) : 0;
      ns = min((min(sinks, L) + kRows - 1) / kRows, w0);
    }
    count = ns + nt - w0;
  }
  __device__ __forceinline__ int tile(int n) const { return n < ns ? n : w0 + n - ns; }
};

// What query i sees of it.
template <int kRows>
struct QueryTiles {
  SeqTiles<kRows> seq;
  int n_vis, lo, sinks;  // rows j < n_vis with j >= lo or j < sinks
  int a, b, e;           // list tiles [0, a) and [b, e)
  __device__ __forceinline__ QueryTiles() : n_vis(0), lo(0), sinks(0), a(0), b(0), e(0) {}
  __device__ __forceinline__ QueryTiles(int L, int Q, int i, int window, int sinks_) : seq(L, Q, window, sinks_) {
    const long long t = (long long)L - Q + i;
    n_vis = t >= 0 ? (int)t + 1 : 0;
    sinks = window > 0 ? sinks_ : 0;
    const long long l = t - window + 1;
    lo = (window > 0 && l > 0) ? (int)l : 0;
    // A sink tile's list number is its own number: either the list is contiguous there, or
    // the sinks' tiles all lie below ns.
    a = (min(sinks, n_vis) + kRows - 1) / kRows;
    b = max(a, lo / kRows - seq.w0 + seq.ns);
    e = n_vis > 0 ? max(b, (n_vis + kRows - 1) / kRows - seq.w0 + seq.ns) : 0;
    if (n_vis <= 0) a = b = 0;
  }
  // The first seen list tile at or after n (e when there is none).
  __device__ __forceinline__ int seek(int n) const { return n < a ? n : max(n, b); }
  __device__ __forceinline__ bool row(int j) const { return j < n_vis && (j >= lo || j < sinks); }
  // Any / every row of [j0, j0 + n).
  __device__ __forceinline__ bool any_row(int j0, int n) const {
    return j0 < n_vis && (j0 + n > lo || j0 < sinks);
  }
  __device__ __forceinline__ bool every_row(int j0, int n) const {
    return j0 + n <= n_vis && (j0 >= lo || j0 + n <= sinks);
  }
};

}  // namespace window
}  // namespace mla
