// usp_window.cuh -- geometry shared by the sliding-window attention kernels.
//
// Visibility (positions are rows of a [B][S] sequence, optionally cut into
// packed documents): key j is seen by query i iff
//   lo_i <= j <= i   and   (i - j < W  or  j - lo_i < ns),
// lo_i the first row of i's document: a causal window of W keys that includes
// the query's own, and the document's first ns keys (sinks).
//
// A query tile of rows [q0, qe) therefore walks the sinks of the document of row
// q0 (a document that starts inside the tile has its sinks inside the window
// tiles) and the window tiles up to the diagonal. A
// key tile walks one run of query tiles, from the diagonal to the last query in
// the band of its last key; the queries behind that run which still see its
// sinks are the far kernel's (usp_window_sink.cu). Every role of a CTA
// evaluates these closed forms itself; nothing is published between warps.
#pragma once

#include <climits>

#include "usp_attn_common.cuh"
#include "usp_internal.h"

namespace usp {

__device__ __forceinline__ void win_span(const WinGeo& g, int i, int& lo, int& hi) {
  lo = 0;
  hi = g.S;
  if (g.cu) {
    const int d = doc_of(g.cu, g.n_docs, i);
    lo = min(max(__ldg(g.cu + d), 0), i);  // unusable boundaries stay inside the sequence
    hi = min(max(__ldg(g.cu + d + 1), i + 1), g.S);
  }
}
__device__ __forceinline__ int win_lo(const WinGeo& g, int i) {
  int lo, hi;
  win_span(g, i, lo, hi);
  return lo;
}

// Key tiles of the query rows [q0, qe): the sinks of the first row's document
// below the window tiles, if any, as one tile of up to 128 keys from the
// document's first on (n_s = 1; a TMA box may start at any row), then the window
// tiles from w0; nt in all. Few sinks make a narrow tile: the products then take
// 16 or 32 keys instead of 128.
struct KeyRun {
  int lo, w0, n_s, cols, nt;  // cols: the sink tile's keys in use, rounded up to 16 (128 when more than 32)
  __device__ __forceinline__ bool sink(int it) const { return it < n_s; }
  __device__ __forceinline__ int base(int it) const { return it < n_s ? lo : (w0 + it - n_s) * kBN; }
  // the keys in use of tile it: a multiple of 16
  __device__ __forceinline__ int width(int it) const { return it < n_s ? cols : kBN; }
};
__device__ __forceinline__ KeyRun key_run(const WinGeo& g, int q0, int qe) {
  KeyRun r;
  r.lo = win_lo(g, q0);
  const int wlo = max(r.lo, q0 - g.W + 1);
  r.w0 = wlo / kBN;
  const int n = min(r.lo + g.ns, r.w0 * kBN) - r.lo;  // sinks below the window tiles (at most 128)
  r.n_s = n > 0 ? 1 : 0;
  r.cols = n > 32 ? kBN : (n + 15) & ~15;
  r.nt = r.n_s + (qe - 1) / kBN + 1 - r.w0;
  return r;
}

// Visible columns of a tile of KeyRun kr for one query row, 32 from c0 on: the
// row's window [first, i] and sinks [lo, sink_end) at tile `it`, whose keys start
// at k0 (a sink tile ends where the window tiles begin).
struct RowSpan {
  int lo, first, sink_end, end;  // end: i + 1
};
__device__ __forceinline__ RowSpan row_span(const WinGeo& g, int i) {
  RowSpan r{0, INT_MAX, 0, 0};  // a row past the end of the sequence sees nothing
  if (i < g.S) {
    r.lo = win_lo(g, i);
    r.first = max(r.lo, i - g.W + 1);
    r.sink_end = min(r.lo + g.ns, i + 1);
    r.end = i + 1;
  }
  return r;
}
__device__ __forceinline__ uint32_t bits_between(int a, int b, int c0);
__device__ __forceinline__ uint32_t visible_bits(const RowSpan& r, const KeyRun& kr, int it, int k0, int c0) {
  if (kr.sink(it)) return bits_between(r.lo - k0, min(r.sink_end, kr.w0 * kBN) - k0, c0);
  return bits_between(r.first - k0, r.end - k0, c0) | bits_between(r.lo - k0, r.sink_end - k0, c0);
}

// The last query tile in the band of key tile n (its first is n).
__device__ __forceinline__ int last_qtile(const WinGeo& g, int n) {
  const int jl = min(n * kBN + kBN, g.S) - 1;
  int lo, hi;
  win_span(g, jl, lo, hi);
  return (min(hi, jl + g.W) - 1) / kBM;  // W <= S, S < 2^30: no overflow
}

// Bits [a, b) of a 32-column group that starts at column c0 (any integers).
__device__ __forceinline__ uint32_t bits_between(int a, int b, int c0) {
  const int lo = min(max(a - c0, 0), 32), hi = min(max(b - c0, 0), 32);
  const uint32_t below_hi = hi >= 32 ? 0xFFFFFFFFu : ((1u << hi) - 1u);
  const uint32_t from_lo = lo >= 32 ? 0u : (0xFFFFFFFFu << lo);
  return below_hi & from_lo;
}

}  // namespace usp
