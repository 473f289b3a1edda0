// usp_window.cuh -- geometry shared by the sliding-window attention kernels.
//
// Visibility (positions are rows of a [B][S] sequence, optionally cut into
// packed documents): key j is seen by query i iff
//   lo_i <= j <= i   and   (i - j < W  or  j - lo_i < ns),
// lo_i the first row of i's document: a causal window of W keys that includes
// the query's own, and the document's first ns keys (sinks).
//
// A query tile of rows [q0, qe) therefore walks two runs of key tiles: the sink
// tiles of the document of row q0 (a document that starts inside the tile has
// its sinks inside the window run) and the window tiles up to the diagonal. A
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

// Key tiles of the query rows [q0, qe): n_s sink tiles from s0, then the window
// tiles from w0; nt in all.
struct KeyRun {
  int s0, n_s, w0, nt;
  __device__ __forceinline__ int tile(int it) const { return it < n_s ? s0 + it : w0 + it - n_s; }
};
__device__ __forceinline__ KeyRun key_run(const WinGeo& g, int q0, int qe) {
  const int lo = win_lo(g, q0);
  const int wlo = max(lo, q0 - g.W + 1);
  KeyRun r;
  r.w0 = wlo / kBN;
  r.s0 = lo / kBN;
  const int s_end = min(lo + g.ns, wlo);  // sinks below the window
  r.n_s = s_end > lo ? min((s_end - 1) / kBN + 1, r.w0) - r.s0 : 0;
  r.nt = r.n_s + (qe - 1) / kBN + 1 - r.w0;
  return r;
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
