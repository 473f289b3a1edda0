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
#include "usp_div.cuh"
#include "usp_internal.h"
#include "usp_ptx.cuh"

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
// below the window tiles, 32 at a time from the document's first key on (n_s tiles; a
// TMA box may start at any row), then the window tiles from w0; nt in all. A sink
// tile's products take 16 or 32 keys instead of 128.
constexpr int kSinkTile = 32;
struct KeyRun {
  int lo, w0, n_s, sinks, nt;
  __device__ __forceinline__ int base(int it) const { return it < n_s ? lo + it * kSinkTile : (w0 + it - n_s) * kBN; }
  // the keys that the products of tile it take: 16, 32 or 128
  __device__ __forceinline__ int width(int it) const {
    return it >= n_s ? kBN : sinks - it * kSinkTile > 16 ? 32 : 16;
  }
};
__device__ __forceinline__ KeyRun key_run(const WinGeo& g, int q0, int qe) {
  KeyRun r;
  r.lo = win_lo(g, q0);
  const int wlo = max(r.lo, q0 - g.W + 1);
  r.w0 = wlo / kBN;
  r.sinks = max(min(r.lo + g.ns, r.w0 * kBN) - r.lo, 0);  // below the window tiles
  r.n_s = (r.sinks + kSinkTile - 1) / kSinkTile;
  r.nt = r.n_s + (qe - 1) / kBN + 1 - r.w0;
  return r;
}

// An item's number, taken apart: which of n heads (or pairs of heads) it is, of which batch, and the rest.
struct ItemDiv {
  Div heads, batch;
};
inline ItemDiv make_item_div(int n, int B) { return ItemDiv{make_div(n), make_div(B)}; }
struct ItemParts {
  int head, b, rest;
};
__device__ __forceinline__ ItemParts item_parts(const ItemDiv& d, int idx) {
  const uint32_t x = quot(d.heads, idx), y = quot(d.batch, x);
  return ItemParts{static_cast<int>(idx - x * d.heads.d), static_cast<int>(x - y * d.batch.d), static_cast<int>(y)};
}

// Words of the workspace header behind the status word: the kernels' item counters.
enum : int { kCounterFwd = 16, kCounterDq = 32, kCounterDkdv = 48 };

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

// A position in a ring of kN stages: the stage, and the parity of its current use.
template <int kN>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == kN) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// ---------------------------------------------------------------- row stores
// A warp's 32 rows of 32 bf16 columns, row = lane, 64 bytes of it in pk: exchanged between
// neighbouring lanes so that lane 2a + k holds 32-byte piece k of rows 2a and 2a + 1, and a
// store instruction covers the whole 64-byte runs of sixteen rows. (One row per lane touches 32
// cache lines with 16 bytes each; an item's stores then cost the CTA 2 us. Pieces of 16 bytes
// among four lanes take twice the exchanges.) Rows below `rows` are stored at
// base + row * row_step; an output that is only 16-byte aligned takes two stores for one.
__device__ __forceinline__ void store_rows32(__nv_bfloat16* base, size_t row_step, int row0, int rows, int c0,
                                             uint32_t (&pk)[16]) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1;
#pragma unroll
  for (int e = 0; e < 8; ++e) {  // even lanes give their second piece for the neighbour's first
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? pk[e] : pk[8 + e], 1);
    if (odd)
      pk[e] = got;
    else
      pk[8 + e] = got;
  }
  const bool whole = (reinterpret_cast<uintptr_t>(base) & 31u) == 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = row0 + (lane & ~1) + j;
    if (r >= rows) break;
    __nv_bfloat16* const p = base + r * row_step + c0 + (lane & 1) * 16;
    const uint32_t* v = pk + 8 * j;
    if (whole) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                   "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                   : "memory");
    } else {
      reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}

// ---------------------------------------------------------------- work items
// Hands a persistent CTA its work items: the first is its block number, each next one
// the grid's counter says when the CTA is ready for it (items differ: documents,
// short walks at the start of a sequence). One warp asks ahead; the
// others take the number from a slot.
struct ItemFeed {
  uint64_t full[2], empty[2];
  int idx[2];
};
__device__ __forceinline__ void feed_init(ItemFeed& f, int takers) {  // takers: warps that call feed_take
  for (int s = 0; s < 2; ++s) {
    mbar_init(&f.full[s], 1);
    mbar_init(&f.empty[s], takers);
  }
}
// The CTA's k-th item (k >= 1), asked for and handed out by the giving warp.
__device__ __forceinline__ bool feed_give(ItemFeed& f, int k, int* counter, const WaitCtl& w, int site, int& idx) {
  int x = 0;
  if ((threadIdx.x & 31) == 0) x = static_cast<int>(gridDim.x) + atomicAdd(counter, 1);
  idx = __shfl_sync(0xffffffffu, x, 0);
  const int s = k & 1;
  if (k > 2 && !mbar_wait_w(&f.empty[s], ((k - 1) / 2 - 1) & 1, w, site)) return false;
  if ((threadIdx.x & 31) == 0) f.idx[s] = idx;
  __syncwarp();
  mbar_arrive_w(&f.full[s]);
  return true;
}
__device__ __forceinline__ bool feed_take(ItemFeed& f, int k, const WaitCtl& w, int site, int& idx) {
  const int s = k & 1;
  if (!mbar_wait_w(&f.full[s], ((k - 1) / 2) & 1, w, site)) return false;
  idx = *reinterpret_cast<volatile int*>(&f.idx[s]);
  mbar_arrive_warp(&f.empty[s]);
  return true;
}

// Programmatic launches: a kernel lets the next one of its stream start once all its
// CTAs run, and waits for the one before it to end before it touches memory.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
  if (e == cudaSuccess) note_launch();
  return e == cudaSuccess ? cudaGetLastError() : e;
}

// Sets the elements of r whose bit of vis is clear (32 columns of one row per lane), most often for
// all of a warp's rows alike: a group of columns that every row sees costs a vote.
__device__ __forceinline__ void hide_columns(uint32_t (&r)[32], uint32_t vis, uint32_t value) {
  if (__all_sync(0xffffffffu, vis == 0xFFFFFFFFu)) return;
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!((vis >> c) & 1u)) r[c] = value;
}
constexpr uint32_t kMinusInf = 0xFF800000u;

}  // namespace usp
