// usp_window_dq.cu -- backward of sliding-window attention with sinks, the
// query-major half (dQ) on sm_100a:
//   dQ_i = scale sum_j P_ij (dO_i.v_j - Delta_i) k_j
// over the key tiles that the forward walks (usp_window.cuh). dQ accumulates in
// TMEM over the walk and is written once, as bf16.
//
// A persistent CTA (one per SM, 320 threads) takes work items: one 128-row query
// tile of one head.
//   warp 0      TMA producer: Q, dO per item, K (3 stages) and V (2 stages) per key tile
//   warp 1      UMMA issuer: S = Q K^T (two buffers), dP = dO V^T, dQ += dS K
//   warps 2..9  two warpgroups of 64 key columns; thread = query row
// The gradient sums of a row cancel: sum_j dS_ij = 0 with the exact Delta_i =
// sum_j P_ij dP_ij, while dO.O of the bf16 output is off by up to 2^-8 |dO||O|. The
// kernel adds up the residue r_i = sum_j dS_ij in fp32 and writes Delta_i + r_i back
// to the table, for the key-major kernels that run after it. Its own sum is off by
// r_i sum_j P_ij k_j, which matters next to dQ's own rounding only where few keys
// share a row's weight (the ratio falls with the root of their number: 1.2 of the
// rounding at 4 keys, 0.4 at 64): query tiles with rows of fewer than 48 keys walk
// the tiles of those rows' keys twice. Where these are all tiles, the first walk only
// finds r and the second makes dQ with Delta + r (8192 tokens, 16 heads, window 8: 73 -> 71 us
// against two walks that both add); else the second adds dS = -r_i P_ij.
//
// TMEM: S / dS at 0 and 128, dP at 256, dQ at 384. The key tiles of all items of
// a CTA form one stream: S runs two tiles and dP one tile ahead, into the next
// item, whose first dQ product waits for dS, written by the warps that read this
// item's dQ before it.
//
// Bound by the compute warps' own work (about 1500 cycles per key tile, as much as the
// three products; the two overlap but for the handing over: 1.25 to 1.4 us) and by about
// 3.5 us per item (masked tiles, epilogue, the next item's rows). B=1 S=32768 H=16/4 D=128
// W=2048, 4 sinks: 761 us, 1052 TFLOP/s (6 D flops per visible pair).
#include <math.h>

#include "usp_ptx.cuh"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kThreads = 320;
constexpr int kComputeWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColDP = 256, kColDQ = 384;
__host__ __device__ constexpr uint32_t col_s(int b) { return 128u * b; }

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanelBytes = 128 * 128;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr int kKSt = 3;
  static constexpr int kVSt = 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffDO = kTileBytes;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kKSt * kTileBytes;
  static constexpr int kOffBar = kOffV + kVSt * kTileBytes;
  static constexpr int kOffRes = kOffBar + 320;  // residues: [item parity][warpgroup][row]
  static constexpr int kSmemBytes = kOffRes + 2 * 2 * 128 * 4;
};

struct Args {
  WinGeo g;
  ItemDiv div;
  const float* lse2;
  float* delta;
  int Lp;
  __nv_bfloat16* dq;
  int n_items;
  int* status;
  unsigned long long wait_ns;
};

struct Bars {
  uint64_t q_full, q_empty, do_full, do_empty;
  uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
  uint64_t s_full[2], dp_full, dp_free, dq_done[2], drain;
  // One per S buffer: dP of the next tile is issued ahead of the wait for dS, so the warps can
  // finish two tiles before the issuer looks for the first one's arrivals, whose phase a single
  // barrier would have left again by then. They cannot finish a third: its dP is issued behind.
  uint64_t ds_full[2];
  uint64_t r_full;  // both warpgroups' residues of the item are in sRes
  ItemFeed feed;
  uint32_t tmem_base;
  int abort_flag;
};

enum : int {
  kSiteQEmpty = 0x601, kSiteDoEmpty = 0x602, kSiteKEmpty = 0x603, kSiteVEmpty = 0x604, kSiteQ = 0x611, kSiteDo = 0x612,
  kSiteK = 0x613, kSiteV = 0x614, kSiteDpFree = 0x615, kSiteDs = 0x616, kSiteDqDone = 0x617, kSiteS = 0x621,
  kSiteDp = 0x622, kSiteEpi = 0x623, kSiteRes = 0x624, kSiteFeed = 0x631, kSiteAlign = 0x6FF
};

struct Item {
  int b, h, q0;
};
__device__ __forceinline__ Item item_of(const Args& a, int idx) {
  // as in the forward: the last rows of every head first, the heads side by side
  const ItemParts p = item_parts(a.div, idx);
  return Item{p.b, p.head, (a.g.n_tiles - 1 - p.rest) * kBM};
}
// The item's key tiles, n1 of them, and for its rows of few keys the last n2 again
// (such a row's keys end at the diagonal; nt in all).
constexpr int kFewKeys = 48;
struct DqRun {
  KeyRun kr;
  int n1, n2, nt;
  // the first pass adds to dQ (no second pass over all tiles follows)
  __device__ __forceinline__ bool adds(int it) const { return it >= n1 || n2 != n1; }
  __device__ __forceinline__ int pass_it(int it) const { return it < n1 ? it : it - n2; }
  __device__ __forceinline__ int base(int it) const { return kr.base(pass_it(it)); }
  __device__ __forceinline__ int width(int it) const { return kr.width(pass_it(it)); }
};
__device__ __forceinline__ DqRun run_of(const WinGeo& g, const Item& x) {
  DqRun r;
  const int qe = min(x.q0 + kBM, g.S);
  r.kr = key_run(g, x.q0, qe);
  r.n1 = r.kr.nt;
  if (g.W + g.ns < kFewKeys || x.q0 - r.kr.lo + 1 < kFewKeys)
    r.n2 = r.n1;  // every row, or a document that starts in or just before the tile: two or three tiles
  else
    r.n2 = win_lo(g, qe - 1) > x.q0 ? 1 : 0;  // documents that start inside: the diagonal tile
  r.nt = r.n1 + r.n2;
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kSiteAlign);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  static_assert(sizeof(Bars) <= 320, "barrier block");
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sDO = smem + C::kOffDO;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  float* sRes = reinterpret_cast<float*>(smem + C::kOffRes);
  const WinGeo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    feed_init(bars->feed, 1 + kComputeWarps);
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    mbar_init(&bars->do_full, 1);
    mbar_init(&bars->do_empty, 1);
    for (int s = 0; s < C::kKSt; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < C::kVSt; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->dq_done[s], 1);
      mbar_init(&bars->ds_full[s], kComputeWarps);
    }
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->dp_free, kComputeWarps);
    mbar_init(&bars->r_full, kComputeWarps);
    mbar_init(&bars->drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    // (not before: a CTA of the next kernel must not take the columns that this one waits for)
    let_next_start();
  }
  wait_for_previous();
  if (threadIdx.x == 0) bars->abort_flag = *reinterpret_cast<volatile int*>(a.status) != 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl w{&bars->abort_flag, a.status, a.wait_ns};
  const bool skip = bars->abort_flag != 0;

  if (skip) {
    // nothing issued, nothing to drain
  } else if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
      tma_prefetch_desc(&tm_do);
    }
    __syncwarp();
    int nk = 0, nv = 0, n_q = 0, n_do = 0;
    bool ok = true;
    auto panels = [&](const CUtensorMap* tm, uint64_t* bar, uint8_t* dst, int head, int row, int b) {
      mbar_expect_tx_w(bar, C::kTileBytes);
      for (int p = 0; p < C::kPanels; ++p) tma_load_4d_w(tm, bar, dst + p * C::kPanelBytes, p * 64, head, row, b);
    };
    int idx = blockIdx.x, next = 0;
    for (int k = 1; ok && idx < a.n_items; ++k, idx = next) {
      const Item x = item_of(a, idx);
      const DqRun kr = run_of(g, x);
      const int kvh = x.h / g.G;
      for (int it = 0; it < kr.nt; ++it) {
        const int sk = nk % C::kKSt, sv = nv % C::kVSt;
        if (nk >= C::kKSt && !mbar_wait_w(&bars->k_empty[sk], ((nk / C::kKSt) - 1) & 1, w, kSiteKEmpty)) { ok = false; break; }
        panels(&tm_k, &bars->k_full[sk], sK + sk * C::kTileBytes, kvh, kr.base(it), x.b);
        ++nk;
        if (it == 0) {  // Q behind the first K, dO behind it: in the order in which their buffers free
          if (n_q >= 1 && !mbar_wait_w(&bars->q_empty, (n_q - 1) & 1, w, kSiteQEmpty)) { ok = false; break; }
          panels(&tm_q, &bars->q_full, sQ, x.h, x.q0, x.b);
          ++n_q;
          if (n_do >= 1 && !mbar_wait_w(&bars->do_empty, (n_do - 1) & 1, w, kSiteDoEmpty)) { ok = false; break; }
          panels(&tm_do, &bars->do_full, sDO, x.h, x.q0, x.b);
          ++n_do;
          if (!feed_give(bars->feed, k, a.status + kCounterDq, w, kSiteFeed, next)) { ok = false; break; }
        }
        if (nv >= C::kVSt && !mbar_wait_w(&bars->v_empty[sv], ((nv / C::kVSt) - 1) & 1, w, kSiteVEmpty)) { ok = false; break; }
        panels(&tm_v, &bars->v_full[sv], sV + sv * C::kTileBytes, kvh, kr.base(it), x.b);
        ++nv;
      }
    }
    // Every copy this warp started lands before the CTA ends, whoever may have given up since.
    if (n_q > 0) mbar_wait_drain(&bars->q_full, (n_q - 1) & 1);
    if (n_do > 0) mbar_wait_drain(&bars->do_full, (n_do - 1) & 1);
    for (int it = nk - C::kKSt < 0 ? 0 : nk - C::kKSt; it < nk; ++it)
      mbar_wait_drain(&bars->k_full[it % C::kKSt], (it / C::kKSt) & 1);
    for (int it = nv - C::kVSt < 0 ? 0 : nv - C::kVSt; it < nv; ++it)
      mbar_wait_drain(&bars->v_full[it % C::kVSt], (it / C::kVSt) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    constexpr uint32_t kIdKM = idesc_bf16_f32(128, D, 0, 1);
    const uint64_t dQ0 = sdesc_sw128(smem_addr(sQ), 16, 1024), dDO0 = sdesc_sw128(smem_addr(sDO), 16, 1024);
    const uint64_t dK0 = sdesc_sw128(smem_addr(sK), 16, 1024), dV0 = sdesc_sw128(smem_addr(sV), 16, 1024);
    const uint64_t dKmn = sdesc_sw128(smem_addr(sK), C::kPanelBytes, 1024);
    bool issued_any = false;
    // The loop below is one warp's chain of dependent steps between the products, so it
    // keeps its state in a few counters: ring positions of the K stage that S takes next
    // and that dQ takes next, of the V stage that dP takes next, and the S buffers' turns.
    Ring<C::kKSt> k_s, k_q;
    Ring<C::kVSt> v_d;
    uint32_t s_turn = 0, q_turn = 0;  // tiles whose S, dQ have been issued
    uint32_t item = 0;
    // X = A B^T of 128 rows and the first `keys` rows of B (128; 16 or 32 in a narrow tile)
    auto xt = [&](uint32_t acc, uint64_t a0, uint64_t b0, int keys) {
      auto go = [&](uint32_t idesc) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kPanelBytes + (kk & 3) * 32) >> 4;
          umma_bf16_w(acc, a0 + off, b0 + off, idesc, kk > 0 ? 1u : 0u);
        }
      };
      if (keys == kBN)
        go(idesc_bf16_f32(128, 128, 0, 0));
      else
        go(idesc_bf16_f32(128, keys, 0, 0));
    };
    auto issue_s = [&](int keys) -> bool {  // S into the buffer whose turn it is
      if (!mbar_wait_w(&bars->k_full[k_s.at], k_s.phase, w, kSiteK)) return false;
      // dQ two tiles back has read its dS from the buffer
      if (s_turn >= 2 && !mbar_wait_w(&bars->dq_done[s_turn & 1], ((s_turn - 2) >> 1) & 1, w, kSiteDqDone)) return false;
      tc_fence_after();
      xt(tmem + col_s(s_turn & 1), dQ0, dK0 + ((k_s.at * C::kTileBytes) >> 4), keys);
      umma_commit_w(&bars->s_full[s_turn & 1]);
      ++s_turn;
      k_s.next();
      issued_any = true;
      return true;
    };
    uint32_t d_turn = 0;  // tiles whose dP has been issued
    auto issue_dp = [&](int keys) -> bool {  // dP = dO V^T, once the previous dP has been read
      if (!mbar_wait_w(&bars->v_full[v_d.at], v_d.phase, w, kSiteV)) return false;
      if (d_turn >= 1 && !mbar_wait_w(&bars->dp_free, (d_turn - 1) & 1, w, kSiteDpFree)) return false;
      tc_fence_after();
      xt(tmem + kColDP, dDO0, dV0 + ((v_d.at * C::kTileBytes) >> 4), keys);
      umma_commit_w(&bars->dp_full);
      umma_commit_w(&bars->v_empty[v_d.at]);
      ++d_turn;
      v_d.next();
      return true;
    };
    auto issue_dq = [&](int keys, bool first, bool adds) -> bool {  // dQ += dS K
      if (!mbar_wait_w(&bars->ds_full[q_turn & 1], (q_turn >> 1) & 1, w, kSiteDs)) return false;
      tc_fence_after();
      const uint64_t kd = dKmn + ((k_q.at * C::kTileBytes) >> 4);
      const uint32_t ds = tmem + col_s(q_turn & 1);
      auto step = [&](int kk) {
        umma_bf16_tmem_a_w(tmem + kColDQ, ds + (kk < 4 ? 0u : 64u) + (kk & 3) * 8, kd + ((kk * 16 * 128) >> 4), kIdKM,
                           (!first || kk > 0) ? 1u : 0u);
      };
      if (!adds) {
        // (the warps have read the tile: its buffers are free)
      } else if (keys == kBN) {
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk) step(kk);
      } else {
#pragma unroll 1
        for (int kk = 0; kk < keys / 16; ++kk) step(kk);
      }
      umma_commit_w(&bars->dq_done[q_turn & 1]);
      umma_commit_w(&bars->k_empty[k_q.at]);
      ++q_turn;
      k_q.next();
      return true;
    };
    bool ok = true;
    int idx = blockIdx.x;
    DqRun r{};
    if (idx < a.n_items) {
      r = run_of(g, item_of(a, idx));
      ok = mbar_wait_w(&bars->q_full, 0, w, kSiteQ) && issue_s(r.width(0));
      if (ok && r.nt == 1) umma_commit_w(&bars->q_empty);
      ok = ok && mbar_wait_w(&bars->do_full, 0, w, kSiteDo) && issue_dp(r.width(0));
      if (ok && r.nt == 1) umma_commit_w(&bars->do_empty);
    }
    while (ok && idx < a.n_items) {
      // here the item's first S and dP have been issued
      const int nt = r.nt;
      auto width = [&](int it) { return r.width(it); };
      if (nt > 1) {
        ok = issue_s(width(1));
        if (nt == 2) umma_commit_w(&bars->q_empty);
      }
      for (int it = 0; ok && it < nt; ++it) {
        // dP of the next tile as soon as this one's has been read, ahead of dQ
        if (it + 1 < nt) {
          ok = issue_dp(width(it + 1));
          if (it + 2 == nt) umma_commit_w(&bars->do_empty);
        }
        ok = ok && issue_dq(width(it), it == (r.n2 == r.n1 ? r.n1 : 0), r.adds(it));
        if (ok && it + 2 < nt) {  // S two tiles ahead
          ok = issue_s(width(it + 2));
          if (it + 3 == nt) umma_commit_w(&bars->q_empty);
        }
      }
      ++item;
      if (!ok || !(ok = feed_take(bars->feed, item, w, kSiteFeed, idx)) || idx >= a.n_items) break;
      // the next item's first tile, behind this one's last dQ: its Q and dO may still be on their way
      r = run_of(g, item_of(a, idx));
      ok = mbar_wait_w(&bars->q_full, item & 1, w, kSiteQ) && issue_s(r.width(0));
      if (ok && r.nt == 1) umma_commit_w(&bars->q_empty);
      ok = ok && mbar_wait_w(&bars->do_full, item & 1, w, kSiteDo) && issue_dp(r.width(0));
      if (ok && r.nt == 1) umma_commit_w(&bars->do_empty);
    }
    if (issued_any) {  // the products too: the warps that wait for the last ones may have given up
      umma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ compute warps
    const int wg = (warp - 2) >> 2;  // key columns [64 wg, 64 wg + 64)
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const int cbase = wg * 64;
    const float2 sl2 = make_float2(g.scale_log2, g.scale_log2);
    bool ok = true;
    int n = 0, item = 0, idx = blockIdx.x;
    for (; ok && idx < a.n_items; ++item) {
      const Item x = item_of(a, idx);
      const DqRun kr = run_of(g, x);
      const int i = x.q0 + row;
      const bool store = i < g.S;
      const size_t tab = (static_cast<size_t>(x.b) * g.Hq + x.h) * a.Lp + i;  // Lp covers the whole tile
      const float nl = a.lse2[tab];  // -inf on padding rows: their P is 0
      const float nd = a.delta[tab];
      const float2 nl2 = make_float2(nl, nl);
      float2 nd2 = make_float2(nd, nd), z2 = make_float2(1.f, 1.f);  // dS = P (z dP + nd)
      // visible keys of the row: [first, end) and the sinks [lo, sink_end); none past the end
      const int lo = store ? win_lo(g, i) : 1 << 30, end = i + 1;
      const int first = max(lo, i - g.W + 1), sink_end = min(lo + g.ns, i + 1);
      const int w0 = kr.kr.w0 * kBN;
      const int q_last = min(x.q0 + kBM, g.S) - 1;
      const int first_all = max(win_lo(g, q_last), q_last - g.W + 1);
      float2 res2 = make_float2(0.f, 0.f);
      float res = 0.f;
      for (int it = 0; it < kr.nt; ++it, ++n) {
        if (it == kr.n1) {  // the second pass needs the row's residue
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->r_full, item & 1, w, kSiteRes));
          if (!ok) break;
          const float* s = sRes + (item & 1) * 256 + row;
          res = s[0] + s[128];
          if (kr.n2 == kr.n1) {
            nd2 = make_float2(nd - res, nd - res);
          } else {  // the repeated tiles hold all keys of the rows of few, and only of those
            const float fix = i - lo + 1 < kFewKeys ? -res : 0.f;
            nd2 = make_float2(fix, fix);
            z2 = make_float2(0.f, 0.f);
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[n & 1], (n >> 1) & 1, w, kSiteS));
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->dp_full, n & 1, w, kSiteDp));
        if (!ok) break;
        tc_fence_after();
        const uint32_t cS = col_s(n & 1);
        const int k0 = kr.base(it), width = kr.width(it);
        const bool whole = k0 >= first_all && k0 + kBN - 1 <= x.q0;
        // (one copy of the code for both halves: the kernel's instructions stay in the cache)
        const int c_end = min(cbase + 64, width);  // a narrow tile has the first 32 columns at most: warpgroup 0
        if (cbase >= c_end) mbar_arrive_warp(&bars->dp_free);
#pragma unroll 1
        for (int c0 = cbase; c0 < c_end; c0 += 32) {
          uint32_t rs[32], rp[32];
          tmem_ld32(trow + kColDP + c0, rp);
          tmem_ld32(trow + cS + c0, rs);
          tmem_ld_wait();
          reg_fence32(rp);
          reg_fence32(rs);
          if (c0 + 32 >= c_end) {  // the tile's dP has been read: the next one's may start
            tc_fence_before();
            mbar_arrive_warp(&bars->dp_free);
          }
          if (!whole) {
            // (a sink tile ends where the window tiles begin)
            const uint32_t vis = k0 < w0 ? bits_between(lo - k0, min(sink_end, w0) - k0, c0)
                                         : bits_between(first - k0, end - k0, c0) | bits_between(lo - k0, sink_end - k0, c0);
            hide_columns(rs, vis, kMinusInf);
            // columns past a narrow tile's width hold what was there before (a hidden key's dP is finite: P = 0 hides it)
            if (width != kBN) hide_columns(rp, vis, 0u);
          }
          uint32_t dk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 y = ffma2(make_float2(__uint_as_float(rs[c]), __uint_as_float(rs[c + 1])), sl2, nl2);
            const float2 pv = make_float2(ex2_approx(y.x), ex2_approx(y.y));  // -inf -> 0
            const float2 ds =
                fmul2(pv, ffma2(make_float2(__uint_as_float(rp[c]), __uint_as_float(rp[c + 1])), z2, nd2));
            res2 = fadd2(res2, ds);
            dk[c >> 1] = pack_bf16x2(ds.x, ds.y);
          }
          if (kr.adds(it)) tmem_st16(trow + cS + cbase + (c0 - cbase) / 2, dk);
        }
        if (it + 1 == kr.n1) sRes[(item & 1) * 256 + wg * 128 + row] = res2.x + res2.y;
        tmem_st_wait();
        tc_fence_before();
        if (it + 1 == kr.n1) mbar_arrive_warp(&bars->r_full);
        mbar_arrive_warp(&bars->ds_full[n & 1]);
      }
      if (ok && kr.nt == kr.n1) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->r_full, item & 1, w, kSiteRes));
        const float* s = sRes + (item & 1) * 256 + row;
        res = s[0] + s[128];
      }
      if (ok && store && wg == 0) a.delta[tab] = nd - res;  // -(Delta + r): both warpgroups have read it
      // ------------------------------------------------------------ epilogue: dQ rows
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->dq_done[(n - 1) & 1], ((n - 1) >> 1) & 1, w, kSiteEpi));
      if (ok) {
        tc_fence_after();
        __nv_bfloat16* const dq0 = a.dq + (static_cast<size_t>(x.b) * g.S * g.Hq + x.h) * D;  // row 0 of the head
#pragma unroll 1
        for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
          uint32_t o[32], pk[16];
          tmem_ld32(trow + kColDQ + c0, o);
          tmem_ld_wait();
          reg_fence32(o);
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            pk[c >> 1] = pack_bf16x2(__uint_as_float(o[c]) * g.scale, __uint_as_float(o[c + 1]) * g.scale);
          store_rows32(dq0, static_cast<size_t>(g.Hq) * D, x.q0 + wq * 32, g.S, c0, pk);
        }
        ok = feed_take(bars->feed, item + 1, w, kSiteFeed, idx);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_d(const WinLaunch& L, cudaStream_t stream) {
  using C = Cfg<D>;
  static_assert(C::kSmemBytes <= 227 * 1024, "shared memory budget");
  cudaError_t e =
      cudaFuncSetAttribute(window_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  Args a{};
  a.g = L.g;
  a.div = make_item_div(L.g.Hq, L.g.B);
  a.lse2 = L.lse2;
  a.delta = L.delta;
  a.Lp = L.Lp;
  a.dq = static_cast<__nv_bfloat16*>(L.dq);
  a.status = L.status;
  a.wait_ns = L.wait_ns;
  const long long items = static_cast<long long>(L.g.n_tiles) * L.g.Hq * L.g.B;
  if (items > 0x3FFFFFFFLL) return cudaErrorInvalidConfiguration;
  a.n_items = static_cast<int>(items);
  const int sms = sm_count();
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  return launch_behind(window_dq_kernel<D>, dim3(grid), kThreads, C::kSmemBytes, stream, L.tm_q, L.tm_k, L.tm_v, L.tm_do, a);
}

}  // namespace

cudaError_t launch_window_dq(const WinLaunch& L, cudaStream_t stream) {
  return L.D == 128 ? launch_d<128>(L, stream) : L.D == 64 ? launch_d<64>(L, stream) : cudaErrorInvalidValue;
}

}  // namespace usp
