// usp_window_fwd.cu -- forward of causal attention with a sliding window and
// sinks (visibility: usp_window.cuh), on sm_100a.
//
// O_i = sum_j p_ij v_j, p = softmax over the visible keys of scale q_i.k_j, by
// one pass over the key tiles with a running maximum and sum; LSE natural log.
//
// A persistent CTA (one per SM, 352 threads) takes work items: two 128-row query
// tiles that share every key tile -- the same rows of two heads of a group when
// the group is even (then both tiles need exactly the same keys), else two
// consecutive row tiles of a head, each taking the key tiles of its own window. Items of
// one query tile take 55 to 65 % of a pair's time; the pairs that would leave half of the
// SMs idle at the end of the launch are taken apart into them. Roles:
//   warp 0      TMA producer of K (3 stages) and of the item's two Q tiles
//   warp 10     TMA producer of V
//   warp 1      UMMA issuer: per key tile and query tile t, O_t += P_t V (A = P_t
//               from TMEM, in two halves of 64 keys), then S_t of the next tile
//   warps 2..5, 6..9  softmax of tile 0 / 1: thread = query row = TMEM lane
// The CTAs take the items from a counter as they get ready (ItemFeed).
// TMEM: S_t / P_t at 128 t, O_t at 256 + 128 t. The key tiles of all items of a
// CTA form one stream: the S of the next item's first tile is issued behind the
// last PV of this one, so its loads and products overlap this item's epilogue;
// its first PV cannot overtake the epilogue's reads of O because it waits for P,
// which the same warps write after them.
//
// Bound by the chain S -> softmax -> PV -> S of each query tile, two of which
// alternate (1.86 us per key tile of a pair; the products alone take 1.1), and by
// about 4 us per item (first scores, masked edges, 64 KB of stores). B=1 S=32768 H=16/4
// D=128 W=2048, 4 sinks: 537 us, 994 TFLOP/s of visible pairs; S=16384 H=32/8 W=1024:
// 315 us, 849 TFLOP/s.
#include <math.h>

#include "usp_ptx.cuh"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kThreads = 352;
constexpr int kWarpV = 10;
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThresh = 8.0f;  // log2 units: O is rescaled only when the max grows by more than 2^8

__host__ __device__ constexpr uint32_t col_s(int t) { return 128u * t; }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * t; }

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanelBytes = 128 * 128;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr int kKSt = 3;
  static constexpr int kVSt = D == 128 ? 2 : 3;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = 2 * kTileBytes;
  static constexpr int kOffV = kOffK + kKSt * kTileBytes;
  static constexpr int kOffBar = kOffV + kVSt * kTileBytes;
  static constexpr int kSmemBytes = kOffBar + 320;
};

struct Args {
  WinGeo g;
  ItemDiv div;
  int n_pairs;  // the items from here on are single query tiles; 0: all, numbered by head
  __nv_bfloat16* out;
  float* lse;
  int n_items;
  int* status;
  unsigned long long wait_ns;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full[2], p_half[2], p_full[2], pv_done[2];
  uint64_t drain;
  ItemFeed feed;
  uint32_t tmem_base;
  int abort_flag;
};

enum : int {
  kSiteQEmpty = 0x401, kSiteKEmpty = 0x402, kSiteVEmpty = 0x403, kSiteQ = 0x411, kSiteK = 0x412, kSiteV = 0x413,
  kSiteP = 0x414, kSitePvDone = 0x415, kSiteS = 0x421, kSiteO = 0x422,
  kSiteFeed = 0x431, kSiteAlign = 0x4FF
};

struct Item {
  int b, h, q0;     // batch, head and first row of query tile 0
  int dh, dq;       // what tile 1 adds to them
  bool one;         // there is no tile 1
  __device__ __forceinline__ int q_end(const WinGeo& g) const { return min(q0 + dq + kBM, g.S); }
};

// The last rows of every head come first, the heads of a batch side by side: their
// key tiles are in L2 for the rows before them, and the short walks of the first rows
// fill the end of the launch.
__device__ __forceinline__ Item item_of(const Args& a, int idx) {
  const WinGeo& g = a.g;
  Item x;
  x.dh = x.dq = 0;
  x.one = idx >= a.n_pairs;
  const int half = x.one && a.n_pairs > 0 ? (idx - a.n_pairs) & 1 : 0;
  if (x.one && a.n_pairs > 0) idx = a.n_pairs + ((idx - a.n_pairs) >> 1);
  const ItemParts p = item_parts(a.div, idx);
  x.b = p.b;
  if (a.n_pairs == 0) {
    x.h = p.head;
    x.q0 = (g.n_tiles - 1 - p.rest) * kBM;
  } else if (g.pair_heads) {
    x.h = 2 * p.head + half;
    x.q0 = (g.n_tiles - 1 - p.rest) * kBM;
    x.dh = x.one ? 0 : 1;
  } else {
    x.h = p.head;
    x.q0 = (2 * ((g.n_tiles + 1) / 2 - 1 - p.rest) + half) * kBM;
    x.dq = x.one ? 0 : kBM;
  }
  return x;
}

// The key tiles of an item, and those of them that query tile t takes: the sinks' and
// the window's [begin[t], end[t]) (numbers of the run); none at all without rows.
struct ItemRun {
  KeyRun kr;
  int begin1, end0, end1;  // tile 0 begins, and the later of the two ends, with the run
  __device__ __forceinline__ bool takes(int t, int it) const {
    return t == 0 ? it < end0 : it < end1 && (it < kr.n_s || it >= begin1);
  }
};
__device__ __forceinline__ ItemRun run_of(const WinGeo& g, const Item& x) {
  ItemRun r;
  r.kr = key_run(g, x.q0, x.q_end(g));
  r.end0 = r.end1 = r.kr.nt;
  r.begin1 = r.kr.n_s;
  if (x.dq) {
    const int q1 = x.q0 + x.dq;
    if (q1 < g.S) {
      const int lo1 = win_lo(g, q1);
      r.end0 = r.kr.nt - 1;
      int first = max(lo1, q1 - g.W + 1) / kBN;
      // its sinks may lie among the window's first tiles
      if (lo1 + g.ns > r.kr.w0 * kBN) first = min(first, lo1 / kBN);
      r.begin1 = r.kr.n_s + max(first - r.kr.w0, 0);
    } else {
      r.end1 = 0;
    }
  }
  if (x.one) r.end1 = 0;
  return r;
}

// kHeads: the pairs are two heads of a group (both tiles take every key tile).
template <int D, bool kHeads>
__global__ void __launch_bounds__(kThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kSiteAlign);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  static_assert(sizeof(Bars) <= 320, "barrier block");
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinGeo& g = a.g;

  if (threadIdx.x == 0) {
    bars->abort_flag = *reinterpret_cast<volatile int*>(a.status) != 0;
    feed_init(bars->feed, 10);  // the V producer, the issuer and eight softmax warps take
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_half[t], 4);  // one arrival per softmax warp
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->pv_done[t], 1);
    }
    mbar_init(&bars->drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&bars->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl w{&bars->abort_flag, a.status, a.wait_ns};
  const bool skip = bars->abort_flag != 0;

  if (skip) {
    // nothing issued, nothing to drain
  } else if (warp == 0 || warp == kWarpV) {
    // ------------------------------------------------------------ TMA producers
    const bool kside = warp == 0;
    const int n_st = kside ? C::kKSt : C::kVSt;
    uint64_t* full = kside ? bars->k_full : bars->v_full;
    uint64_t* empty = kside ? bars->k_empty : bars->v_empty;
    const CUtensorMap* tm = kside ? &tm_k : &tm_v;
    uint8_t* sbuf = kside ? sK : sV;
    if (lane == 0) {
      if (kside) tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(tm);
    }
    __syncwarp();
    int issued = 0, n_q = 0;
    bool ok = true;
    int idx = blockIdx.x, next = 0;
    for (int k = 1; ok && idx < a.n_items; ++k, idx = next) {
      const Item x = item_of(a, idx);
      const KeyRun kr = key_run(g, x.q0, x.q_end(g));
      for (int it = 0; it < kr.nt; ++it) {
        const int s = issued % n_st;
        if (issued >= n_st &&
            !mbar_wait_w(&empty[s], ((issued / n_st) - 1) & 1, w, kside ? kSiteKEmpty : kSiteVEmpty)) {
          ok = false;
          break;
        }
        mbar_expect_tx_w(&full[s], C::kTileBytes);
        for (int p = 0; p < C::kPanels; ++p)
          tma_load_4d_w(tm, &full[s], sbuf + s * C::kTileBytes + p * C::kPanelBytes, p * 64, x.h / g.G,
                        kr.base(it), x.b);
        ++issued;
        if (kside && it == 0) {
          // Q behind the first K: its buffer frees last, when the previous item's last S is done
          if (n_q >= 1 && !mbar_wait_w(&bars->q_empty, (n_q - 1) & 1, w, kSiteQEmpty)) {
            ok = false;
            break;
          }
          const int n_t = x.one ? 1 : 2;
          mbar_expect_tx_w(&bars->q_full, n_t * C::kTileBytes);
          for (int t = 0; t < n_t; ++t)
            for (int p = 0; p < C::kPanels; ++p)
              tma_load_4d_w(&tm_q, &bars->q_full, sQ + t * C::kTileBytes + p * C::kPanelBytes, p * 64, x.h + t * x.dh,
                            x.q0 + t * x.dq, x.b);
          ++n_q;
          if (!feed_give(bars->feed, k, a.status + kCounterFwd, w, kSiteFeed, next)) {
            ok = false;
            break;
          }
        }
      }
      if (ok && !kside) ok = feed_take(bars->feed, k, w, kSiteFeed, next);
    }
    // Every copy this warp started lands before the CTA ends, whoever may have given up since.
    if (n_q > 0) mbar_wait_drain(&bars->q_full, (n_q - 1) & 1);
    for (int it = issued - n_st < 0 ? 0 : issued - n_st; it < issued; ++it)
      mbar_wait_drain(&full[it % n_st], (it / n_st) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, D, 0, 1);
    const uint64_t dQ0 = sdesc_sw128(smem_addr(sQ), 16, 1024);
    const uint64_t dK0 = sdesc_sw128(smem_addr(sK), 16, 1024);
    const uint64_t dV0 = sdesc_sw128(smem_addr(sV), C::kPanelBytes, 1024);
    bool ok = true, issued_any = false;
    Ring<C::kKSt> k_s;                // the K stage that S takes next
    Ring<C::kVSt> v_p;                // the V stage that PV takes
    uint32_t n_pv[2] = {0, 0};        // PV issued so far of each query tile
    // S_t = Q_t K^T with the first `keys` rows of stage k_s (128; 16 or 32 in a sink tile); it overwrites
    // P_t, so it waits for the last PV_t
    auto issue_s = [&](int t, int keys) -> bool {
      if (n_pv[t] > 0 && !mbar_wait_w(&bars->pv_done[t], (n_pv[t] - 1) & 1, w, kSitePvDone)) return false;
      tc_fence_after();
      const uint64_t qd = dQ0 + ((t * C::kTileBytes) >> 4), kd = dK0 + ((k_s.at * C::kTileBytes) >> 4);
      auto go = [&](uint32_t idesc) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kPanelBytes + (kk & 3) * 32) >> 4;
          umma_bf16_w(tmem + col_s(t), qd + off, kd + off, idesc, kk > 0 ? 1u : 0u);
        }
      };
      if (keys == kBN)
        go(idesc_bf16_f32(kBM, kBN, 0, 0));
      else
        go(idesc_bf16_f32(kBM, keys, 0, 0));
      umma_commit_w(&bars->s_full[t]);
      issued_any = true;
      return true;
    };
    // O_t += P_t V in two halves of 64 keys, each as soon as its P is in TMEM
    auto issue_pv = [&](int t, int keys, bool first) -> bool {
      if (!mbar_wait_w(&bars->p_half[t], n_pv[t] & 1, w, kSiteP)) return false;
      tc_fence_after();
      const uint64_t vd = dV0 + ((v_p.at * C::kTileBytes) >> 4);
      auto step = [&](int kk) {
        umma_bf16_tmem_a_w(tmem + col_o(t), tmem + col_s(t) + kk * 8, vd + ((kk * 16 * 128) >> 4), kIdescPV,
                           (!first || kk > 0) ? 1u : 0u);
      };
      if (keys == kBN) {
#pragma unroll
        for (int kk = 0; kk < kBN / 32; ++kk) step(kk);
        if (!mbar_wait_w(&bars->p_full[t], n_pv[t] & 1, w, kSiteP)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = kBN / 32; kk < kBN / 16; ++kk) step(kk);
      } else {  // a sink tile: one or two steps, all of its P handed over at once
#pragma unroll 1
        for (int kk = 0; kk < keys / 16; ++kk) step(kk);
        if (!mbar_wait_w(&bars->p_full[t], n_pv[t] & 1, w, kSiteP)) return false;
      }
      umma_commit_w(&bars->pv_done[t]);
      ++n_pv[t];
      return true;
    };
    uint32_t item = 0;
    int idx = blockIdx.x;
    while (ok && idx < a.n_items) {
      const ItemRun r = run_of(g, item_of(a, idx));
      const int nt = r.kr.nt;
      auto takes = [&](int t, int it) { return kHeads ? t == 0 || r.end1 > 0 : r.takes(t, it); };
      // the item's first S, behind the last PV of the item before
      ok = mbar_wait_w(&bars->q_full, item & 1, w, kSiteQ) && mbar_wait_w(&bars->k_full[k_s.at], k_s.phase, w, kSiteK);
      for (int t = 0; ok && t < 2; ++t)
        if (takes(t, 0)) ok = issue_s(t, r.kr.width(0));
      if (!ok) break;
      umma_commit_w(&bars->k_empty[k_s.at]);
      k_s.next();
      if (nt == 1) umma_commit_w(&bars->q_empty);
      for (int it = 0; ok && it < nt; ++it) {
        if (!mbar_wait_w(&bars->v_full[v_p.at], v_p.phase, w, kSiteV)) { ok = false; break; }
        const bool more = it + 1 < nt;
        // per query tile PV_t, then S_t of the next key tile: the tensor core runs one tile's products
        // while the other's softmax works
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (takes(t, it) && !issue_pv(t, r.kr.width(it), kHeads || t == 0 || r.kr.n_s > 0 ? it == 0 : it == r.begin1)) {
            ok = false;
            break;
          }
          if (t == 1) umma_commit_w(&bars->v_empty[v_p.at]);
          if (more) {
            if (t == 0 && !mbar_wait_w(&bars->k_full[k_s.at], k_s.phase, w, kSiteK)) { ok = false; break; }
            if (takes(t, it + 1) && !issue_s(t, r.kr.width(it + 1))) { ok = false; break; }
            if (t == 1) {
              umma_commit_w(&bars->k_empty[k_s.at]);
              if (it + 2 == nt) umma_commit_w(&bars->q_empty);
            }
          }
        }
        if (!ok) break;
        v_p.next();
        if (more) k_s.next();
      }
      ++item;
      if (ok) ok = feed_take(bars->feed, item, w, kSiteFeed, idx);
    }
    if (issued_any) {  // the products too: the warps that wait for the last ones may have given up
      umma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int t = (warp - 2) >> 2;
    const int wq = warp & 3;  // TMEM lane quarter
    const int row = wq * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t cS = col_s(t), cO = col_o(t);
    bool ok = true;
    int n = 0;  // key tile of the CTA's stream
    int idx = blockIdx.x;
    for (int k = 1; ok && idx < a.n_items; ++k) {
      const Item x = item_of(a, idx);
      const ItemRun r = run_of(g, x);
      const KeyRun& kr = r.kr;
      const int h = x.h + t * x.dh, q0 = x.q0 + t * x.dq;
      const int i = q0 + row;
      const bool store = i < g.S;
      // the row's document start; one that no key reaches for a row past the end
      const int lo = store ? win_lo(g, i) : 1 << 30;
      // the first key that every row of the tile sees
      const int q_last = min(q0 + kBM, g.S) - 1;
      const int first_all = q_last < q0 ? INT_MAX : max(win_lo(g, q_last), q_last - g.W + 1);
      // l_run: sum of the fp32 weights (LSE); lb_run: sum of the bf16-rounded weights that the
      // PV product takes (O's divisor, so that O stays a convex combination of V rows)
      float m_use = -INFINITY, l_run = 0.f, lb_run = 0.f;
      const int n0 = n;
      // this tile's window tiles, from k0 on, behind the sinks'
      const int t_begin = kHeads || t == 0 ? kr.n_s : r.begin1, t_end = t == 0 ? r.end0 : r.end1;
      const int n_sink = t_end > 0 ? kr.n_s : 0, n_end = n + n_sink + max(t_end - t_begin, 0);
      const float2 sl2 = make_float2(g.scale_log2, g.scale_log2);
      auto rescale_o = [&](float alpha) {  // the previous PV has landed: S_t is issued behind it
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32];
          tmem_ld32(trow + cO + c0, o);
          tmem_ld_wait();
          reg_fence32(o);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
          tmem_st32(trow + cO + c0, o);
        }
      };
      const int w0 = kr.w0 * kBN;
      for (int k0 = kr.lo, y = 0; y < n_sink; ++y, ++n, k0 += kSinkTile) {  // sink tiles: one group of 32 columns
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[t], n & 1, w, kSiteS));
        if (!ok) break;
        tc_fence_after();
        uint32_t r[32];
        tmem_ld32(trow + cS, r);
        tmem_ld_wait();
        reg_fence32(r);
        const uint32_t vis = bits_between(lo - k0, min(min(lo + g.ns, i + 1), w0) - k0, 0);
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          if (!((vis >> c) & 1u)) r[c] = 0xFF800000u;
          mx = fmaxf(mx, __uint_as_float(r[c]));
        }
        const float m_tile = mx * g.scale_log2;
        const bool bump = m_tile > m_use + (y == 0 ? 0.f : kRescaleThresh);
        float alpha = 1.f;
        if (bump) {
          alpha = ex2_approx(m_use - m_tile);
          m_use = m_tile;
        }
        if (y > 0 && __any_sync(0xffffffffu, bump)) rescale_o(alpha);
        const float m_safe = m_use == -INFINITY ? 0.f : m_use;
        float2 acc = make_float2(0.f, 0.f), accb = acc;
        uint32_t pk[16];
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 y = ffma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sl2,
                                 make_float2(-m_safe, -m_safe));
          const float2 pv = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          acc = fadd2(acc, pv);
          pk[c >> 1] = pack_bf16x2(pv.x, pv.y);
          accb = add_bf16x2_f32(accb, pk[c >> 1]);
        }
        l_run = l_run * alpha + (acc.x + acc.y);
        lb_run = lb_run * alpha + (accb.x + accb.y);
        tmem_st16(trow + cS, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_half[t]);
        mbar_arrive_warp(&bars->p_full[t]);
      }
      if (!ok) break;
      int k0 = w0 + (t_begin - kr.n_s) * kBN;
      for (; n < n_end; ++n) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[t], n & 1, w, kSiteS));
        if (!ok) break;
        tc_fence_after();
        uint32_t r0[32], r1[32], r2[32], r3[32];
        tmem_ld32(trow + cS + 0, r0);
        tmem_ld32(trow + cS + 32, r1);
        tmem_ld32(trow + cS + 64, r2);
        tmem_ld32(trow + cS + 96, r3);
        tmem_ld_wait();
        reg_fence32(r0);
        reg_fence32(r1);
        reg_fence32(r2);
        reg_fence32(r3);
        if (!(k0 >= first_all && k0 + kBN - 1 <= q0)) {  // not visible as a whole: -inf where it is not
          const int first = max(lo, i - g.W + 1), sink_end = min(lo + g.ns, i + 1);
          auto hide = [&](uint32_t (&r)[32], int c0) {
            hide_columns(r, bits_between(first - k0, i + 1 - k0, c0) | bits_between(lo - k0, sink_end - k0, c0), kMinusInf);
          };
          hide(r0, 0);
          hide(r1, 32);
          hide(r2, 64);
          hide(r3, 96);
        }
        float pm[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          pm[q] = fmax3(__uint_as_float(r0[q]), __uint_as_float(r1[q]), __uint_as_float(r2[q]));
#pragma unroll
        for (int c = 8; c < 32; c += 8) {
#pragma unroll
          for (int q = 0; q < 8; ++q) pm[q] = fmax3(pm[q], __uint_as_float(r0[c + q]), __uint_as_float(r1[c + q]));
#pragma unroll
          for (int q = 0; q < 8; ++q) pm[q] = fmax3(pm[q], __uint_as_float(r2[c + q]), __uint_as_float(r3[c + q]));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) pm[q] = fmaxf(pm[q], __uint_as_float(r3[q]));
        const float mx = fmaxf(fmax3(pm[0], pm[1], pm[2]), fmax3(pm[3], pm[4], fmax3(pm[5], pm[6], pm[7])));
        const float m_tile = mx * g.scale_log2;
        const bool bump = m_tile > m_use + kRescaleThresh;
        float alpha = 1.f;
        if (bump) {
          alpha = ex2_approx(m_use - m_tile);
          m_use = m_tile;
        }
        const float m_safe = m_use == -INFINITY ? 0.f : m_use;
        float2 acc[2], accb[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) acc[q] = accb[q] = make_float2(0.f, 0.f);
        const float2 nm = make_float2(-m_safe, -m_safe);
        auto emit = [&](const uint32_t (&r)[32], uint32_t col) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 y = ffma2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sl2, nm);
            const float2 pv = make_float2(ex2_approx(y.x), ex2_approx(y.y));
            acc[(c >> 1) & 1] = fadd2(acc[(c >> 1) & 1], pv);
            pk[c >> 1] = pack_bf16x2(pv.x, pv.y);
            accb[(c >> 1) & 1] = add_bf16x2_f32(accb[(c >> 1) & 1], pk[c >> 1]);
          }
          tmem_st16(trow + cS + col, pk);
        };
        emit(r0, 0);
        emit(r1, 16);
        // before the first half of P is handed over
        if (n > n0 && __any_sync(0xffffffffu, bump)) rescale_o(alpha);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_half[t]);
        emit(r2, 32);
        emit(r3, 48);
        const float rs = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
        const float rsb = (accb[0].x + accb[0].y) + (accb[1].x + accb[1].y);
        l_run = l_run * alpha + rs;
        lb_run = lb_run * alpha + rsb;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_full[t]);
        k0 += kBN;
      }
      // ------------------------------------------------------------ epilogue
      if (ok && n > n0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[t], (n - 1) & 1, w, kSiteO));
      if (ok && n > n0) {
        tc_fence_after();
        const float inv_l = lb_run > 0.f ? 1.f / lb_run : 0.f;
        const size_t row_idx = (static_cast<size_t>(x.b) * g.S + (store ? i : 0)) * g.Hq + h;
        __nv_bfloat16* const o0 = a.out + (static_cast<size_t>(x.b) * g.S * g.Hq + h) * D;  // row 0 of the head
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t o[32], pk[16];
          tmem_ld32(trow + cO + c0, o);
          tmem_ld_wait();
          reg_fence32(o);
#pragma unroll
          for (int c = 0; c < 32; c += 2)
            pk[c >> 1] = pack_bf16x2(__uint_as_float(o[c]) * inv_l, __uint_as_float(o[c + 1]) * inv_l);
          store_rows32(o0, static_cast<size_t>(g.Hq) * D, q0 + wq * 32, g.S, c0, pk);
        }
        if (store) a.lse[row_idx] = (m_use + __log2f(l_run)) * 0.6931471805599453f;  // every row sees itself
      }
      if (ok) ok = feed_take(bars->feed, k, w, kSiteFeed, idx);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool kHeads>
cudaError_t launch_d(const WinLaunch& L, cudaStream_t stream) {
  using C = Cfg<D>;
  static_assert(C::kSmemBytes <= 227 * 1024, "shared memory budget");
  cudaError_t e =
      cudaFuncSetAttribute(window_fwd_kernel<D, kHeads>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  Args a{};
  a.g = L.g;
  a.g.pair_heads = kHeads;
  a.out = static_cast<__nv_bfloat16*>(L.out);
  a.lse = L.lse;
  a.status = L.status;
  a.wait_ns = L.wait_ns;
  const int heads = kHeads ? L.g.Hq / 2 : L.g.Hq, rows = kHeads ? L.g.n_tiles : (L.g.n_tiles + 1) / 2;
  const long long pairs = static_cast<long long>(rows) * heads * L.g.B;
  if (pairs > 0x1FFFFFFFLL) return cudaErrorInvalidConfiguration;
  // What the SMs' last round would take of the pairs, if it is no more than half a round, as single
  // tiles (512 head pairs on 148 SMs, 2 or 3 key tiles each: 36.9 -> 35.4 us). The last row pair of a head may lack its
  // second tile: it comes first, and is not taken apart.
  const int sms = sm_count();
  const long long rest = pairs % sms;
  a.n_pairs = static_cast<int>(pairs);
  long long items = pairs;
  if (pairs == rest && 2 * rest <= sms) {
    a.n_pairs = 0;
    items = static_cast<long long>(L.g.n_tiles) * L.g.Hq * L.g.B;
  } else if (2 * rest <= sms && (kHeads || L.g.n_tiles % 2 == 0 || rest <= pairs - static_cast<long long>(heads) * L.g.B)) {
    a.n_pairs = static_cast<int>(pairs - rest);
    items = pairs + rest;
  }
  a.div = make_item_div(a.n_pairs ? heads : L.g.Hq, L.g.B);
  a.n_items = static_cast<int>(items);
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  window_fwd_kernel<D, kHeads><<<grid, kThreads, C::kSmemBytes, stream>>>(L.tm_q, L.tm_k, L.tm_v, a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd(const WinLaunch& L, cudaStream_t stream) {
  const bool heads = L.g.G % 2 == 0;
  if (L.D == 128) return heads ? launch_d<128, true>(L, stream) : launch_d<128, false>(L, stream);
  if (L.D == 64) return heads ? launch_d<64, true>(L, stream) : launch_d<64, false>(L, stream);
  return cudaErrorInvalidValue;
}

}  // namespace usp
