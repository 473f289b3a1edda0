// usp_window_fwd.cu -- forward of causal attention with a sliding window and
// sinks (visibility: usp_window.cuh), on sm_100a.
//
// O_i = sum_j p_ij v_j, p = softmax over the visible keys of scale q_i.k_j, by
// one pass over the key tiles with a running maximum and sum; LSE natural log.
//
// A persistent CTA (one per SM, 352 threads) takes work items: two 128-row query
// tiles that share every key tile -- the same rows of two heads of a group when
// the group is even (then both tiles need exactly the same keys), else two
// consecutive row tiles of a head. Roles:
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
  __device__ __forceinline__ int q_end(const WinGeo& g) const { return min(q0 + dq + kBM, g.S); }
};

// Items of one head unit run from the last rows back (the causally heaviest first).
__device__ __forceinline__ Item item_of(const WinGeo& g, int idx) {
  Item x;
  const int n_m = g.pair_heads ? g.n_tiles : (g.n_tiles + 1) / 2;
  const int m = n_m - 1 - idx % n_m;
  idx /= n_m;
  const int n_u = g.pair_heads ? g.Hq / 2 : g.Hq;
  const int u = idx % n_u;
  x.b = idx / n_u;
  if (g.pair_heads) {
    x.h = 2 * u;
    x.q0 = m * kBM;
    x.dh = 1;
    x.dq = 0;
  } else {
    x.h = u;
    x.q0 = 2 * m * kBM;
    x.dh = 0;
    x.dq = kBM;
  }
  return x;
}

template <int D>
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
      const Item x = item_of(g, idx);
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
          mbar_expect_tx_w(&bars->q_full, 2 * C::kTileBytes);
          for (int t = 0; t < 2; ++t)
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
    if (*reinterpret_cast<volatile int*>(&bars->abort_flag)) {
      // let every copy this warp started land before the CTA exits
      if (n_q > 0) mbar_wait_drain(&bars->q_full, (n_q - 1) & 1, a.wait_ns);
      for (int it = issued - n_st < 0 ? 0 : issued - n_st; it < issued; ++it)
        mbar_wait_drain(&full[it % n_st], (it / n_st) & 1, a.wait_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, D, 0, 1);
    const uint64_t dQ0 = sdesc_sw128(smem_addr(sQ), 16, 1024);
    const uint64_t dK0 = sdesc_sw128(smem_addr(sK), 16, 1024);
    const uint64_t dV0 = sdesc_sw128(smem_addr(sV), C::kPanelBytes, 1024);
    // S_t = Q_t K^T with stage ks; the narrow form takes the stage's first `keys` (16 or 32)
    auto issue_s_as = [&](int t, int ks, uint32_t idesc) {
      const uint64_t qd = dQ0 + ((t * C::kTileBytes) >> 4), kd = dK0 + ((ks * C::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::kPanelBytes + (kk & 3) * 32) >> 4;
        umma_bf16_w(tmem + col_s(t), qd + off, kd + off, idesc, kk > 0 ? 1u : 0u);
      }
      umma_commit_w(&bars->s_full[t]);
    };
    auto issue_s = [&](int t, int ks, int keys) {
      if (keys == kBN)
        issue_s_as(t, ks, idesc_bf16_f32(kBM, kBN, 0, 0));
      else
        issue_s_as(t, ks, idesc_bf16_f32(kBM, keys, 0, 0));
    };
    auto run_of = [&](int idx) {
      const Item x = item_of(g, idx);
      return key_run(g, x.q0, x.q_end(g));
    };
    bool ok = true, issued_any = false;
    int idx = blockIdx.x;
    if (idx < a.n_items) {
      KeyRun kr = run_of(idx);
      int it = 0, item = 0;
      ok = mbar_wait_w(&bars->q_full, 0, w, kSiteQ) && mbar_wait_w(&bars->k_full[0], 0, w, kSiteK);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0, kr.width(0));
        issue_s(1, 0, kr.width(0));
        umma_commit_w(&bars->k_empty[0]);
        if (kr.nt == 1) umma_commit_w(&bars->q_empty);
        issued_any = true;
      }
      for (int n = 0; ok; ++n) {  // n: key tile of the CTA's stream, it: of the item
        const int s = n % C::kVSt, s1 = (n + 1) % C::kKSt;
        const bool last = it + 1 == kr.nt;
        int next = 0;
        if (last && !feed_take(bars->feed, item + 1, w, kSiteFeed, next)) { ok = false; break; }
        const bool more = !last || next < a.n_items;
        const KeyRun next_kr = last && more ? run_of(next) : kr;
        const int next_it = last ? 0 : it + 1;
        const int pv_steps = kr.width(it) / 16;  // 16-key steps of this tile's products: 1, 2 or 8
        if (!mbar_wait_w(&bars->v_full[s], (n / C::kVSt) & 1, w, kSiteV)) { ok = false; break; }
        const uint64_t vd = dV0 + ((s * C::kTileBytes) >> 4);
        auto issue_pv = [&](int t) -> bool {  // in two halves of 64 keys, each as soon as its P is in TMEM
          if (!mbar_wait_w(&bars->p_half[t], n & 1, w, kSiteP)) return false;
          tc_fence_after();
          if (pv_steps == kBN / 16) {
#pragma unroll
            for (int kk = 0; kk < kBN / 32; ++kk)
              umma_bf16_tmem_a_w(tmem + col_o(t), tmem + col_s(t) + kk * 8, vd + ((kk * 16 * 128) >> 4), kIdescPV,
                                 (it > 0 || kk > 0) ? 1u : 0u);
            if (!mbar_wait_w(&bars->p_full[t], n & 1, w, kSiteP)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = kBN / 32; kk < kBN / 16; ++kk)
              umma_bf16_tmem_a_w(tmem + col_o(t), tmem + col_s(t) + kk * 8, vd + ((kk * 16 * 128) >> 4), kIdescPV, 1u);
          } else {  // a narrow tile: one or two steps, all of its P handed over at once
#pragma unroll 1
            for (int kk = 0; kk < pv_steps; ++kk)
              umma_bf16_tmem_a_w(tmem + col_o(t), tmem + col_s(t) + kk * 8, vd + ((kk * 16 * 128) >> 4), kIdescPV,
                                 (it > 0 || kk > 0) ? 1u : 0u);
            if (!mbar_wait_w(&bars->p_full[t], n & 1, w, kSiteP)) return false;
          }
          umma_commit_w(&bars->pv_done[t]);
          if (t == 1) umma_commit_w(&bars->v_empty[s]);
          return true;
        };
        auto next_s = [&](int t) -> bool {  // S_t of the next tile overwrites P_t: behind this tile's PV_t
          if (!mbar_wait_w(&bars->pv_done[t], n & 1, w, kSitePvDone)) return false;
          tc_fence_after();
          issue_s(t, s1, next_kr.width(next_it));
          if (t == 1) {
            umma_commit_w(&bars->k_empty[s1]);
            if (next_it + 1 == next_kr.nt) umma_commit_w(&bars->q_empty);
          }
          return true;
        };
        auto next_k = [&]() { return mbar_wait_w(&bars->k_full[s1], ((n + 1) / C::kKSt) & 1, w, kSiteK); };
        if (!last) {
          ok = issue_pv(0) && next_k() && next_s(0) && issue_pv(1) && next_s(1);
        } else {  // the next item's Q may still be on its way: this item's products first
          ok = issue_pv(0) && issue_pv(1);
          if (ok && more) ok = mbar_wait_w(&bars->q_full, (item + 1) & 1, w, kSiteQ) && next_k() && next_s(0) && next_s(1);
        }
        if (!ok || !more) break;
        if (last) ++item;
        kr = next_kr;
        it = next_it;
      }
    }
    if (!ok && issued_any) {
      umma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0, a.wait_ns);
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
      const Item x = item_of(g, idx);
      const KeyRun kr = key_run(g, x.q0, x.q_end(g));
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
      const int n_end = n + kr.nt;
      const float2 sl2 = make_float2(g.scale_log2, g.scale_log2);
      auto rescale_o = [&](float alpha) {  // the previous PV has landed: S_t is issued behind it
#pragma unroll
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
      for (int k0 = kr.lo, y = 0; y < kr.n_s; ++y, ++n, k0 += kSinkTile) {  // sink tiles: one group of 32 columns
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
      int k0 = w0;
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
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->pv_done[t], (n - 1) & 1, w, kSiteO));
      if (ok) {
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
        ok = feed_take(bars->feed, k, w, kSiteFeed, idx);
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
      cudaFuncSetAttribute(window_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  Args a{};
  a.g = L.g;
  a.g.pair_heads = L.g.G % 2 == 0;
  a.out = static_cast<__nv_bfloat16*>(L.out);
  a.lse = L.lse;
  a.status = L.status;
  a.wait_ns = L.wait_ns;
  const long long items = a.g.pair_heads ? static_cast<long long>(L.g.n_tiles) * (L.g.Hq / 2) * L.g.B
                                         : static_cast<long long>((L.g.n_tiles + 1) / 2) * L.g.Hq * L.g.B;
  if (items > 0x3FFFFFFFLL) return cudaErrorInvalidConfiguration;
  a.n_items = static_cast<int>(items);
  const int sms = sm_count();
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  window_fwd_kernel<D><<<grid, kThreads, C::kSmemBytes, stream>>>(L.tm_q, L.tm_k, L.tm_v, a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_fwd(const WinLaunch& L, cudaStream_t stream) {
  return L.D == 128 ? launch_d<128>(L, stream) : L.D == 64 ? launch_d<64>(L, stream) : cudaErrorInvalidValue;
}

}  // namespace usp
