// usp_window_dq.cu -- backward of sliding-window attention with sinks, the
// query-major half (dQ) on sm_100a:
//   dQ_i = scale sum_j P_ij (dO_i.v_j - Delta_i) k_j
// over the key tiles that the forward walks (usp_window.cuh). dQ accumulates in
// TMEM over the walk and is written once, as bf16.
//
// A persistent CTA (one per SM, 320 threads) takes work items: one 128-row query
// tile of one head.
//   warp 0      TMA producer: Q, dO per item, K (3 stages) and V (2 stages) per key tile
//   warp 1      UMMA issuer: S = Q K^T, dP = dO V^T, A += P K, B += dS K
//   warps 2..9  two warpgroups of 64 key columns; thread = query row
// The gradient sums of a row cancel: sum_j dS_ij = 0 with the exact Delta_i =
// sum_j P_ij dP_ij, while dO.O of the bf16 output is off by up to 2^-8 |dO||O|. With
// that Delta', the residue r_i = sum_j dS'_ij = Delta_i - Delta'_i (added up in fp32) and
//   dQ_i / scale = sum_j dS'_ij k_j - r_i sum_j P_ij k_j = B_i - r_i A_i.
// A is a fourth product beside the three, for every row: without it dQ is off by
// r_i A_i, which stands beside a dQ that cancels alike wherever a row's keys or
// values have much in common (one key with most of the weight, a common part, or
// repeated tokens: 4 to 49 times the bound of the roundings in such rows), not only where a
// row has few keys. r and A are good to 2^-8, so what is left of r is as small beside
// it as a rounding. Delta_i goes back to the table, for the key-major kernels that run after.
//
// TMEM: S / P at 0 (D=64: a second buffer at 384), dP / dS at 128, B at 256, A behind
// it. The key tiles of all items of a CTA form one stream: the next item's first S and
// dP are issued behind this one's last products, and its first A and B wait for P and
// dS, written by the warps that read this item's A and B before them.
//
// Bound by the compute warps' two phases, one behind the other, and four products that
// take 1.1 us of the 1.8 us per key tile (tensor pipe 60 % active), and by about 3.5 us per
// item. B=1 S=32768 H=16/4 D=128 W=2048, 4 sinks: 930 us, 861 TFLOP/s of 6 D flops per visible
// pair (8 D with A); with the three products 761. Backward of 8192 tokens, W=8, where every row
// had walked its keys twice for the residue: 107 us against 136.
#include <math.h>

#include "usp_ptx.cuh"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kThreads = 320;
constexpr int kComputeWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColDP = 128, kColB = 256;
__host__ __device__ constexpr uint32_t col_s(int b) { return 384u * b; }

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanelBytes = 128 * 128;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr int kKSt = 3;
  static constexpr int kVSt = 2;
  static constexpr int kSSt = D == 64 ? 2 : 1;  // S buffers
  static constexpr uint32_t kColA = kColB + D;
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
  // One p_full per S buffer: with two, the warps can have made P of two tiles before the issuer looks for
  // the first one's arrivals (dP of the second is on its way by then), but not of a third, whose S waits for A.
  uint64_t s_full[2], p_full[2], p_used[2], dp_full, ds_full, ds_used, drain;
  uint64_t r_full;  // both warpgroups' residues of the item are in sRes
  ItemFeed feed;
  uint32_t tmem_base;
  int abort_flag;
};

enum : int {
  kSiteQEmpty = 0x601, kSiteDoEmpty = 0x602, kSiteKEmpty = 0x603, kSiteVEmpty = 0x604, kSiteQ = 0x611, kSiteDo = 0x612,
  kSiteK = 0x613, kSiteV = 0x614, kSitePUsed = 0x615, kSiteDs = 0x616, kSiteDsUsed = 0x617, kSiteP = 0x618, kSiteS = 0x621,
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
__device__ __forceinline__ KeyRun run_of(const WinGeo& g, const Item& x) {
  return key_run(g, x.q0, min(x.q0 + kBM, g.S));
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
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_full[s], kComputeWarps);
      mbar_init(&bars->p_used[s], 1);
    }
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->ds_full, kComputeWarps);
    mbar_init(&bars->ds_used, 1);
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
      const KeyRun kr = run_of(g, x);
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
    // and that A and B take next, of the V stage that dP takes next, and tiles issued so far.
    Ring<C::kKSt> k_s, k_q;
    Ring<C::kVSt> v_d;
    Ring<C::kSSt> s_b, p_b;             // the S buffers of S, and of A and B
    uint32_t n_s = 0, n_d = 0, n_q = 0;  // tiles whose S; dP; A and B have been issued
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
    // acc += X K of the tile whose P or dS are in the columns from x on, packed: warpgroup c's 64 keys at 64c
    auto xk = [&](uint32_t acc, uint32_t x, int keys, bool first) {
      const uint64_t kd = dKmn + ((k_q.at * C::kTileBytes) >> 4);
      auto step = [&](int kk) {
        umma_bf16_tmem_a_w(tmem + acc, tmem + x + (kk < 4 ? 0u : 64u) + (kk & 3) * 8, kd + ((kk * 16 * 128) >> 4), kIdKM,
                           (!first || kk > 0) ? 1u : 0u);
      };
      if (keys == kBN) {
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk) step(kk);
      } else {
#pragma unroll 1
        for (int kk = 0; kk < keys / 16; ++kk) step(kk);
      }
    };
    auto issue_s = [&](int keys) -> bool {  // once A has read P from the buffer
      if (!mbar_wait_w(&bars->k_full[k_s.at], k_s.phase, w, kSiteK)) return false;
      if (n_s >= C::kSSt && !mbar_wait_w(&bars->p_used[s_b.at], s_b.phase ^ 1u, w, kSitePUsed)) return false;
      tc_fence_after();
      xt(tmem + col_s(s_b.at), dQ0, dK0 + ((k_s.at * C::kTileBytes) >> 4), keys);
      umma_commit_w(&bars->s_full[s_b.at]);
      ++n_s;
      s_b.next();
      k_s.next();
      issued_any = true;
      return true;
    };
    auto issue_dp = [&](int keys) -> bool {  // dP = dO V^T, once B has read dS from its columns
      if (!mbar_wait_w(&bars->v_full[v_d.at], v_d.phase, w, kSiteV)) return false;
      if (n_d >= 1 && !mbar_wait_w(&bars->ds_used, (n_d - 1) & 1, w, kSiteDsUsed)) return false;
      tc_fence_after();
      xt(tmem + kColDP, dDO0, dV0 + ((v_d.at * C::kTileBytes) >> 4), keys);
      umma_commit_w(&bars->dp_full);
      umma_commit_w(&bars->v_empty[v_d.at]);
      ++n_d;
      v_d.next();
      return true;
    };
    auto issue_a = [&](int keys, bool first) -> bool {  // A += P K
      if (!mbar_wait_w(&bars->p_full[p_b.at], p_b.phase, w, kSiteP)) return false;
      tc_fence_after();
      xk(C::kColA, col_s(p_b.at), keys, first);
      umma_commit_w(&bars->p_used[p_b.at]);
      p_b.next();
      return true;
    };
    auto issue_b = [&](int keys, bool first) -> bool {  // B += dS K
      if (!mbar_wait_w(&bars->ds_full, n_q & 1, w, kSiteDs)) return false;
      tc_fence_after();
      xk(kColB, kColDP, keys, first);
      umma_commit_w(&bars->ds_used);
      umma_commit_w(&bars->k_empty[k_q.at]);
      ++n_q;
      k_q.next();
      return true;
    };
    bool ok = true;
    int idx = blockIdx.x;
    KeyRun r{};
    // the first S and dP of the CTA's item number `item`, behind the last B of the one before: its Q and
    // dO may still be on their way
    auto begin = [&]() -> bool {
      r = run_of(g, item_of(a, idx));
      if (!mbar_wait_w(&bars->q_full, item & 1, w, kSiteQ) || !issue_s(r.width(0))) return false;
      if (r.nt == 1) umma_commit_w(&bars->q_empty);
      if (!mbar_wait_w(&bars->do_full, item & 1, w, kSiteDo) || !issue_dp(r.width(0))) return false;
      if (r.nt == 1) umma_commit_w(&bars->do_empty);
      return true;
    };
    while (ok && idx < a.n_items) {
      if (!(ok = begin())) break;
      const int nt = r.nt;
      if (C::kSSt == 2 && nt > 1) {
        ok = issue_s(r.width(1));
        if (nt == 2) umma_commit_w(&bars->q_empty);
      }
      for (int it = 0; ok && it < nt; ++it) {
        ok = issue_a(r.width(it), it == 0);
        if (ok && it + C::kSSt < nt) {  // S as many tiles ahead as there are buffers
          ok = issue_s(r.width(it + C::kSSt));
          if (it + C::kSSt + 1 == nt) umma_commit_w(&bars->q_empty);
        }
        ok = ok && issue_b(r.width(it), it == 0);
        if (ok && it + 1 < nt) {
          ok = issue_dp(r.width(it + 1));
          if (it + 2 == nt) umma_commit_w(&bars->do_empty);
        }
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
    // ------------------------------------------------------------ compute warps
    const int wg = (warp - 2) >> 2;  // key columns [64 wg, 64 wg + 64)
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const int cbase = wg * 64;
    const float2 sl2 = make_float2(g.scale_log2, g.scale_log2);
    bool ok = true;
    int n = 0, item = 0, idx = blockIdx.x;
    Ring<C::kSSt> s_b;  // the S buffer of the tile
    for (; ok && idx < a.n_items; ++item) {
      const Item x = item_of(a, idx);
      const KeyRun kr = run_of(g, x);
      const int i = x.q0 + row;
      const bool store = i < g.S;
      const size_t tab = (static_cast<size_t>(x.b) * g.Hq + x.h) * a.Lp + i;  // Lp covers the whole tile
      const float nl = a.lse2[tab];  // -inf on padding rows: their P is 0
      const float nd = a.delta[tab];
      const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
      // visible keys of the row: [first, end) and the sinks [lo, sink_end); none past the end
      const int lo = store ? win_lo(g, i) : 1 << 30, end = i + 1;
      const int first = max(lo, i - g.W + 1), sink_end = min(lo + g.ns, i + 1);
      const int w0 = kr.w0 * kBN;
      const int q_last = min(x.q0 + kBM, g.S) - 1;
      const int first_all = max(win_lo(g, q_last), q_last - g.W + 1);
      float2 res2 = make_float2(0.f, 0.f);
      for (int it = 0; it < kr.nt; ++it, ++n) {
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full[s_b.at], s_b.phase, w, kSiteS));
        if (!ok) break;
        tc_fence_after();
        const uint32_t cS = col_s(s_b.at);
        const int k0 = kr.base(it), width = kr.width(it);  // a narrow tile has the first 32 columns at most
        const bool whole = k0 >= first_all && k0 + kBN - 1 <= x.q0;
        auto seen = [&](int c0) {  // (a sink tile ends where the window tiles begin)
          return k0 < w0 ? bits_between(lo - k0, min(sink_end, w0) - k0, c0)
                         : bits_between(first - k0, end - k0, c0) | bits_between(lo - k0, sink_end - k0, c0);
        };
        // Phase 1: P = exp2(s * scale * log2e - LSE * log2e) as bf16 over the S columns; the fp32 values
        // stay in registers for dS.
        float2 pr[32];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c0 = cbase + half * 32;
          if (c0 >= width) break;
          uint32_t rs[32];
          tmem_ld32(trow + cS + c0, rs);
          tmem_ld_wait();
          reg_fence32(rs);
          if (!whole) hide_columns(rs, seen(c0), kMinusInf);
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 y = ffma2(make_float2(__uint_as_float(rs[c]), __uint_as_float(rs[c + 1])), sl2, nl2);
            const float2 pv = make_float2(ex2_approx(y.x), ex2_approx(y.y));  // -inf -> 0
            pr[half * 16 + (c >> 1)] = pv;
            pk[c >> 1] = pack_bf16x2(pv.x, pv.y);
          }
          tmem_st16(trow + cS + cbase + half * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_full[s_b.at]);
        s_b.next();
        // Phase 2: dS' = P (dP - Delta') as bf16 over the dP columns, and its sum
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->dp_full, n & 1, w, kSiteDp));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c0 = cbase + half * 32;
          if (c0 >= width) break;
          uint32_t rp[32];
          tmem_ld32(trow + kColDP + c0, rp);
          tmem_ld_wait();
          reg_fence32(rp);
          // columns past a narrow tile's width hold what was there before (a hidden key's dP is finite: P = 0 hides it)
          if (width != kBN) hide_columns(rp, seen(c0), 0u);
          uint32_t dk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 ds = fmul2(pr[half * 16 + (c >> 1)],
                                    fadd2(make_float2(__uint_as_float(rp[c]), __uint_as_float(rp[c + 1])), nd2));
            res2 = fadd2(res2, ds);
            dk[c >> 1] = pack_bf16x2(ds.x, ds.y);
          }
          tmem_st16(trow + kColDP + cbase + half * 16, dk);
        }
        if (it + 1 == kr.nt) sRes[(item & 1) * 256 + wg * 128 + row] = res2.x + res2.y;
        tmem_st_wait();
        tc_fence_before();
        if (it + 1 == kr.nt) mbar_arrive_warp(&bars->r_full);
        mbar_arrive_warp(&bars->ds_full);
      }
      // ------------------------------------------------------------ epilogue: the table's row, dQ rows
      float res = 0.f;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->r_full, item & 1, w, kSiteRes));
      if (ok) {
        const float* s = sRes + (item & 1) * 256 + row;
        res = s[0] + s[128];
        if (store && wg == 0) a.delta[tab] = nd - res;  // -(Delta' + r): both warpgroups have read it
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->ds_used, (n - 1) & 1, w, kSiteEpi));
      }
      if (ok) {
        tc_fence_after();
        __nv_bfloat16* const dq0 = a.dq + (static_cast<size_t>(x.b) * g.S * g.Hq + x.h) * D;  // row 0 of the head
        const float2 nr2 = make_float2(-res, -res), sc2 = make_float2(g.scale, g.scale);
#pragma unroll 1
        for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
          uint32_t o[32], p[32], pk[16];
          tmem_ld32(trow + kColB + c0, o);
          tmem_ld32(trow + C::kColA + c0, p);
          tmem_ld_wait();
          reg_fence32(o);
          reg_fence32(p);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 y = fmul2(ffma2(make_float2(__uint_as_float(p[c]), __uint_as_float(p[c + 1])), nr2,
                                         make_float2(__uint_as_float(o[c]), __uint_as_float(o[c + 1]))), sc2);
            pk[c >> 1] = pack_bf16x2(y.x, y.y);
          }
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
