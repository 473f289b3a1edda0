// usp_window_bwd.cu -- backward of sliding-window attention with sinks, the
// key-major half (dK, dV) on sm_100a.
//
//   P_ij = exp(scale q_i.k_j - LSE_i), dP = dO V^T, dS = P (dP - Delta),
//   dK = scale dS^T Q, dV = P^T dO, summed over the query heads of a group,
// over the query tiles in the band of each key tile (usp_window.cuh). Rows of
// sinks add what the far kernel made of the queries behind that band.
//
// A persistent CTA (one per SM, 320 threads) takes work items: one 128-key tile
// of one kv head, walked by steps (query head of the group, query tile):
//   warp 0      TMA producer: K, V per item; Q, dO and the row tables per step (2 stages)
//   warp 1      UMMA issuer: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   warps 2..9  two warpgroups of 64 query columns; thread = key row
// TMEM: S^T / P^T [0,128), dP^T / dS^T [128,256), dV at 256, dK at 384. The steps
// of all items of a CTA form one stream: the next item's S^T and dP^T are issued
// as soon as this item's last products have read those columns, so they overlap
// its epilogue; its dV and dK cannot overtake the epilogue's reads because they
// wait for P^T and dS^T, which the same warps write after them.
//
// Bound by the chain S^T -> P^T -> dV -> S^T (1.8 us per step; the four products take
// 1.1) and by about 5 us per item (64 KB of stores among them). B=1 S=32768 H=16/4 D=128
// W=2048, 4 sinks: 870 us, 1227 TFLOP/s (8 D flops per visible pair).
#include <math.h>

#include "usp_ptx.cuh"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kThreads = 320;
constexpr int kComputeWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 256, kColDK = 384;
// Key pairs (of every 8) whose exp2 runs on the FMA pipe: backward of 8192 tokens, 16/4 heads, window 2048,
// with 0, 2, 3, 4: 434, 428, 429, 434 us (D=64: 371, 363, 362, 364).
constexpr int kPolyPer8 = 2;

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanelBytes = 128 * 128;
  static constexpr int kTileBytes = kPanels * kPanelBytes;
  static constexpr int kStages = 2;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTileBytes;
  static constexpr int kOffQ = 2 * kTileBytes;
  static constexpr int kOffDO = kOffQ + kStages * kTileBytes;
  static constexpr int kOffRow = kOffDO + kStages * kTileBytes;  // per stage: -LSE*log2e [128], -Delta [128]
  static constexpr int kOffBar = kOffRow + kStages * 1024;
  static constexpr int kSmemBytes = kOffBar + 256;
};

struct Args {
  WinGeo g;
  ItemDiv div;
  const float* lse2;
  const float* delta;
  int Lp;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float* far_part;  // see WinLaunch
  int far_chunk;
  const float* far_sum;
  int n_items;
  int* status;
  unsigned long long wait_ns;
};

struct Bars {
  uint64_t kv_full, kv_empty;
  uint64_t qd_full[2], qd_empty[2];
  uint64_t s_full, dp_full, p_full, ds_full, p_used, ds_used, drain;
  uint64_t far_full;  // the runs of the item's far sinks have been added up
  ItemFeed feed;
  uint32_t tmem_base;
  int abort_flag;
};

enum : int {
  kSiteKvEmpty = 0x501, kSiteQdEmpty = 0x502, kSiteKv = 0x511, kSiteQd = 0x512, kSiteP = 0x513, kSitePUsed = 0x514,
  kSiteDs = 0x515, kSiteDsUsed = 0x516, kSiteS = 0x521, kSiteDp = 0x522, kSiteQdC = 0x523, kSiteEpi = 0x524,
  kSiteFar = 0x525,
  kSiteFeed = 0x531,
  kSiteAlign = 0x5FF
};

struct Item {
  int b, gl, n;   // batch, kv head, key tile
  int n_m, steps; // query tiles n .. n + n_m - 1 of every head of the group
};
__device__ __forceinline__ Item item_of(const Args& a, int idx) {
  const WinGeo& g = a.g;
  // the first keys of every head first (the causally heaviest), the heads side by side
  const ItemParts p = item_parts(a.div, idx);
  Item x;
  x.gl = p.head;
  x.b = p.b;
  x.n = p.rest;
  x.n_m = last_qtile(g, x.n) - x.n + 1;
  x.steps = x.n_m * g.G;
  return x;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    window_dkdv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                       const Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_addr(smem) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicCAS(a.status, 0, kSiteAlign);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);
  static_assert(sizeof(Bars) <= 256, "barrier block");
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sDO = smem + C::kOffDO;
  float* sRow = reinterpret_cast<float*>(smem + C::kOffRow);
  const WinGeo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    feed_init(bars->feed, 1 + kComputeWarps);
    mbar_init(&bars->kv_full, 1);
    mbar_init(&bars->kv_empty, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->qd_full[s], 1);
      mbar_init(&bars->qd_empty[s], 1);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->p_full, kComputeWarps);
    mbar_init(&bars->ds_full, kComputeWarps);
    mbar_init(&bars->far_full, kComputeWarps);
    mbar_init(&bars->p_used, 1);
    mbar_init(&bars->ds_used, 1);
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
    int issued = 0, n_kv = 0;
    bool ok = true;
    int idx = blockIdx.x, next = 0;
    for (int item = 1; ok && idx < a.n_items; ++item, idx = next) {
      const Item x = item_of(a, idx);
      for (int k = 0, m = 0, h = x.gl * g.G; k < x.steps; ++k) {  // m: query tile of head h
        const int s = issued % C::kStages;
        const int q0 = (x.n + m) * kBM;
        if (issued >= C::kStages && !mbar_wait_w(&bars->qd_empty[s], ((issued / C::kStages) - 1) & 1, w, kSiteQdEmpty)) {
          ok = false;
          break;
        }
        mbar_expect_tx_w(&bars->qd_full[s], 2 * C::kTileBytes + 1024);
        for (int p = 0; p < C::kPanels; ++p) {
          tma_load_4d_w(&tm_q, &bars->qd_full[s], sQ + s * C::kTileBytes + p * C::kPanelBytes, p * 64, h, q0, x.b);
          tma_load_4d_w(&tm_do, &bars->qd_full[s], sDO + s * C::kTileBytes + p * C::kPanelBytes, p * 64, h, q0, x.b);
        }
        const size_t rowbase = (static_cast<size_t>(x.b) * g.Hq + h) * a.Lp + q0;
        bulk_load_1d_w(sRow + s * 256, a.lse2 + rowbase, 512, &bars->qd_full[s]);
        bulk_load_1d_w(sRow + s * 256 + 128, a.delta + rowbase, 512, &bars->qd_full[s]);
        ++issued;
        if (++m == x.n_m) m = 0, ++h;
        if (k == 0) {  // K, V behind the first Q, dO: their buffers free last
          if (n_kv >= 1 && !mbar_wait_w(&bars->kv_empty, (n_kv - 1) & 1, w, kSiteKvEmpty)) {
            ok = false;
            break;
          }
          mbar_expect_tx_w(&bars->kv_full, 2 * C::kTileBytes);
          for (int p = 0; p < C::kPanels; ++p) {
            tma_load_4d_w(&tm_k, &bars->kv_full, sK + p * C::kPanelBytes, p * 64, x.gl, x.n * kBN, x.b);
            tma_load_4d_w(&tm_v, &bars->kv_full, sV + p * C::kPanelBytes, p * 64, x.gl, x.n * kBN, x.b);
          }
          ++n_kv;
          if (!feed_give(bars->feed, item, a.status + kCounterDkdv, w, kSiteFeed, next)) {
            ok = false;
            break;
          }
        }
      }
    }
    // Every copy this warp started lands before the CTA ends, whoever may have given up since.
    if (n_kv > 0) mbar_wait_drain(&bars->kv_full, (n_kv - 1) & 1);
    for (int it = issued - C::kStages < 0 ? 0 : issued - C::kStages; it < issued; ++it)
      mbar_wait_drain(&bars->qd_full[it % C::kStages], (it / C::kStages) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ UMMA issuer
    constexpr uint32_t kIdSS = idesc_bf16_f32(128, 128, 0, 0);  // both K-major
    constexpr uint32_t kIdKM = idesc_bf16_f32(128, D, 0, 1);    // A K-major (TMEM), B MN-major
    const uint64_t dK0 = sdesc_sw128(smem_addr(sK), 16, 1024), dV0 = sdesc_sw128(smem_addr(sV), 16, 1024);
    const uint64_t dQ0 = sdesc_sw128(smem_addr(sQ), 16, 1024), dDO0 = sdesc_sw128(smem_addr(sDO), 16, 1024);
    const uint64_t dQmn = sdesc_sw128(smem_addr(sQ), C::kPanelBytes, 1024);
    const uint64_t dDOmn = sdesc_sw128(smem_addr(sDO), C::kPanelBytes, 1024);
    auto issue_xt = [&](uint32_t col, uint64_t a0, uint64_t b0, int s) {  // X^T = A B_s^T
      const uint64_t bd = b0 + ((s * C::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::kPanelBytes + (kk & 3) * 32) >> 4;
        umma_bf16_w(tmem + col, a0 + off, bd + off, kIdSS, kk > 0 ? 1u : 0u);
      }
    };
    auto issue_acc = [&](uint32_t acc, uint32_t xcol, uint64_t y0, int s, bool first) {  // acc += X^T Y_s
      const uint64_t yd = y0 + ((s * C::kTileBytes) >> 4);
#pragma unroll
      for (int kk = 0; kk < kBM / 16; ++kk) {
        const uint32_t pcol = (kk < 4 ? 0u : 64u) + (kk & 3) * 8;
        umma_bf16_tmem_a_w(tmem + acc, tmem + xcol + pcol, yd + ((kk * 16 * 128) >> 4), kIdKM,
                           (!first || kk > 0) ? 1u : 0u);
      }
    };
    bool ok = true, issued_any = false;
    int idx = blockIdx.x;
    if (idx < a.n_items) {
      int steps = item_of(a, idx).steps, it = 0, item = 0;
      ok = mbar_wait_w(&bars->kv_full, 0, w, kSiteKv) && mbar_wait_w(&bars->qd_full[0], 0, w, kSiteQd);
      if (ok) {
        tc_fence_after();
        issue_xt(kColS, dK0, dQ0, 0);
        umma_commit_w(&bars->s_full);
        issue_xt(kColDP, dV0, dDO0, 0);
        umma_commit_w(&bars->dp_full);
        if (steps == 1) umma_commit_w(&bars->kv_empty);
        issued_any = true;
      }
      for (int k = 0; ok; ++k) {  // k: step of the CTA's stream, it: of the item
        const int s = k % C::kStages, s1 = (k + 1) % C::kStages;
        const bool last = it + 1 == steps;
        if (last && !feed_take(bars->feed, item + 1, w, kSiteFeed, idx)) { ok = false; break; }
        const bool more = !last || idx < a.n_items;
        const int next_steps = last && more ? item_of(a, idx).steps : steps;
        if (!mbar_wait_w(&bars->p_full, k & 1, w, kSiteP)) { ok = false; break; }
        tc_fence_after();
        issue_acc(kColDV, kColS, dDOmn, s, it == 0);  // dV += P^T dO
        umma_commit_w(&bars->p_used);
        auto next_s = [&]() -> bool {  // S^T of the next step once dV has read P^T from its columns
          if (!mbar_wait_w(&bars->qd_full[s1], ((k + 1) / C::kStages) & 1, w, kSiteQd)) return false;
          if (!mbar_wait_w(&bars->p_used, k & 1, w, kSitePUsed)) return false;
          tc_fence_after();
          issue_xt(kColS, dK0, dQ0, s1);
          umma_commit_w(&bars->s_full);
          return true;
        };
        if (!last && !next_s()) { ok = false; break; }
        if (!mbar_wait_w(&bars->ds_full, k & 1, w, kSiteDs)) { ok = false; break; }
        tc_fence_after();
        issue_acc(kColDK, kColDP, dQmn, s, it == 0);  // dK += dS^T Q
        umma_commit_w(&bars->ds_used);
        umma_commit_w(&bars->qd_empty[s]);
        if (!more) break;
        if (last && !(mbar_wait_w(&bars->kv_full, (item + 1) & 1, w, kSiteKv) && next_s())) { ok = false; break; }
        // dP^T of the next step overwrites the dS^T that dK reads
        if (!mbar_wait_w(&bars->ds_used, k & 1, w, kSiteDsUsed)) { ok = false; break; }
        tc_fence_after();
        issue_xt(kColDP, dV0, dDO0, s1);
        umma_commit_w(&bars->dp_full);
        if (last ? next_steps == 1 : it + 2 == steps) umma_commit_w(&bars->kv_empty);
        if (last) {
          steps = next_steps;
          it = 0;
          ++item;
        } else {
          ++it;
        }
      }
    }
    if (issued_any) {  // the products too: the warps that wait for the last ones may have given up
      umma_commit_w(&bars->drain);
      mbar_wait_drain(&bars->drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ compute warps
    const int wg = (warp - 2) >> 2;  // query columns [64 wg, 64 wg + 64)
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const int cbase = wg * 64;
    const float2 sl2 = make_float2(g.scale_log2, g.scale_log2);
    bool ok = true;
    int k = 0, idx = blockIdx.x, n_far = 0;
    for (int item = 1; ok && idx < a.n_items; ++item) {
      const Item x = item_of(a, idx);
      const int k0 = x.n * kBN, j = k0 + row;
      const bool store = j < g.S;
      // queries that see the key: [j, q_end); none past the end of the sequence
      int lo = 0, hi = 0, q_end = 0, sink = -1;
      if (store) {
        win_span(g, j, lo, hi);
        if (j - lo < g.ns) sink = j - lo;
        q_end = sink >= 0 ? hi : min(hi, j + g.W);
      }
      // the last query row that sees every key of the tile from the diagonal on
      int lo0, hi0;
      win_span(g, k0, lo0, hi0);
      const int q_all = min(hi0, k0 + g.W);
      // The far queries' part of the sinks' gradients: of the document of the tile's last key (any other
      // ends inside the tile), by runs f0 .. f1 whose first tiles are multiples of the chunk or the
      // document's first tile, from the first query tile outside the key tile's band on. The runs are added
      // up, over the first one, while the item's first tiles are on their way.
      const float* far = nullptr;
      bool far_wait = false;
      if (a.far_part) {
        const int jl = min(k0 + kBN, g.S) - 1;
        int lol, hil;
        win_span(g, jl, lol, hil);
        const int mf = x.n + x.n_m, me = (hil - 1) / kBM + 1, s0 = max(k0 - lol, 0), s1 = min(g.ns, jl + 1 - lol);
        if (mf < me && s0 < s1) {
          const size_t bh = static_cast<size_t>(x.b) * g.Hkv + x.gl, run = static_cast<size_t>(g.ns) * (2 * D);
          if (a.far_sum) {
            const int d = g.cu ? doc_of(g.cu, g.n_docs, jl) : 0;
            far = a.far_sum + (bh * g.n_docs + d) * run;
          } else {
            const int f0 = mf / a.far_chunk, f1 = (me - 1) / a.far_chunk, md = (lol + kBM - 1) / kBM;
            float* const base = a.far_part + bh * g.n_tiles * run;
            float* const sum = base + max(f0 * a.far_chunk, md) * run;
            far = sum;
            for (int u = s0 * (2 * D) + (threadIdx.x - 64) * 4; u < s1 * (2 * D); u += 32 * kComputeWarps * 4) {
              float4 t = *reinterpret_cast<const float4*>(sum + u);
#pragma unroll 8
              for (int y = f0 + 1; y <= f1; ++y) {
                const float4 p = *reinterpret_cast<const float4*>(base + y * a.far_chunk * run + u);
                t.x += p.x;
                t.y += p.y;
                t.z += p.z;
                t.w += p.w;
              }
              *reinterpret_cast<float4*>(sum + u) = t;
            }
            mbar_arrive_warp(&bars->far_full);
            far_wait = true;
          }
        }
      }
      for (int it = 0, m = 0; it < x.steps; ++it, ++k) {
        const int s = k % C::kStages;
        const int q0 = (x.n + m) * kBM;
        if (++m == x.n_m) m = 0;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->qd_full[s], (k / C::kStages) & 1, w, kSiteQdC));
        if (!ok) break;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->s_full, k & 1, w, kSiteS));
        if (!ok) break;
        tc_fence_after();
        const float* nlse2 = sRow + s * 256;
        const float* ndl = nlse2 + 128;
        const bool whole = q0 >= k0 + kBN - 1 && min(q0 + kBM, g.S) <= q_all && k0 + kBN <= g.S;
        float2 pr[32];
        // Phase 1 (while the tensor core computes dP^T): P^T = exp2(s*scale*log2e - LSE*log2e)
        // as bf16 over the S^T columns; the fp32 values stay in registers for dS.
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c0 = cbase + half * 32;
          uint32_t rs[32];
          tmem_ld32(trow + kColS + c0, rs);
          tmem_ld_wait();
          reg_fence32(rs);
          if (!whole) {
            hide_columns(rs, bits_between(j - q0, q_end - q0, c0), kMinusInf);
          }
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 nl = *reinterpret_cast<const float2*>(nlse2 + c0 + c);
            const float2 y = ffma2(make_float2(__uint_as_float(rs[c]), __uint_as_float(rs[c + 1])), sl2, nl);
            // a -inf score gets ~2^-125 from the polynomial: a weight no dK/dV sum resolves
            const float2 pv =
                ((c >> 1) % 8 < kPolyPer8) ? exp2_poly2(y) : make_float2(ex2_approx(y.x), ex2_approx(y.y));
            pr[half * 16 + (c >> 1)] = pv;
            pk[c >> 1] = pack_bf16x2(pv.x, pv.y);
          }
          tmem_st16(trow + kColS + cbase + half * 16, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars->p_full);
        // Phase 2 (while the tensor core computes dV): dS^T = P^T o (dP^T - Delta) as bf16 over
        // the dP^T columns (the softmax scale is applied to dK at the end).
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->dp_full, k & 1, w, kSiteDp));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c0 = cbase + half * 32;
          uint32_t rp[32];
          tmem_ld32(trow + kColDP + c0, rp);
          tmem_ld_wait();
          reg_fence32(rp);
          uint32_t dk[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 nd = *reinterpret_cast<const float2*>(ndl + c0 + c);
            const float2 ds = fmul2(pr[half * 16 + (c >> 1)],
                                    fadd2(make_float2(__uint_as_float(rp[c]), __uint_as_float(rp[c + 1])), nd));
            dk[c >> 1] = pack_bf16x2(ds.x, ds.y);
          }
          tmem_st16(trow + kColDP + cbase + half * 16, dk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive_warp(&bars->ds_full);
      }
      // ------------------------------------------------------------ dK, dV epilogue
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&bars->ds_used, (k - 1) & 1, w, kSiteEpi));
      if (ok && far_wait) ok = __all_sync(0xffffffffu, mbar_wait(&bars->far_full, n_far++ & 1, w, kSiteFar));
      if (ok) {
        tc_fence_after();
        const size_t kv0 = (static_cast<size_t>(x.b) * g.S * g.Hkv + x.gl) * D;  // row 0 of the kv head
        // a row of far sinks: dK, then dV (a document that ends inside the tile has none)
        const bool add = far && sink >= 0 && hi > (x.n + x.n_m) * kBM;
        if (add) far += static_cast<size_t>(sink) * (2 * D);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {  // dK, then dV
          const uint32_t col = half == 0 ? kColDK : kColDV;
          const float f = half == 0 ? g.scale : 1.0f;
          __nv_bfloat16* const dst = (half == 0 ? a.dk : a.dv) + kv0;
#pragma unroll 1
          for (int c0 = wg * (D / 2); c0 < (wg + 1) * (D / 2); c0 += 32) {
            uint32_t r[32], pk[16];
            tmem_ld32(trow + col + c0, r);
            tmem_ld_wait();
            reg_fence32(r);
            if (add) {
              const float4* p = reinterpret_cast<const float4*>(far + half * D + c0);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const float4 f4 = p[c];
                r[4 * c] = __float_as_uint(__uint_as_float(r[4 * c]) + f4.x);
                r[4 * c + 1] = __float_as_uint(__uint_as_float(r[4 * c + 1]) + f4.y);
                r[4 * c + 2] = __float_as_uint(__uint_as_float(r[4 * c + 2]) + f4.z);
                r[4 * c + 3] = __float_as_uint(__uint_as_float(r[4 * c + 3]) + f4.w);
              }
            }
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              pk[c >> 1] = pack_bf16x2(__uint_as_float(r[c]) * f, __uint_as_float(r[c + 1]) * f);
            store_rows32(dst, static_cast<size_t>(g.Hkv) * D, k0 + wq * 32, g.S, c0, pk);
          }
        }
        ok = feed_take(bars->feed, item, w, kSiteFeed, idx);
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
      cudaFuncSetAttribute(window_dkdv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  Args a{};
  a.g = L.g;
  a.div = make_item_div(L.g.Hkv, L.g.B);
  a.lse2 = L.lse2;
  a.delta = L.delta;
  a.Lp = L.Lp;
  a.dk = static_cast<__nv_bfloat16*>(L.dk);
  a.dv = static_cast<__nv_bfloat16*>(L.dv);
  a.far_part = L.far_part;
  a.far_chunk = L.far_chunk;
  a.far_sum = L.far_sum;
  a.status = L.status;
  a.wait_ns = L.wait_ns;
  const long long items = static_cast<long long>(L.g.n_tiles) * L.g.Hkv * L.g.B;
  if (items > 0x3FFFFFFFLL) return cudaErrorInvalidConfiguration;
  a.n_items = static_cast<int>(items);
  const int sms = sm_count();
  const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
  return launch_behind(window_dkdv_kernel<D>, dim3(grid), kThreads, C::kSmemBytes, stream, L.tm_q, L.tm_k, L.tm_v,
                       L.tm_do, a);
}

}  // namespace

cudaError_t launch_window_dkdv(const WinLaunch& L, cudaStream_t stream) {
  return L.D == 128 ? launch_d<128>(L, stream) : L.D == 64 ? launch_d<64>(L, stream) : cudaErrorInvalidValue;
}

}  // namespace usp
