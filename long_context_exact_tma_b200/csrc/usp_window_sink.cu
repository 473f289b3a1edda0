// usp_window_sink.cu -- backward of sliding-window attention with sinks: dK and
// dV of the sinks from the far queries, those whose tile lies behind the band of
// the sink's key tile (usp_window.cuh) and that the key-major kernel so never
// visits. A query tile has far sinks of one document only, that of its first row:
// any other document with rows in the tile starts inside it.
//
//   dV_s = sum_i P_is dO_i,  dK_s / scale = sum_i P_is (dO_i.v_s - Delta_i) Q_i
//
// A few keys against every query is bound by reading Q and dO once, so the
// products run on the warp-level 16x8x16 matrix instruction (a 128-key tensor tile
// would hold 4 keys in 128): a warp has 8 sinks, always the instruction's 8 columns:
// S [rows x sinks] and dP with K, V fragments that stay in registers, then dV^T and
// dK^T [D x sinks], over 16 query rows at a time. A CTA takes a run of query tiles of
// one document and kv head and streams its rows, tile by tile and head by head; every
// warp fetches 16 of a tile's rows through its own ring of cp.async buffers. With up
// to 8 sinks it also works on just these; with more, two, four or all eight warps have
// a group of 8 sinks each and work on each other's rows, so that the rows are read
// once for 64 sinks and not for 8 (backward of 8192 tokens, 16/4 heads, window 128,
// 32 sinks: 170 -> 150 us, 128 sinks: 319 -> 255). The warps' fp32 sums are
// joined in a fixed order and written per run; the key-major kernel's items add the
// runs of their sinks up in order, or, where they are many, take their sums, which a
// second kernel makes in a fixed order. No atomics: the result does not depend on
// scheduling.
//
// B=1 S=32768 H=16/4 D=128, 4 sinks: 44 us, 6.2 TB/s of Q and dO.
#include <math.h>

#include "usp_mma.cuh"
#include "usp_ptx.cuh"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kGroup = 8;   // sinks at a time
constexpr int kStages = 3;  // (tile, head) steps in flight
constexpr long long kFarOwn = 1 << 16;  // floats of runs that the key-major kernel adds up itself

struct FarArgs {
  WinGeo g;
  const __nv_bfloat16 *q, *k, *v, *dO;
  const float *lse2, *delta;
  int Lp;
  int chunk;  // tiles of a CTA: its runs start at multiples of it and where a document's tiles start
  int n_chunks;
  float* part;  // [b][kv head][first tile of the run][sink][2][D]
  float* sum;
};

template <int D>
struct FarCfg {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  static constexpr int kHalf = 16 * kRowBytes;
  static constexpr int kStageBytes = 2 * kHalf + 128;  // a warp's 16 rows of Q, of dO, and of the two tables
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kSmemBytes = kWarps * kWarpBytes;
  static_assert(kGroup * 2 * D * 4 <= kWarpBytes, "a warp's sums fit over its buffers");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

template <int D>
__device__ __forceinline__ uint32_t at(int row, int chunk) {  // byte of a chunk: swizzled against bank conflicts
  return row * FarCfg<D>::kRowBytes + ((chunk ^ (row & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) far_kernel(const FarArgs a) {
  using C = FarCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const WinGeo& g = a.g;
  const int cx = blockIdx.x % a.n_chunks, gl = blockIdx.x / a.n_chunks % g.Hkv, b = blockIdx.x / a.n_chunks / g.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_addr(smem), mine = base + warp * C::kWarpBytes;
  const int m_end = min((cx + 1) * a.chunk, g.n_tiles);
  let_next_start();
  wait_for_previous();

  for (int m0 = cx * a.chunk, m1; m0 < m_end; m0 = m1) {
    // the run [m0, m1): tiles whose first rows are of one document [lo, hi)
    int lo, hi;
    win_span(g, m0 * kBM, lo, hi);
    m1 = min(m_end, (hi - 1) / kBM + 1);
    const int n_sinks = min(g.ns, hi - lo);
    // band ends grow with the key: tiles from here on have far sinks
    const int mf = max(m0, last_qtile(g, lo / kBN) + 1);
    if (mf >= m1) continue;
    float* out = a.part + ((static_cast<size_t>(b) * g.Hkv + gl) * g.n_tiles + m0) * g.ns * (2 * D);
    const int steps = (m1 - mf) * g.G;

    // `team` neighbouring warps work on each other's rows, each for its own 8 sinks
    const int team = n_sinks <= kGroup ? 1 : n_sinks <= 2 * kGroup ? 2 : n_sinks <= 4 * kGroup ? 4 : 8;
    const int part = warp / team, member = warp - part * team;
    auto team_sync = [&]() {
      if (team == 1)
        __syncwarp();
      else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + part), "r"(32 * team) : "memory");
    };

    for (int sb = 0; sb < n_sinks; sb += kGroup * team) {
      const int s0 = sb + member * kGroup;  // this warp's sinks
      auto fetch = [&](int st) {
        if (st < steps) {
          const int h = gl * g.G + st % g.G, row0 = (mf + st / g.G) * kBM + warp * 16;
          const uint32_t dst = mine + (st % kStages) * C::kStageBytes;
          if (lane < 8) {
            const float* tab = (lane < 4 ? a.lse2 : a.delta) + (static_cast<size_t>(b) * g.Hq + h) * a.Lp + row0;
            cp_async16(dst + 2 * C::kHalf + lane * 16, tab + (lane & 3) * 4, true);
          }
#pragma unroll
          for (int y = 0; y < 16 * C::kChunks / 32; ++y) {
            const int r = y * (32 / C::kChunks) + lane / C::kChunks, ch = lane % C::kChunks;
            const bool ok = row0 + r < g.S;
            const size_t e = ((static_cast<size_t>(b) * g.S + (ok ? row0 + r : 0)) * g.Hq + h) * D + ch * 8;
            cp_async16(dst + at<D>(r, ch), a.q + e, ok);
            cp_async16(dst + C::kHalf + at<D>(r, ch), a.dO + e, ok);
          }
        }
        cp_async_commit();
      };
      for (int st = 0; st < kStages - 1; ++st) fetch(st);
      // B fragments of K and V: lane (g = lane/4, c = lane%4) holds elements 2c, 2c+1 and 2c+8, 2c+9 of
      // every 16 of sink g's row
      uint32_t kb[D / 16][2], vb[D / 16][2];
      {
        const int s = s0 + (lane >> 2);
        const size_t e = ((static_cast<size_t>(b) * g.S + lo + (s < n_sinks ? s : 0)) * g.Hkv + gl) * D + (lane & 3) * 2;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            kb[kk][y] = s < n_sinks ? *reinterpret_cast<const uint32_t*>(a.k + e + kk * 16 + y * 8) : 0u;
            vb[kk][y] = s < n_sinks ? *reinterpret_cast<const uint32_t*>(a.v + e + kk * 16 + y * 8) : 0u;
          }
      }
      // first far tile of this lane's two sink columns
      int far_from[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s = s0 + (lane & 3) * 2 + e;
        far_from[e] = s < n_sinks ? last_qtile(g, (lo + s) / kBN) + 1 : INT_MAX;
      }
      float av[D / 16][4], ak[D / 16][4];  // dV^T, dK^T: 16 elements x 8 sinks each
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) av[x][e] = ak[x][e] = 0.f;

      for (int st = 0; st < steps; ++st) {
        cp_async_wait<kStages - 2>();
        team_sync();  // the step's rows are there, and every warp is done with the stage that is filled next
        fetch(st + kStages - 1);
        const int m = mf + st / g.G;
        for (int w = part * team; w < part * team + team && s0 < n_sinks; ++w) {  // the rows that warp w has fetched
          const uint32_t sq = base + w * C::kWarpBytes + (st % kStages) * C::kStageBytes, sd = sq + C::kHalf;
          const float* tab = reinterpret_cast<const float*>(smem + (sd + C::kHalf - base)) + (lane >> 2);
          const int i0 = m * kBM + w * 16 + (lane >> 2);
          const float nl[2] = {tab[0], tab[8]}, nd[2] = {tab[16], tab[24]};
          // S = Q K^T, dP = dO V^T of 16 rows and 8 sinks, even and odd steps apart
          float sc[2][4] = {}, dp[2][4] = {};
          const int ar = lane & 15, ac = lane >> 4;  // rows and half chunks of the fragments
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t qa[4], da[4];
            ldsm_x4(qa, sq + at<D>(ar, 2 * kk + ac));
            ldsm_x4(da, sd + at<D>(ar, 2 * kk + ac));
            mma_16816(sc[kk & 1], qa, kb[kk][0], kb[kk][1]);
            mma_16816(dp[kk & 1], da, vb[kk][0], vb[kk][1]);
          }
          uint32_t pt[2], dt[2];  // P, dS as B fragments: rows x sinks, rows 0..7 and 8..15
#pragma unroll
          for (int half = 0; half < 2; ++half) {   // rows i0, i0 + 8
            const bool live = i0 + half * 8 < hi;  // a row of the same document (hi <= S)
            float p[2], ds[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float sv = sc[0][half * 2 + e] + sc[1][half * 2 + e], dv = dp[0][half * 2 + e] + dp[1][half * 2 + e];
              p[e] = live && m >= far_from[e] ? ex2_approx(sv * g.scale_log2 + nl[half]) : 0.f;
              ds[e] = p[e] * (dv + nd[half]);
            }
            // bf16 operands, as P and dS have in the key-major kernel; sums stay fp32
            pt[half] = mov_trans(pack_bf16x2(p[0], p[1]));
            dt[half] = mov_trans(pack_bf16x2(ds[0], ds[1]));
          }
          // A fragments of dO^T, Q^T: the transposed 8x8 blocks, element octets by row octets
          const int tr = (lane & 7) + ((lane >> 4) << 3), tc = (lane >> 3) & 1;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            uint32_t da[4], qa[4];
            ldsm_x4_trans(da, sd + at<D>(tr, 2 * x + tc));
            ldsm_x4_trans(qa, sq + at<D>(tr, 2 * x + tc));
            mma_16816(av[x], da, pt[0], pt[1]);
            mma_16816(ak[x], qa, dt[0], dt[1]);
          }
        }
      }
      cp_async_wait<0>();
      __syncthreads();  // every warp is done with the buffers
      // the warps' sums over their own buffers, then added warp by warp
      float* mysum = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = (lane & 3) * 2 + (e & 1), d = x * 16 + (lane >> 2) + (e >> 1) * 8;
          mysum[(s * 2 + 0) * D + d] = ak[x][e];
          mysum[(s * 2 + 1) * D + d] = av[x][e];
        }
      __syncthreads();
      const int n = min(kGroup * team, n_sinks - sb) * 2 * D;
      for (int x = tid; x < n; x += kThreads) {
        constexpr int kOne = kGroup * 2 * D;  // a warp's sums
        const int who = x / kOne;
        float t = 0.f;
        for (int y = who; y < kWarps; y += team) t += reinterpret_cast<const float*>(smem + y * C::kWarpBytes)[x - who * kOne];
        out[static_cast<size_t>(sb) * 2 * D + x] = t;
      }
      __syncthreads();  // read before the buffers are filled again
    }
  }
  cp_async_wait<0>();
}

// sum[b][gl][d][s] = the partials of sink s of document d over the runs with far
// tiles, in four interleaved series added in order.
template <int D>
__global__ void __launch_bounds__(8 * D) far_sum_kernel(const FarArgs a) {
  __shared__ float series[4][2 * D];
  const WinGeo& g = a.g;
  const int s = blockIdx.x % g.ns, d = blockIdx.x / g.ns % g.n_docs;
  const int gl = blockIdx.x / g.ns / g.n_docs % g.Hkv, b = blockIdx.x / g.ns / g.n_docs / g.Hkv;
  let_next_start();
  wait_for_previous();
  int lo = 0, hi = g.S;
  if (g.cu) {
    lo = min(max(__ldg(g.cu + d), 0), g.S);
    hi = min(max(__ldg(g.cu + d + 1), lo), g.S);
  }
  if (lo + s >= hi) return;  // no such key: nothing reads its sum
  // far tiles of the sink: [mf, me); its document's tiles start at md
  const int mf = last_qtile(g, (lo + s) / kBN) + 1, me = (hi - 1) / kBM + 1, md = (lo + kBM - 1) / kBM;
  const int col = threadIdx.x % (2 * D), y = threadIdx.x / (2 * D);
  const size_t tile = static_cast<size_t>(g.ns) * 2 * D;
  const float* p = a.part + (static_cast<size_t>(b) * g.Hkv + gl) * g.n_tiles * tile + static_cast<size_t>(s) * 2 * D + col;
  float t = 0.f;
  if (mf < me) {
    const int c0 = mf / a.chunk, c1 = (me - 1) / a.chunk;
#pragma unroll 8
    for (int c = c0 + y; c <= c1; c += 4) t += p[static_cast<size_t>(max(c * a.chunk, md)) * tile];
  }
  series[y][col] = t;
  __syncthreads();
  if (y == 0)
    a.sum[(((static_cast<size_t>(b) * g.Hkv + gl) * g.n_docs + d) * g.ns + s) * (2 * D) + col] =
        (series[0][col] + series[1][col]) + (series[2][col] + series[3][col]);
}

template <int D>
cudaError_t launch_d(const WinLaunch& L, cudaStream_t stream) {
  using C = FarCfg<D>;
  cudaError_t e = cudaFuncSetAttribute(far_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  FarArgs a{};
  a.g = L.g;
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.k = static_cast<const __nv_bfloat16*>(L.k);
  a.v = static_cast<const __nv_bfloat16*>(L.v);
  a.dO = static_cast<const __nv_bfloat16*>(L.dO);
  a.lse2 = L.lse2;
  a.delta = L.delta;
  a.Lp = L.Lp;
  a.part = L.far_part;
  a.chunk = L.far_chunk;
  a.n_chunks = (L.g.n_tiles + a.chunk - 1) / a.chunk;
  const long long n_far = static_cast<long long>(L.g.Hkv) * L.g.B * a.n_chunks;
  if (n_far > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  e = launch_behind(far_kernel<D>, dim3(static_cast<unsigned>(n_far)), kThreads, C::kSmemBytes, stream, a);
  if (e != cudaSuccess || !L.far_sum) return e;
  const long long n_sum = static_cast<long long>(L.g.Hkv) * L.g.B * L.g.n_docs * L.g.ns;
  if (n_sum > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  a.sum = L.far_sum;
  return launch_behind(far_sum_kernel<D>, dim3(static_cast<unsigned>(n_sum)), 8 * D, 0, stream, a);
}

}  // namespace

// One wave of equal CTAs while the kv heads leave several to each (a run's start and end cost some
// microseconds), else three, so that the last wave's idle share is small.
int window_far_chunk(const WinGeo& g) {
  const long long heads = static_cast<long long>(g.Hkv) * g.B;
  const long long sms = sm_count(), per_head = (heads <= sms / 2 ? sms : 3 * sms) / heads;
  return per_head > 1 ? static_cast<int>((g.n_tiles + per_head - 1) / per_head) : g.n_tiles;
}

// Documents of less than 32 tokens on average: few of them reach past their tile's band, and the sums
// would make most of the workspace.
bool window_far_summable(const WinGeo& g) { return g.n_docs <= 4LL * g.n_tiles; }
// Up to 256 KB of runs for a (document, kv head) the key-major kernel's items add them up themselves (the
// backward of 8192 tokens, 16/4 heads, window 128: 133 us against 136 with a launch for 128 KB of runs;
// window 512: 200 against 202 for 128 KB, but 231 against 221 for 544 KB).
bool window_far_summed(const WinGeo& g, int D) {
  const long long chunk = window_far_chunk(g), runs = (g.n_tiles + chunk - 1) / chunk;
  return window_far_summable(g) && runs * g.ns * 2 * D > kFarOwn;
}

cudaError_t launch_window_far(const WinLaunch& L, cudaStream_t stream) {
  return L.D == 128 ? launch_d<128>(L, stream) : L.D == 64 ? launch_d<64>(L, stream) : cudaErrorInvalidValue;
}

}  // namespace usp
