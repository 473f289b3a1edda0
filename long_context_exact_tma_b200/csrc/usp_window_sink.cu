// usp_window_sink.cu -- backward of sliding-window attention with sinks: dK and
// dV of the sinks from the far queries, those whose tile lies behind the band of
// the sink's key tile (usp_window.cuh) and that the key-major kernel so never
// visits. A query tile m has far sinks of one document only, that of its first
// row: any other document with rows in m starts inside m.
//
//   dV_s = sum_i P_is dO_i,  dK_s / scale = sum_i P_is (dO_i.v_s - Delta_i) Q_i
//
// A few keys against every query is bound by reading Q and dO once, so the
// products run on the warp-level 16x8x16 matrix instruction (a 128-key tensor
// tile would be 4 keys in 128): warp = 16 query rows, 16 sinks at a time. One CTA
// per (query tile, kv head, batch) writes the fp32 sums over its rows and the
// group's heads, warp by warp in a fixed order; a second kernel adds the tiles in
// a fixed order. No atomics: the result does not depend on scheduling.
#include <math.h>

#include "usp_mma.cuh"
#include "usp_ptx.cuh"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 16;  // sinks at a time

struct FarArgs {
  WinGeo g;
  const __nv_bfloat16 *q, *k, *v, *dO;
  const float *lse2, *delta;
  int Lp;
  float* part;
  float* sum;
};

// The sink at position j is far from query tile m.
__device__ __forceinline__ bool is_far(const WinGeo& g, int j, int m) { return last_qtile(g, j / kBN) < m; }

template <int D>
struct FarCfg {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  static constexpr int kTile = kBM * kRowBytes;
  static constexpr int kOffDO = kTile;
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = kOffK + kGroup * kRowBytes;
  static constexpr int kOffSum = kOffV + kGroup * kRowBytes;  // fp32 [kGroup][2][D]
  static constexpr int kSmemBytes = kOffSum + kGroup * 2 * D * 4;
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
  const int m = blockIdx.x % g.n_tiles, gl = blockIdx.x / g.n_tiles % g.Hkv, b = blockIdx.x / g.n_tiles / g.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int q0 = m * kBM;
  int lo, hi;
  win_span(g, q0, lo, hi);
  const int n_sinks = min(g.ns, hi - lo);
  if (!is_far(g, lo, m)) return;  // band ends grow with the key: no sink is far
  const uint32_t s_base = smem_addr(smem);
  float* sums = reinterpret_cast<float*>(smem + C::kOffSum);
  float* part = a.part + ((static_cast<size_t>(b) * g.Hkv + gl) * g.n_tiles + m) * g.ns * (2 * D);

  for (int s0 = 0; s0 < n_sinks; s0 += kGroup) {
    __syncthreads();
    for (int x = tid; x < kGroup * C::kChunks; x += kThreads) {
      const int r = x / C::kChunks, ch = x % C::kChunks;
      uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
      if (s0 + r < n_sinks) {
        const size_t e = ((static_cast<size_t>(b) * g.S + lo + s0 + r) * g.Hkv + gl) * D + ch * 8;
        kv = *reinterpret_cast<const uint4*>(a.k + e);
        vv = *reinterpret_cast<const uint4*>(a.v + e);
      }
      *reinterpret_cast<uint4*>(smem + C::kOffK + at<D>(r, ch)) = kv;
      *reinterpret_cast<uint4*>(smem + C::kOffV + at<D>(r, ch)) = vv;
    }
    for (int x = tid; x < kGroup * 2 * D; x += kThreads) sums[x] = 0.f;
    // which of this lane's sink columns (2c, 2c+1 and 2c+8, 2c+9 of the group) are far
    bool far[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int s = s0 + u * 8 + (lane & 3) * 2 + e;
        far[u][e] = s < n_sinks && is_far(g, lo + s, m);
      }
    float av[D / 8][4], ak[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) av[x][e] = ak[x][e] = 0.f;

    for (int hh = 0; hh < g.G; ++hh) {
      const int h = gl * g.G + hh;
      __syncthreads();  // the previous head's tiles have been read
#pragma unroll 4
      for (int x = tid; x < kBM * C::kChunks; x += kThreads) {
        const int r = x / C::kChunks, ch = x % C::kChunks;
        uint4 qv = make_uint4(0, 0, 0, 0), dv = qv;
        if (q0 + r < g.S) {
          const size_t e = ((static_cast<size_t>(b) * g.S + q0 + r) * g.Hq + h) * D + ch * 8;
          qv = *reinterpret_cast<const uint4*>(a.q + e);
          dv = *reinterpret_cast<const uint4*>(a.dO + e);
        }
        *reinterpret_cast<uint4*>(smem + at<D>(r, ch)) = qv;
        *reinterpret_cast<uint4*>(smem + C::kOffDO + at<D>(r, ch)) = dv;
      }
      __syncthreads();
      // S = Q K^T, dP = dO V^T of 16 rows and 16 sinks
      float sc[2][4] = {}, dp[2][4] = {};
      const int ar = warp * 16 + (lane & 15), ac = lane >> 4;         // A rows and half chunks
      const int br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;  // B: sinks and halves
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint32_t qa[4], da[4], kb[4], vb[4];
        ldsm_x4(qa, s_base + at<D>(ar, 2 * kk + ac));
        ldsm_x4(da, s_base + C::kOffDO + at<D>(ar, 2 * kk + ac));
        ldsm_x4(kb, s_base + C::kOffK + at<D>(br, 2 * kk + bc));
        ldsm_x4(vb, s_base + C::kOffV + at<D>(br, 2 * kk + bc));
        mma_16816(sc[0], qa, kb[0], kb[1]);
        mma_16816(sc[1], qa, kb[2], kb[3]);
        mma_16816(dp[0], da, vb[0], vb[1]);
        mma_16816(dp[1], da, vb[2], vb[3]);
      }
      uint32_t pt[4], dt[4];  // P^T, dS^T: sinks x rows
      const int i0 = q0 + warp * 16 + (lane >> 2);
      const size_t tab = (static_cast<size_t>(b) * g.Hq + h) * a.Lp + i0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // rows i0, i0 + 8
        const bool live = i0 + half * 8 < hi;   // a row of the same document (hi <= S)
        const float nl = a.lse2[tab + half * 8], nd = a.delta[tab + half * 8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          float p[2], ds[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[e] = live && far[u][e] ? ex2_approx(sc[u][half * 2 + e] * g.scale_log2 + nl) : 0.f;
            ds[e] = p[e] * (dp[u][half * 2 + e] + nd);
          }
          // bf16 operands, as P and dS have in the key-major kernel; sums stay fp32
          pt[half * 2 + u] = mov_trans(pack_bf16x2(p[0], p[1]));
          dt[half * 2 + u] = mov_trans(pack_bf16x2(ds[0], ds[1]));
        }
      }
      const int tr = warp * 16 + (lane & 15), tc = lane >> 4;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        uint32_t db[4], qb[4];
        ldsm_x4_trans(db, s_base + C::kOffDO + at<D>(tr, 2 * x + tc));
        ldsm_x4_trans(qb, s_base + at<D>(tr, 2 * x + tc));
        mma_16816(av[2 * x], pt, db[0], db[1]);
        mma_16816(av[2 * x + 1], pt, db[2], db[3]);
        mma_16816(ak[2 * x], dt, qb[0], qb[1]);
        mma_16816(ak[2 * x + 1], dt, qb[2], qb[3]);
      }
    }
    for (int y = 0; y < kThreads / 32; ++y) {  // warp by warp: a fixed order of the sum
      __syncthreads();
      if (warp == y) {
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int s = (lane >> 2) + (e >> 1) * 8, d = x * 8 + (lane & 3) * 2 + (e & 1);
            sums[(s * 2 + 0) * D + d] += ak[x][e];
            sums[(s * 2 + 1) * D + d] += av[x][e];
          }
      }
    }
    __syncthreads();
    const int n = min(kGroup, n_sinks - s0) * 2 * D;
    for (int x = tid; x < n; x += kThreads) part[static_cast<size_t>(s0) * 2 * D + x] = sums[x];
  }
}

// sum[b][gl][d][s] = the far tiles' partials of sink s of document d, in four
// interleaved runs added in order.
template <int D>
__global__ void __launch_bounds__(8 * D) far_sum_kernel(const FarArgs a) {
  __shared__ float run[4][2 * D];
  const WinGeo& g = a.g;
  const int s = blockIdx.x % g.ns, d = blockIdx.x / g.ns % g.n_docs;
  const int gl = blockIdx.x / g.ns / g.n_docs % g.Hkv, b = blockIdx.x / g.ns / g.n_docs / g.Hkv;
  int lo = 0, hi = g.S;
  if (g.cu) {
    lo = min(max(__ldg(g.cu + d), 0), g.S);
    hi = min(max(__ldg(g.cu + d + 1), lo), g.S);
  }
  if (lo + s >= hi) return;  // no such key: nothing reads its sum
  const int m0 = last_qtile(g, (lo + s) / kBN) + 1, m1 = (hi - 1) / kBM;
  const int col = threadIdx.x % (2 * D), y = threadIdx.x / (2 * D);
  const size_t tile = static_cast<size_t>(g.ns) * 2 * D;
  const float* p = a.part + (static_cast<size_t>(b) * g.Hkv + gl) * g.n_tiles * tile + static_cast<size_t>(s) * 2 * D + col;
  float t = 0.f;
#pragma unroll 8
  for (int m = m0 + y; m <= m1; m += 4) t += p[m * tile];
  run[y][col] = t;
  __syncthreads();
  if (y == 0)
    a.sum[(((static_cast<size_t>(b) * g.Hkv + gl) * g.n_docs + d) * g.ns + s) * (2 * D) + col] =
        (run[0][col] + run[1][col]) + (run[2][col] + run[3][col]);
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
  a.sum = L.far_sum;
  const long long heads = static_cast<long long>(L.g.Hkv) * L.g.B, n_far = heads * L.g.n_tiles;
  const long long n_sum = heads * L.g.n_docs * L.g.ns;
  if (n_far > 0x7FFFFFFFLL || n_sum > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  far_kernel<D><<<static_cast<unsigned>(n_far), kThreads, C::kSmemBytes, stream>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  far_sum_kernel<D><<<static_cast<unsigned>(n_sum), 8 * D, 0, stream>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_far(const WinLaunch& L, cudaStream_t stream) {
  return L.D == 128 ? launch_d<128>(L, stream) : L.D == 64 ? launch_d<64>(L, stream) : cudaErrorInvalidValue;
}

}  // namespace usp
