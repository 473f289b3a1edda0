// usp_window_decode.cu -- sliding-window attention with sinks for the newest n
// tokens of each sequence over a cache of keys and values (visibility as in
// usp_window.cuh with one document: token t of a sequence of len tokens sits at
// position len - n + t).
//
// Bound by reading the visible cache rows once: 4 D bytes per key and kv head
// against 4 D flops per key and query row. The n tokens of the heads of a group
// share the kv head's rows, 16 query rows per warp tile, so the products run on the
// 16x8x16 warp-level matrix instruction, whose rate is far above what the memory
// feeds. The keys are split over CTAs and inside a CTA over four streams: a stream
// is one warp that takes 16 keys at a time, or two that share 32 when there are more
// than 16 query rows, from its own ring of cp.async buffers (no block
// barrier in the loop) with its own running maximum, sum and O. The streams'
// results are joined in shared memory; up to 8 splits form a cluster and join
// through distributed shared memory in the same launch.
//
// Few sequences of long and unequal lengths need more: there the CTAs share out the
// keys of all sequences of a kv head in equal chunks (each works its share out from
// lens; 4 conversations of 30 to 128 thousand tokens took 199 us in equal splits of
// each), write fp32 partials, and a second kernel joins a row's by their LSE.
//
// 64 sequences, W=4096, H=32/8, D=128: 154 us on the device, 6.9 TB/s of visible
// rows; 4 tokens of 4 conversations, H=32/4: 115 us and 9 us of joining.
#include <math.h>

#include "../../include/usp.h"
#include "usp_internal.h"
#include "usp_mma.cuh"
#include "usp_ptx.cuh"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kStreams = 4;
constexpr int kMaxCluster = 8;  // splits that join in one launch (the portable cluster size)
constexpr int kMaxShares = 296;  // CTAs of a kv head that share out the keys
constexpr int kSms = 148;
constexpr float kRescale = 8.f;  // log2 units: O is rescaled only when the maximum grows by more than 2^8

struct DecArgs {
  const __nv_bfloat16 *q, *k, *v;
  const int* lens;
  long long k_sn, k_st, k_sh, v_sn, v_st, v_sh;
  __nv_bfloat16* out;
  float* lse;
  // shares: fp32 partials [Hkv][row block][share][row][D] and [..][row]
  float* o_part;
  float* lse_part;
  int N, n, cap, Hq, Hkv, G, W, ns;
  int cluster;   // splits of a sequence that join in the launch
  int n_shares;  // or, with cluster = 1, the CTAs of a (kv head, row block) that share the keys out; 0: none
  int row_blocks;
  float scale_log2;
};

// kRt: row tiles (warps) of a stream. One leaves room for two CTAs on an SM, two
// take more steps in flight instead.
template <int D, int kRt>
struct DecCfg {
  static constexpr int kThreads = 32 * kStreams * kRt;
  static constexpr int kUnit = 16 * kRt;  // keys of a stream's step
  static constexpr int kStages = 3;
  static constexpr int kChunks = D / 8;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kStageBytes = 2 * kUnit * kRowBytes;  // K then V
  static constexpr int kStreamBytes = kStages * kStageBytes;
  static constexpr int kSmemBytes = kStreams * kStreamBytes;
  // a stream's results over its own buffers: O [16 kRt][D] fp32, then m, l, lb per row
  static constexpr int kRows = 16 * kRt;
  static_assert(kRows * D * 4 + 3 * kRows * 4 <= kStreamBytes, "results fit over the buffers");
};

// The keys that any of a sequence's tokens sees, listed: sinks [0, sE), then the window [wlo, len).
struct SeqKeys {
  int len, wlo, sE, total;
};
__device__ __forceinline__ SeqKeys seq_keys(const DecArgs& a, int seq) {
  SeqKeys k;
  k.len = min(max(__ldg(a.lens + seq), 0), a.cap);
  k.wlo = max(0, k.len - a.n - a.W + 1);
  k.sE = min(a.ns, k.wlo);
  k.total = k.sE + k.len - k.wlo;
  return k;
}

// How the n_shares CTAs of a kv head share out the keys of all sequences: chunks of `chunk` steps of
// kStep keys, the smallest that needs no more than n_shares CTAs; ceil(steps / chunk) for a sequence.
// A warp's work; every lane returns the same.
template <int kStep>
struct Shares {
  int chunk;
  __device__ __forceinline__ static int steps(const DecArgs& a, int seq) {
    return (seq_keys(a, seq).total + kStep - 1) / kStep;
  }
  __device__ __forceinline__ static int sum(int v) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  }
  __device__ __forceinline__ int needs(const DecArgs& a, int c) const {
    const int lane = threadIdx.x & 31;
    int t = 0;
    for (int s = lane; s < a.N; s += 32) t += (steps(a, s) + c - 1) / c;
    return sum(t);
  }
  __device__ __forceinline__ void plan(const DecArgs& a) {
    const int lane = threadIdx.x & 31;
    long long all = 0;
    int most = 0;
    for (int s = lane; s < a.N; s += 32) {
      const int t = steps(a, s);
      all += t;
      most = max(most, t);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
      all += __shfl_xor_sync(0xffffffffu, all, d);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
    }
    int lo = static_cast<int>((all + a.n_shares - 1) / a.n_shares), hi = max(most, 1);  // hi: one CTA a sequence
    lo = max(lo, 1);
    while (lo < hi) {  // needs() falls with the chunk
      const int mid = (lo + hi) / 2;
      if (needs(a, mid) <= a.n_shares)
        hi = mid;
      else
        lo = mid + 1;
    }
    chunk = hi;
  }
  // The sequence whose share x is, and its number there; false past the last.
  __device__ __forceinline__ bool locate(const DecArgs& a, int x, int& seq, int& split) const {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int s0 = 0; s0 < a.N; s0 += 32) {
      const int mine = s0 + lane < a.N ? (steps(a, s0 + lane) + chunk - 1) / chunk : 0;
      int incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, x >= before + incl - mine && x < before + incl);
      if (hit) {
        const int who = __ffs(hit) - 1;
        seq = s0 + who;
        split = x - before - __shfl_sync(0xffffffffu, incl - mine, who);
        return true;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;
  }
  // The first share of sequence seq.
  __device__ __forceinline__ int first(const DecArgs& a, int seq) const {
    const int lane = threadIdx.x & 31;
    int t = 0;
    for (int s = lane; s < seq; s += 32) t += (steps(a, s) + chunk - 1) / chunk;
    return sum(t);
  }
};

__device__ __forceinline__ float ld_peer(const float* p, int rank) {  // this address in the cluster's CTA `rank`
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

template <int D, int kRt>
__global__ void __launch_bounds__(DecCfg<D, kRt>::kThreads, kRt == 1 ? 2 : 1) window_decode_kernel(const DecArgs a) {
  using C = DecCfg<D, kRt>;
  constexpr int kUnit = C::kUnit;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g4 = lane >> 2, c4 = lane & 3;
  const int stream = warp & (kStreams - 1), wrt = warp / kStreams;  // the warp's stream and row tile
  constexpr int kStep = kUnit * kStreams;
  let_next_start();
  int x = blockIdx.x, split, seq, rb, kvh, x0, x1, share = 0;
  if (a.n_shares == 0) {
    split = x % a.cluster;  // a cluster is the splits of one (sequence, kv head, rows)
    x /= a.cluster;
    rb = x % a.row_blocks;
    x /= a.row_blocks;
    kvh = x % a.Hkv;
    seq = x / a.Hkv;
  } else {
    share = x;
    x /= a.n_shares;
    rb = x % a.row_blocks;
    kvh = x / a.row_blocks;
    Shares<kStep> sh;
    sh.plan(a);
    if (!sh.locate(a, share % a.n_shares, seq, split)) return;
    x0 = sh.chunk;
  }
  const int rows = a.n * a.G;  // rows of a (sequence, kv head): token major, then head of the group
  const SeqKeys keys = seq_keys(a, seq);
  const int len = keys.len, wlo = keys.wlo, sE = keys.sE;
  const long long per = a.n_shares ? static_cast<long long>(x0) * kStep
                                   : ((keys.total + a.cluster - 1) / a.cluster + kUnit - 1) / kUnit * kUnit;
  x0 = static_cast<int>(min(split * per, static_cast<long long>(keys.total)));
  x1 = static_cast<int>(min(x0 + per, static_cast<long long>(keys.total)));
  const int units = (x1 - x0 + kUnit - 1) / kUnit;
  const int mine = units > stream ? (units - stream + kStreams - 1) / kStreams : 0;  // stream, stream + kStreams, ...

  const uint32_t buf = smem_addr(smem) + stream * C::kStreamBytes;
  const __nv_bfloat16* kb = a.k + seq * a.k_sn + kvh * a.k_sh;
  const __nv_bfloat16* vb = a.v + seq * a.v_sn + kvh * a.v_sh;
  auto fetch = [&](int it) {  // the stream's warps share the rows of a step
    if (it < mine) {
      const int base = x0 + (stream + it * kStreams) * kUnit;
      const uint32_t dst = buf + (it % C::kStages) * C::kStageBytes;
#pragma unroll
      for (int y = 0; y < kUnit * C::kChunks / 32 / kRt; ++y) {
        const int r = (y * kRt + wrt) * (32 / C::kChunks) + lane / C::kChunks, ch = lane % C::kChunks;
        const int xi = base + r;
        const bool ok = xi < x1;
        const long long key = ok ? (xi < sE ? xi : wlo + xi - sE) : 0;
        const uint32_t off = r * C::kRowBytes + ((ch ^ (r & 7)) << 4);
        cp_async16(dst + off, kb + key * a.k_st + ch * 8, ok);
        cp_async16(dst + kUnit * C::kRowBytes + off, vb + key * a.v_st + ch * 8, ok);
      }
    }
    cp_async_commit();
  };
  auto stream_sync = [&]() {
    if constexpr (kRt == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(1 + stream), "n"(32 * kRt) : "memory");
  };
  for (int it = 0; it < C::kStages - 1; ++it) fetch(it);

  // Q fragments of rows g4 and g4 + 8 of the row tile; the rows' positions
  uint32_t qf[D / 16][4];
  int pos[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = (rb * kRt + wrt) * 16 + g4 + half * 8;
    const bool live = r < rows;
    pos[half] = live ? len - a.n + r / a.G : -1;  // -1: sees nothing
    const __nv_bfloat16* p =
        a.q + ((static_cast<long long>(seq) * a.n + (live ? r / a.G : 0)) * a.Hq + kvh * a.G + (live ? r % a.G : 0)) * D;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      qf[kk][half] = live ? *reinterpret_cast<const uint32_t*>(p + kk * 16 + c4 * 2) : 0u;
      qf[kk][2 + half] = live ? *reinterpret_cast<const uint32_t*>(p + kk * 16 + 8 + c4 * 2) : 0u;
    }
  }
  float o[D / 8][4];
#pragma unroll
  for (int y = 0; y < D / 8; ++y)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[y][e] = 0.f;
  float m_use[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lb[2] = {0.f, 0.f};

  for (int it = 0; it < mine; ++it) {
    cp_async_wait<C::kStages - 2>();
    stream_sync();  // the step's rows are there, and every warp is done with the stage that is filled next
    fetch(it + C::kStages - 1);
    const uint32_t sk = buf + (it % C::kStages) * C::kStageBytes, sv = sk + kUnit * C::kRowBytes;
    constexpr int kN = kUnit / 8;  // 8-key column tiles
    float sc[kN][4] = {};
    const int br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int u = 0; u < kN; u += 2) {
        uint32_t kf[4];
        ldsm_x4(kf, sk + (br + u * 8) * C::kRowBytes + (((2 * kk + bc) ^ (br & 7)) << 4));
        mma_16816(sc[u], qf[kk], kf[0], kf[1]);
        mma_16816(sc[u + 1], qf[kk], kf[2], kf[3]);
      }
    }
    const int base = x0 + (stream + it * kStreams) * kUnit;
    // a step of window keys that every token sees needs no mask (rows past the last are not written)
    const int key0 = wlo + base - sE;
    if (!(base >= sE && base + kUnit <= x1 && key0 + kUnit <= len - a.n + 1 && len - 1 - key0 < a.W)) {
#pragma unroll
      for (int u = 0; u < kN; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int xi = base + u * 8 + c4 * 2 + (e & 1), p = pos[e >> 1];
          const int key = xi < sE ? xi : wlo + xi - sE;
          if (!(xi < x1 && key <= p && (p - key < a.W || key < a.ns))) sc[u][e] = -INFINITY;
        }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < kN; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], sc[u][e]);
    float alpha[2];
    bool bump = false;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 1));
      mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 2));
      mx[half] *= a.scale_log2;
      alpha[half] = 1.f;
      if (mx[half] > m_use[half] + kRescale) {
        alpha[half] = ex2_approx(m_use[half] - mx[half]);
        m_use[half] = mx[half];
        bump = true;
      }
    }
    if (__any_sync(0xffffffffu, bump)) {
#pragma unroll
      for (int y = 0; y < D / 8; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[y][e] *= alpha[e >> 1];
    }
    uint32_t pa[kN / 2][4];
    float rs[2] = {0.f, 0.f}, rb[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kN; ++u)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float ms = m_use[half] == -INFINITY ? 0.f : m_use[half];
        const float p0 = ex2_approx(fmaf(sc[u][2 * half], a.scale_log2, -ms));
        const float p1 = ex2_approx(fmaf(sc[u][2 * half + 1], a.scale_log2, -ms));
        const uint32_t pk = pack_bf16x2(p0, p1);
        rs[half] += p0 + p1;
        const float2 w = add_bf16x2_f32(make_float2(0.f, 0.f), pk);
        rb[half] += w.x + w.y;  // O is divided by the sum of the rounded weights that made it
        pa[u / 2][(u & 1) * 2 + half] = pk;
      }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] = l[half] * alpha[half] + rs[half];
      lb[half] = lb[half] * alpha[half] + rb[half];
    }
    const int vr = lane & 15, vc = lane >> 4;
#pragma unroll
    for (int y = 0; y < D / 16; ++y) {
#pragma unroll
      for (int u = 0; u < kN / 2; ++u) {
        uint32_t vf[4];
        ldsm_x4_trans(vf, sv + (vr + u * 16) * C::kRowBytes + (((2 * y + vc) ^ (vr & 7)) << 4));
        mma_16816(o[2 * y], pa[u], vf[0], vf[1]);
        mma_16816(o[2 * y + 1], pa[u], vf[2], vf[3]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  // the warp's result over its stream's buffers
  float* wo = reinterpret_cast<float*>(smem + stream * C::kStreamBytes);
  float* ws = wo + C::kRows * D;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    lb[half] += __shfl_xor_sync(0xffffffffu, lb[half], 1);
    lb[half] += __shfl_xor_sync(0xffffffffu, lb[half], 2);
    const int r = wrt * 16 + g4 + half * 8;
    if (c4 == 0) {
      ws[r] = m_use[half];
      ws[C::kRows + r] = l[half];
      ws[2 * C::kRows + r] = lb[half];
    }
#pragma unroll
    for (int y = 0; y < D / 8; ++y)
      *reinterpret_cast<float2*>(wo + r * D + y * 8 + c4 * 2) = make_float2(o[y][2 * half], o[y][2 * half + 1]);
  }
  __syncthreads();
  // join the streams: eight threads per row, each with its columns sub * 4 + 32 y
  const int r = threadIdx.x >> 3, sub = threadIdx.x & 7, gr = rb * C::kRows + r;
  float m = -INFINITY, lt = 0.f, lbt = 0.f, f[kStreams];
  float4 t[D / 32];
  {
#pragma unroll
    for (int y = 0; y < kStreams; ++y)
      m = fmaxf(m, reinterpret_cast<float*>(smem + y * C::kStreamBytes)[C::kRows * D + r]);
    const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int y = 0; y < kStreams; ++y) {
      const float* s = reinterpret_cast<float*>(smem + y * C::kStreamBytes) + C::kRows * D;
      f[y] = ex2_approx(s[r] - ms);
      lt += f[y] * s[C::kRows + r];
      lbt += f[y] * s[2 * C::kRows + r];
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      t[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < kStreams; ++y) {
        const float4 w = *reinterpret_cast<const float4*>(smem + y * C::kStreamBytes + (r * D + sub * 4 + e * 32) * 4);
        t[e].x += f[y] * w.x;
        t[e].y += f[y] * w.y;
        t[e].z += f[y] * w.z;
        t[e].w += f[y] * w.w;
      }
    }
  }
  bool write = gr < rows;
  if (a.cluster > 1) {
    // the CTA's result in place of stream 0's (every element is read and written by one thread),
    // then each CTA joins every cluster-th row
    float* co = reinterpret_cast<float*>(smem);
    float* cs = co + C::kRows * D;
    __syncwarp();  // a row's threads have read the streams' m, l, lb
#pragma unroll
    for (int e = 0; e < D / 32; ++e) *reinterpret_cast<float4*>(co + r * D + sub * 4 + e * 32) = t[e];
    if (sub == 0) {
      cs[r] = m;
      cs[C::kRows + r] = lt;
      cs[2 * C::kRows + r] = lbt;
    }
    cluster_sync();
    write = write && r % a.cluster == split;
    if (write) {
      m = -INFINITY;
      for (int c = 0; c < a.cluster; ++c) m = fmaxf(m, ld_peer(cs + r, c));
      const float ms = m == -INFINITY ? 0.f : m;
      lt = lbt = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) t[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < a.cluster; ++c) {
        const float w = ex2_approx(ld_peer(cs + r, c) - ms);
        lt += w * ld_peer(cs + C::kRows + r, c);
        lbt += w * ld_peer(cs + 2 * C::kRows + r, c);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const float* p = co + r * D + sub * 4 + e * 32;
          t[e].x += w * ld_peer(p, c);
          t[e].y += w * ld_peer(p + 1, c);
          t[e].z += w * ld_peer(p + 2, c);
          t[e].w += w * ld_peer(p + 3, c);
        }
      }
    }
    cluster_sync();  // no CTA ends while another reads its results
  }
  if (!write) return;
  const float inv = lbt > 0.f ? 1.f / lbt : 0.f;
  const float lse = lt > 0.f ? (m + __log2f(lt)) * 0.6931471805599453f : -INFINITY;
  if (a.n_shares) {
    const long long prow = static_cast<long long>(share) * C::kRows + r;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
      *reinterpret_cast<float4*>(a.o_part + prow * D + sub * 4 + e * 32) =
          make_float4(t[e].x * inv, t[e].y * inv, t[e].z * inv, t[e].w * inv);
    if (sub == 0) a.lse_part[prow] = lse;
    return;
  }
  const long long orow =
      (static_cast<long long>(seq) * a.n + gr / a.G) * a.Hq + static_cast<long long>(kvh) * a.G + gr % a.G;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) {
    uint2 pk;
    pk.x = pack_bf16x2(t[e].x * inv, t[e].y * inv);
    pk.y = pack_bf16x2(t[e].z * inv, t[e].w * inv);
    *reinterpret_cast<uint2*>(a.out + orow * D + sub * 4 + e * 32) = pk;
  }
  if (sub == 0) a.lse[orow] = lse;
}

// The partials' join, a warp per row: its lanes take the shares' LSE, then four columns each, eight
// shares' loads at a time.
template <int D, int kRt>
__global__ void __launch_bounds__(128) window_join_kernel(const DecArgs a) {
  constexpr int kRows = DecCfg<D, kRt>::kRows, kStep = DecCfg<D, kRt>::kUnit * kStreams;
  const int lane = threadIdx.x & 31;
  const long long row = (static_cast<long long>(blockIdx.x) * 128 + threadIdx.x) >> 5;  // of [N][n][Hq]
  if (row >= static_cast<long long>(a.N) * a.n * a.Hq) return;
  const int h = static_cast<int>(row % a.Hq), t = static_cast<int>(row / a.Hq % a.n);
  const int seq = static_cast<int>(row / a.Hq / a.n), kvh = h / a.G;
  const int r = t * a.G + h % a.G;  // row of the (sequence, kv head)
  Shares<kStep> sh;
  sh.plan(a);
  wait_for_previous();  // lens is an input: only the partials are awaited
  const int n = (Shares<kStep>::steps(a, seq) + sh.chunk - 1) / sh.chunk;
  const long long first =
      (static_cast<long long>(kvh) * a.row_blocks + r / kRows) * a.n_shares + sh.first(a, seq);
  const long long p0 = first * kRows + r % kRows;
  float m = -INFINITY;
  for (int s = lane; s < n; s += 32) m = fmaxf(m, a.lse_part[p0 + static_cast<long long>(s) * kRows]);
#pragma unroll
  for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  const float ms = m == -INFINITY ? 0.f : m;
  const bool mine = lane * 4 < D;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  for (int s0 = 0; s0 < n; s0 += 32) {
    const float w = s0 + lane < n ? expf(a.lse_part[p0 + static_cast<long long>(s0 + lane) * kRows] - ms) : 0.f;
    z += w;
    const int k = min(32, n - s0);
    for (int y0 = 0; y0 < k; y0 += 8) {
      float4 p[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        p[y] = mine && y0 + y < k
                   ? *reinterpret_cast<const float4*>(a.o_part + (p0 + static_cast<long long>(s0 + y0 + y) * kRows) * D + lane * 4)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const float wy = __shfl_sync(0xffffffffu, w, (y0 + y) & 31);
        o.x += wy * p[y].x;
        o.y += wy * p[y].y;
        o.z += wy * p[y].z;
        o.w += wy * p[y].w;
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) z += __shfl_xor_sync(0xffffffffu, z, d);
  const float inv = z > 0.f ? 1.f / z : 0.f;
  if (mine) {
    uint2 pk;
    pk.x = pack_bf16x2(o.x * inv, o.y * inv);
    pk.y = pack_bf16x2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(a.out + row * D + lane * 4) = pk;
  }
  if (lane == 0) a.lse[row] = z > 0.f ? m + logf(z) : -INFINITY;
}

struct DecPlan {
  int rt, row_blocks, cluster, n_shares;
  size_t ws;
};

// Splits of a sequence: as many as fill the SMs (two CTAs each with one row tile a stream, one with
// two), none shorter than a step per stream, up to 8 in a cluster of a power of two. Where the splits
// would be longer than 2048 keys (8 us and more) and the SMs hold several CTAs for each sequence, the
// keys are shared out instead, which costs a second launch (about 5 us) and evens the lengths out.
DecPlan plan(int N, int n, int cap, int Hq, int Hkv, int D, int window, int sinks) {
  DecPlan p{};
  const int rows = n * (Hq / Hkv);
  p.rt = rows > 16 ? 2 : 1;
  p.row_blocks = (rows + 16 * p.rt - 1) / (16 * p.rt);
  const long long most = static_cast<long long>(window) + n - 1 + sinks;
  const long long keys = most < cap ? most : cap;
  const long long heads = static_cast<long long>(Hkv) * p.row_blocks;
  const long long slots = (p.rt == 1 ? 2LL : 1LL) * kSms;
  long long s = slots / (heads * N);
  const int step = 16 * p.rt * kStreams;
  const long long by_keys = (keys + step - 1) / step;
  if (s > by_keys) s = by_keys;
  if (s < 1) s = 1;
  p.cluster = 1;
  while (2 * p.cluster <= s && 2 * p.cluster <= kMaxCluster) p.cluster *= 2;
  p.ws = kStatusBytes;
  if (s > 1 && keys / p.cluster >= 2048) {
    p.cluster = 1;
    const long long share = slots / heads;
    p.n_shares = static_cast<int>(share < kMaxShares ? share : kMaxShares);
    p.ws += static_cast<size_t>(heads) * p.n_shares * (16 * p.rt) * (4 * static_cast<size_t>(D) + 4);
  }
  return p;
}

template <int D, int kRt>
cudaError_t launch_dec(const DecArgs& a, unsigned blocks, cudaStream_t st) {
  using C = DecCfg<D, kRt>;
  static_assert(C::kSmemBytes <= 227 * 1024, "shared memory budget");
  cudaError_t e = cudaFuncSetAttribute(window_decode_kernel<D, kRt>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, window_decode_kernel<D, kRt>, a);
  if (e != cudaSuccess) return e;
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess || a.n_shares == 0) return e;
  const long long rows = static_cast<long long>(a.N) * a.n * a.Hq;
  return launch_behind(window_join_kernel<D, kRt>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, st, a);
}

int check(int N, int n, int cap, int Hq, int Hkv, int D, int window, int sinks) {
  if (N <= 0 || n <= 0 || cap <= 0 || Hq <= 0 || Hkv <= 0) return record_error(USP_ERR_INVALID_ARG, "sizes must be positive");
  if (window < 1) return record_error(USP_ERR_INVALID_ARG, "window must be at least 1 (got %d)", window);
  if (sinks < 0) return record_error(USP_ERR_INVALID_ARG, "sinks must not be negative (got %d)", sinks);
  if (D != 64 && D != 128) return record_error(USP_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", D);
  if (Hq % Hkv != 0) return record_error(USP_ERR_UNSUPPORTED, "Hq %% Hkv != 0");
  if (n > USP_WINDOW_MAX_NEW)
    return record_error(USP_ERR_UNSUPPORTED, "at most %d new tokens a sequence (got %d)", USP_WINDOW_MAX_NEW, n);
  if (sinks > USP_WINDOW_MAX_SINKS)
    return record_error(USP_ERR_UNSUPPORTED, "at most %d sinks (got %d)", USP_WINDOW_MAX_SINKS, sinks);
  if (cap > 1 << 30) return record_error(USP_ERR_UNSUPPORTED, "a cache of more than 2^30 tokens");
  if (static_cast<long long>(N) * n * Hq * 8 >= (1LL << 31)) return record_error(USP_ERR_UNSUPPORTED, "too many rows");
  return USP_OK;
}

}  // namespace
}  // namespace usp

using namespace usp;

extern "C" size_t usp_window_decode_workspace_size(int N, int n, int cap, int Hq, int Hkv, int D, int window,
                                                   int sinks) {
  if (check(N, n, cap, Hq, Hkv, D, window, sinks) != USP_OK) return 0;
  return plan(N, n, cap, Hq, Hkv, D, window < cap ? window : cap, sinks).ws;
}

extern "C" int usp_window_attn_decode(const void* q, const void* k_cache, const void* v_cache, const int* lens,
                                      void* out, float* lse, int N, int n, int cap, int Hq, int Hkv, int D, int window,
                                      int sinks, long long k_sn, long long k_st, long long k_sh, long long v_sn,
                                      long long v_st, long long v_sh, void* workspace, size_t ws_bytes, void* stream) {
  const int rc = check(N, n, cap, Hq, Hkv, D, window, sinks);
  if (rc != USP_OK) return rc;
  const void* ptrs[5] = {q, k_cache, v_cache, out, lse};
  for (const void* p : ptrs) {
    if (!p) return record_error(USP_ERR_INVALID_ARG, "null pointer");
    if (reinterpret_cast<uintptr_t>(p) & 15u) return record_error(USP_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  }
  if (!lens || (reinterpret_cast<uintptr_t>(lens) & 3u)) return record_error(USP_ERR_INVALID_ARG, "null or misaligned lens");
  if (N == 1) k_sn = v_sn = 0;  // a stride of one step says nothing
  if (cap == 1) k_st = v_st = 0;
  if (Hkv == 1) k_sh = v_sh = 0;
  const long long strides[6] = {k_sn, k_st, k_sh, v_sn, v_st, v_sh};
  for (long long s : strides)
    if (s < 0 || s % 8) return record_error(USP_ERR_INVALID_ARG, "cache strides must be multiples of 8 elements");
  if (window > cap) window = cap;
  const DecPlan p = plan(N, n, cap, Hq, Hkv, D, window, sinks);
  const bool parts = p.n_shares > 0;
  if (parts && (!workspace || ws_bytes < p.ws || (reinterpret_cast<uintptr_t>(workspace) & 15u)))
    return record_error(USP_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu)", p.ws, ws_bytes);
  DecArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k_cache);
  a.v = static_cast<const __nv_bfloat16*>(v_cache);
  a.lens = lens;
  a.k_sn = k_sn; a.k_st = k_st; a.k_sh = k_sh;
  a.v_sn = v_sn; a.v_st = v_st; a.v_sh = v_sh;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.N = N; a.n = n; a.cap = cap; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
  a.W = window;
  a.ns = sinks;
  a.cluster = p.cluster;
  a.n_shares = p.n_shares;
  a.row_blocks = p.row_blocks;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  const long long heads = static_cast<long long>(Hkv) * p.row_blocks;
  if (parts) {
    a.o_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
    a.lse_part = a.o_part + static_cast<size_t>(heads) * p.n_shares * (16 * p.rt) * D;
  }
  const long long blocks = parts ? heads * p.n_shares : heads * N * p.cluster;
  if (blocks > 0x7FFFFFFFLL) return record_error(USP_ERR_UNSUPPORTED, "too many rows");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned nb = static_cast<unsigned>(blocks);
  const cudaError_t e = D == 128 ? (p.rt == 1 ? launch_dec<128, 1>(a, nb, st) : launch_dec<128, 2>(a, nb, st))
                                 : (p.rt == 1 ? launch_dec<64, 1>(a, nb, st) : launch_dec<64, 2>(a, nb, st));
  return e == cudaSuccess ? USP_OK : record_error(USP_ERR_CUDA, "window decode launch: %s", cudaGetErrorString(e));
}
