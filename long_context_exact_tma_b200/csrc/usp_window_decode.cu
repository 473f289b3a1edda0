// usp_window_decode.cu -- sliding-window attention with sinks for the newest n
// tokens of each sequence over a cache of keys and values (visibility as in
// usp_window.cuh with one document: token t of a sequence of len tokens sits at
// position len - n + t).
//
// Bound by reading the visible cache rows once: 4 D bytes per key and kv head
// against 4 D flops per key and query row. The n tokens of the heads of a group
// share the kv head's rows, up to 16 query rows per warp tile, so the products run
// on the 16x8x16 warp-level matrix instruction, whose rate is far above what the
// memory feeds. The keys are split over CTAs and inside a CTA over its warps: each
// warp streams 16 keys at a time through its own ring of cp.async buffers (no
// block barrier in the loop), keeps its own running maximum, sum and O, and the
// warps' results are joined at the end. With more than one split the CTAs write
// fp32 partials that the log-sum-exp merge joins.
#include <math.h>

#include "../../include/usp.h"
#include "usp_internal.h"
#include "usp_mma.cuh"
#include "usp_ptx.cuh"

namespace usp {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 16;   // keys of a warp's step
constexpr int kStages = 3;  // steps in flight per warp
constexpr int kMaxSplits = 64;
constexpr int kSms = 148;

struct DecArgs {
  const __nv_bfloat16 *q, *k, *v;
  const int* lens;
  long long k_sn, k_st, k_sh, v_sn, v_st, v_sh;
  __nv_bfloat16* out;  // one split
  float* lse;
  float* o_part;       // more: [n_splits][N*n*Hq][D]
  float* lse_part;
  int N, n, cap, Hq, Hkv, G, W, ns, n_splits, row_tiles;
  float scale_log2;
};

template <int D>
struct DecCfg {
  static constexpr int kChunks = D / 8;
  static constexpr int kRowBytes = D * 2;
  static constexpr int kStageBytes = 2 * kUnit * kRowBytes;  // K then V
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kSmemBytes = kWarps * kWarpBytes;
  // the warps' results: O [16][D] fp32 over the warp's own buffers, then m, l, lb per row
  static_assert(16 * D * 4 + 3 * 16 * 4 <= kWarpBytes, "results fit over the buffers");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2) window_decode_kernel(const DecArgs a) {
  using C = DecCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g4 = lane >> 2, c4 = lane & 3;
  int x = blockIdx.x;
  const int split = x % a.n_splits;
  x /= a.n_splits;
  const int rt = x % a.row_tiles;
  x /= a.row_tiles;
  const int kvh = x % a.Hkv, seq = x / a.Hkv;
  const int rows = a.n * a.G;  // rows of a (sequence, kv head): token major, then head of the group
  const int len = min(max(__ldg(a.lens + seq), 0), a.cap);

  // keys of any of the tokens, listed: sinks [0, sE) and the window [wlo, len)
  const int wlo = max(0, len - a.n - a.W + 1);
  const int sE = min(a.ns, wlo);
  const int total = sE + len - wlo;
  const int per = ((total + a.n_splits - 1) / a.n_splits + kUnit - 1) / kUnit * kUnit;
  const int x0 = min(split * per, total), x1 = min(x0 + per, total);
  const int units = (x1 - x0 + kUnit - 1) / kUnit;
  const int mine = units > warp ? (units - warp + kWarps - 1) / kWarps : 0;  // this warp's: warp, warp + kWarps, ...

  const uint32_t buf = smem_addr(smem) + warp * C::kWarpBytes;
  const __nv_bfloat16* kb = a.k + seq * a.k_sn + kvh * a.k_sh;
  const __nv_bfloat16* vb = a.v + seq * a.v_sn + kvh * a.v_sh;
  auto fetch = [&](int it) {
    if (it < mine) {
      const int base = x0 + (warp + it * kWarps) * kUnit;
      const uint32_t dst = buf + (it % kStages) * C::kStageBytes;
#pragma unroll
      for (int y = 0; y < kUnit * C::kChunks / 32; ++y) {
        const int r = y * (32 / C::kChunks) + lane / C::kChunks, ch = lane % C::kChunks;
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
  for (int it = 0; it < kStages - 1; ++it) fetch(it);

  // Q fragments of rows g4 and g4 + 8 of the row tile; the rows' positions
  uint32_t qf[D / 16][4];
  int pos[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = rt * 16 + g4 + half * 8;
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
    fetch(it + kStages - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t sk = buf + (it % kStages) * C::kStageBytes, sv = sk + kUnit * C::kRowBytes;
    float sc[2][4] = {};
    const int br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t kf[4];
      ldsm_x4(kf, sk + br * C::kRowBytes + (((2 * kk + bc) ^ (br & 7)) << 4));
      mma_16816(sc[0], qf[kk], kf[0], kf[1]);
      mma_16816(sc[1], qf[kk], kf[2], kf[3]);
    }
    const int base = x0 + (warp + it * kWarps) * kUnit;
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int xi = base + u * 8 + c4 * 2 + (e & 1), p = pos[e >> 1];
        const int key = xi < sE ? xi : wlo + xi - sE;
        const bool vis = xi < x1 && key <= p && (p - key < a.W || key < a.ns);
        sc[u][e] = vis ? sc[u][e] * a.scale_log2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], sc[u][e]);
      }
    float alpha[2];
    bool bump = false;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 1));
      mx[half] = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 2));
      alpha[half] = 1.f;
      if (mx[half] > m_use[half]) {
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
    uint32_t pa[4];
    float rs[2] = {0.f, 0.f}, rb[2] = {0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float ms = m_use[half] == -INFINITY ? 0.f : m_use[half];
        const float p0 = ex2_approx(sc[u][2 * half] - ms), p1 = ex2_approx(sc[u][2 * half + 1] - ms);
        const uint32_t pk = pack_bf16x2(p0, p1);
        rs[half] += p0 + p1;
        const float2 w = add_bf16x2_f32(make_float2(0.f, 0.f), pk);
        rb[half] += w.x + w.y;  // O is divided by the sum of the rounded weights that made it
        pa[u * 2 + half] = pk;
      }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] = l[half] * alpha[half] + rs[half];
      lb[half] = lb[half] * alpha[half] + rb[half];
    }
    const int vr = lane & 15, vc = lane >> 4;
#pragma unroll
    for (int y = 0; y < D / 16; ++y) {
      uint32_t vf[4];
      ldsm_x4_trans(vf, sv + vr * C::kRowBytes + (((2 * y + vc) ^ (vr & 7)) << 4));
      mma_16816(o[2 * y], pa, vf[0], vf[1]);
      mma_16816(o[2 * y + 1], pa, vf[2], vf[3]);
    }
    __syncwarp();  // every lane has read the stage before it is filled again
  }
  cp_async_wait<0>();
  __syncwarp();
  // the warp's result over its own buffers
  float* wo = reinterpret_cast<float*>(smem + warp * C::kWarpBytes);
  float* ws = wo + 16 * D;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
    l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
    lb[half] += __shfl_xor_sync(0xffffffffu, lb[half], 1);
    lb[half] += __shfl_xor_sync(0xffffffffu, lb[half], 2);
    const int r = g4 + half * 8;
    if (c4 == 0) {
      ws[r] = m_use[half];
      ws[16 + r] = l[half];
      ws[32 + r] = lb[half];
    }
#pragma unroll
    for (int y = 0; y < D / 8; ++y)
      *reinterpret_cast<float2*>(wo + r * D + y * 8 + c4 * 2) = make_float2(o[y][2 * half], o[y][2 * half + 1]);
  }
  __syncthreads();
  // join the warps: eight threads per row
  const int r = threadIdx.x >> 3, sub = threadIdx.x & 7, gr = rt * 16 + r;
  if (gr >= rows) return;
  float m = -INFINITY;
#pragma unroll
  for (int y = 0; y < kWarps; ++y) m = fmaxf(m, reinterpret_cast<float*>(smem + y * C::kWarpBytes)[16 * D + r]);
  const float ms = m == -INFINITY ? 0.f : m;
  float lt = 0.f, lbt = 0.f, f[kWarps];
#pragma unroll
  for (int y = 0; y < kWarps; ++y) {
    const float* s = reinterpret_cast<float*>(smem + y * C::kWarpBytes) + 16 * D;
    f[y] = ex2_approx(s[r] - ms);
    lt += f[y] * s[16 + r];
    lbt += f[y] * s[32 + r];
  }
  const float inv = lbt > 0.f ? 1.f / lbt : 0.f;
  const float lse = lt > 0.f ? (m + __log2f(lt)) * 0.6931471805599453f : -INFINITY;
  const long long orow =
      (static_cast<long long>(seq) * a.n + gr / a.G) * a.Hq + static_cast<long long>(kvh) * a.G + gr % a.G;
  const long long n_rows = static_cast<long long>(a.N) * a.n * a.Hq;
#pragma unroll
  for (int d = sub * 4; d < D; d += 32) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kWarps; ++y) {
      const float4 w = *reinterpret_cast<const float4*>(smem + y * C::kWarpBytes + (r * D + d) * 4);
      t.x += f[y] * w.x;
      t.y += f[y] * w.y;
      t.z += f[y] * w.z;
      t.w += f[y] * w.w;
    }
    if (a.n_splits == 1) {
      uint2 pk;
      pk.x = pack_bf16x2(t.x * inv, t.y * inv);
      pk.y = pack_bf16x2(t.z * inv, t.w * inv);
      *reinterpret_cast<uint2*>(a.out + orow * D + d) = pk;
    } else {
      *reinterpret_cast<float4*>(a.o_part + (split * n_rows + orow) * D + d) =
          make_float4(t.x * inv, t.y * inv, t.z * inv, t.w * inv);
    }
  }
  if (sub == 0) {
    if (a.n_splits == 1)
      a.lse[orow] = lse;
    else
      a.lse_part[split * n_rows + orow] = lse;
  }
}

struct DecPlan {
  int row_tiles, n_splits;
  size_t ws;
};

// Splits: as many as fill every SM twice, none shorter than 64 keys per warp.
DecPlan plan(int N, int n, int cap, int Hq, int Hkv, int D, int window, int sinks) {
  DecPlan p{};
  p.row_tiles = (n * (Hq / Hkv) + 15) / 16;
  const long long most = static_cast<long long>(window) + n - 1 + sinks;
  const long long keys = most < cap ? most : cap;
  const long long blocks = static_cast<long long>(N) * Hkv * p.row_tiles;
  long long s = (2LL * kSms) / blocks;
  const long long by_keys = keys / (64 * kWarps);
  if (s > by_keys) s = by_keys;
  if (s > kMaxSplits) s = kMaxSplits;
  if (s < 1) s = 1;
  p.n_splits = static_cast<int>(s);
  const size_t rows = static_cast<size_t>(N) * n * Hq;
  p.ws = kStatusBytes + (p.n_splits > 1 ? p.n_splits * rows * (4 * static_cast<size_t>(D) + 4) : 0);
  return p;
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
  if (static_cast<long long>(N) * n * Hq * kMaxSplits >= (1LL << 31)) return record_error(USP_ERR_UNSUPPORTED, "too many rows");
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
  if (!workspace || ws_bytes < p.ws || (reinterpret_cast<uintptr_t>(workspace) & 15u))
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
  a.n_splits = p.n_splits;
  a.row_tiles = p.row_tiles;
  a.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  const long long rows = static_cast<long long>(N) * n * Hq;
  a.o_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
  a.lse_part = a.o_part + static_cast<size_t>(p.n_splits) * rows * D;
  const long long blocks = static_cast<long long>(N) * Hkv * p.row_tiles * p.n_splits;
  if (blocks > 0x7FFFFFFFLL) return record_error(USP_ERR_UNSUPPORTED, "too many rows");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (D == 128) {
    e = cudaFuncSetAttribute(window_decode_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecCfg<128>::kSmemBytes);
    if (e == cudaSuccess) window_decode_kernel<128><<<static_cast<unsigned>(blocks), kThreads, DecCfg<128>::kSmemBytes, st>>>(a);
  } else {
    e = cudaFuncSetAttribute(window_decode_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecCfg<64>::kSmemBytes);
    if (e == cudaSuccess) window_decode_kernel<64><<<static_cast<unsigned>(blocks), kThreads, DecCfg<64>::kSmemBytes, st>>>(a);
  }
  if (e == cudaSuccess) {
    note_launch();
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && p.n_splits > 1)
    e = launch_lse_merge(a.o_part, a.lse_part, p.n_splits, rows, D, out, 0, lse, st);
  return e == cudaSuccess ? USP_OK : record_error(USP_ERR_CUDA, "window decode launch: %s", cudaGetErrorString(e));
}
