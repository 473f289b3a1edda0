// usp_window.cu -- entry points of causal attention with a sliding window and
// sinks over [B][S][H][D] (kernels: usp_window_fwd.cu, usp_window_prep.cu,
// usp_window_dq.cu, usp_window_sink.cu, usp_window_bwd.cu).
#include <math.h>

#include "../../include/usp.h"
#include "usp_internal.h"

using namespace usp;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_shape(int B, int S, int Hq, int Hkv, int D, int window, int sinks, const void* cu, int n_docs, WinGeo* g) {
  if (B <= 0 || S <= 0 || Hq <= 0 || Hkv <= 0) return record_error(USP_ERR_INVALID_ARG, "sizes must be positive");
  if (window < 1) return record_error(USP_ERR_INVALID_ARG, "window must be at least 1 (got %d)", window);
  if (sinks < 0) return record_error(USP_ERR_INVALID_ARG, "sinks must not be negative (got %d)", sinks);
  if (cu && n_docs < 1) return record_error(USP_ERR_INVALID_ARG, "n_docs must be >= 1 with cu_seqlens");
  if (D != 64 && D != 128) return record_error(USP_ERR_UNSUPPORTED, "D must be 64 or 128 (got %d)", D);
  if (Hq % Hkv != 0) return record_error(USP_ERR_UNSUPPORTED, "Hq %% Hkv != 0");
  if (sinks > USP_WINDOW_MAX_SINKS)
    return record_error(USP_ERR_UNSUPPORTED, "at most %d sinks (got %d)", USP_WINDOW_MAX_SINKS, sinks);
  // every query row, rounded up to whole tiles, has a 31-bit number, and so has a position plus a window
  if (S > 1 << 30 || static_cast<long long>(B) * ((S + 127LL) / 128 * 128) * Hq >= (1LL << 31))
    return record_error(USP_ERR_UNSUPPORTED, "too many rows");
  *g = WinGeo{};
  g->B = B; g->S = S; g->Hq = Hq; g->Hkv = Hkv;
  g->G = Hq / Hkv;
  g->W = window < S ? window : S;
  g->ns = sinks < S ? sinks : S;
  g->cu = static_cast<const int*>(cu);
  g->n_docs = cu ? n_docs : 1;
  g->n_tiles = (S + 127) / 128;
  g->scale = 1.0f / sqrtf(static_cast<float>(D));
  g->scale_log2 = g->scale * 1.4426950408889634f;
  return USP_OK;
}

// A window as long as the sequence leaves no query without the sinks in its window.
bool has_far(const WinGeo& g) { return g.ns > 0 && g.W < g.S; }

size_t table_floats(const WinGeo& g) { return static_cast<size_t>(g.B) * g.Hq * g.n_tiles * 128; }
size_t far_part_floats(const WinGeo& g, int D) {
  return has_far(g) ? static_cast<size_t>(g.B) * g.Hkv * g.n_tiles * g.ns * 2 * D : 0;
}
// (none where most documents are far shorter than a tile: window_far_summed)
size_t far_sum_floats(const WinGeo& g, int D) {
  return has_far(g) && window_far_summable(g) ? static_cast<size_t>(g.B) * g.Hkv * g.n_docs * g.ns * 2 * D : 0;
}
// [status][-LSE*log2e][-Delta][far partials][far sums]
size_t bwd_ws(const WinGeo& g, int D) {
  return kStatusBytes + 4 * (2 * table_floats(g) + far_part_floats(g, D) + far_sum_floats(g, D));
}

// [B][S][H][D] bf16 as {D, H, S, B}
int tmap(CUtensorMap* m, const void* base, int D, int H, int S, int B) {
  const unsigned long long row = 2ull * H * D;
  return make_tmap_strided(m, base, D, H, S, B, row, row * S);
}

}  // namespace

extern "C" size_t usp_window_workspace_size(int B, int S, int Hq, int Hkv, int D, int window, int sinks, int n_docs,
                                            int bwd) {
  WinGeo g{};
  // n_docs = 0: no documents (the pointer only says whether there are any)
  if (n_docs < 0 || check_shape(B, S, Hq, Hkv, D, window, sinks, n_docs ? &g : nullptr, n_docs, &g) != USP_OK) return 0;
  return bwd ? bwd_ws(g, D) : static_cast<size_t>(kStatusBytes);
}

extern "C" int usp_window_attn_fwd(const void* q, const void* k, const void* v, void* out, float* lse, int B, int S,
                                   int Hq, int Hkv, int D, int window, int sinks, const int* cu_seqlens, int n_docs,
                                   void* workspace, size_t ws_bytes, void* stream) {
  WinLaunch L{};
  int rc = check_shape(B, S, Hq, Hkv, D, window, sinks, cu_seqlens, n_docs, &L.g);
  if (rc != USP_OK) return rc;
  if (!q || !k || !v || !out || !lse) return record_error(USP_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse))
    return record_error(USP_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  if (!workspace || ws_bytes < static_cast<size_t>(kStatusBytes) || !aligned16(workspace))
    return record_error(USP_ERR_WORKSPACE, "workspace needs %d bytes (got %zu)", kStatusBytes, ws_bytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  L.D = D;
  if ((rc = tmap(&L.tm_q, q, D, Hq, S, B)) != USP_OK) return rc;
  if ((rc = tmap(&L.tm_k, k, D, Hkv, S, B)) != USP_OK) return rc;
  if ((rc = tmap(&L.tm_v, v, D, Hkv, S, B)) != USP_OK) return rc;
  L.out = out;
  L.lse = lse;
  L.status = static_cast<int*>(workspace);
  L.wait_ns = current_wait_ns();
  cudaError_t e = cudaMemsetAsync(workspace, 0, kStatusBytes, st);
  if (e == cudaSuccess) e = launch_window_fwd(L, st);
  return e == cudaSuccess ? USP_OK : record_error(USP_ERR_CUDA, "window attention forward: %s", cudaGetErrorString(e));
}

extern "C" int usp_window_attn_bwd(const void* q, const void* k, const void* v, const void* out, const float* lse,
                                   const void* dO, void* dQ, void* dK, void* dV, int B, int S, int Hq, int Hkv, int D,
                                   int window, int sinks, const int* cu_seqlens, int n_docs, void* workspace,
                                   size_t ws_bytes, void* stream) {
  WinLaunch L{};
  int rc = check_shape(B, S, Hq, Hkv, D, window, sinks, cu_seqlens, n_docs, &L.g);
  if (rc != USP_OK) return rc;
  const void* ptrs[9] = {q, k, v, out, lse, dO, dQ, dK, dV};
  for (const void* p : ptrs) {
    if (!p) return record_error(USP_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(p)) return record_error(USP_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  }
  const size_t need = bwd_ws(L.g, D);
  if (!workspace || ws_bytes < need || !aligned16(workspace))
    return record_error(USP_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu)", need, ws_bytes);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  L.D = D;
  if ((rc = tmap(&L.tm_q, q, D, Hq, S, B)) != USP_OK) return rc;
  if ((rc = tmap(&L.tm_k, k, D, Hkv, S, B)) != USP_OK) return rc;
  if ((rc = tmap(&L.tm_v, v, D, Hkv, S, B)) != USP_OK) return rc;
  if ((rc = tmap(&L.tm_do, dO, D, Hq, S, B)) != USP_OK) return rc;
  L.dq = dQ;
  L.dk = dK;
  L.dv = dV;
  L.q = q;
  L.k = k;
  L.v = v;
  L.dO = dO;
  float* f = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kStatusBytes);
  float* lse2 = f;
  float* delta = lse2 + table_floats(L.g);
  L.lse2 = lse2;
  L.delta = delta;
  L.Lp = L.g.n_tiles * 128;
  if (has_far(L.g)) {
    L.far_part = delta + table_floats(L.g);
    L.far_chunk = window_far_chunk(L.g);
    if (window_far_summed(L.g, D)) L.far_sum = L.far_part + far_part_floats(L.g, D);
  }
  L.status = static_cast<int*>(workspace);
  L.wait_ns = current_wait_ns();
  cudaError_t e = launch_window_prep(L, out, lse, st);
  if (e == cudaSuccess) e = launch_window_dq(L, st);
  if (e == cudaSuccess && L.far_part) e = launch_window_far(L, st);
  if (e == cudaSuccess) e = launch_window_dkdv(L, st);
  return e == cudaSuccess ? USP_OK : record_error(USP_ERR_CUDA, "window attention backward: %s", cudaGetErrorString(e));
}
