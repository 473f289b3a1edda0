// usp_window_prep.cu -- the row tables of the window backward: -LSE*log2(e) and
// -Delta = -sum_d dO_d O_d, per head ([B*Hq][Lp], Lp = S rounded up to 128; -inf
// and 0 on the padding rows, whose weights then are 0). The backward's first kernel:
// it also clears the workspace header (status word, item counters).
//
// Bound by reading O and dO once. Neighbouring lanes read neighbouring 16 bytes
// (D/8 lanes make a row), and a warp asks for all of its 8 or 16 rows before it
// uses the first, so that enough bytes are in flight.
// S=32768 H=16 D=128: 49 us, 5.5 TB/s.
#include <math.h>

#include "usp_internal.h"
#include "usp_window.cuh"

namespace usp {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;  // 16-byte loads of each tensor in flight per lane

template <int D>
__global__ void __launch_bounds__(kThreads) window_prep_kernel(const uint4* __restrict__ out,
                                                               const uint4* __restrict__ dO,
                                                               const float* __restrict__ lse, float* __restrict__ lse2_t,
                                                               float* __restrict__ delta_t,
                                                               int* __restrict__ header, long long rows, int S,
                                                               int Hq, int Lp, long long pad_rows) {
  constexpr int kLanes = D / 8;              // lanes of a row
  constexpr int kRows = 32 / kLanes;         // rows of a step
  let_next_start();
  if (blockIdx.x == 0 && threadIdx.x < kStatusBytes / 4) header[threadIdx.x] = 0;
  const int lane = threadIdx.x & 31;
  const long long warp = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const long long r0 = warp * (kRows * kSteps) + lane / kLanes;
  uint4 x[kSteps], y[kSteps];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const long long r = r0 + s * kRows;
    if (r < rows) {
      x[s] = __ldg(out + r * kLanes + lane % kLanes);
      y[s] = __ldg(dO + r * kLanes + lane % kLanes);
    } else {
      x[s] = y[s] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const __nv_bfloat162* a = reinterpret_cast<const __nv_bfloat162*>(&x[s]);
    const __nv_bfloat162* b = reinterpret_cast<const __nv_bfloat162*>(&y[s]);
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 fa = __bfloat1622float2(a[e]), fb = __bfloat1622float2(b[e]);
      t = fmaf(fa.x, fb.x, t);
      t = fmaf(fa.y, fb.y, t);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
    const long long r = r0 + s * kRows;
    if (lane % kLanes == 0 && r < rows) {
      // (rows have 31-bit numbers: 64-bit divisions made this kernel's time, 67 us for 524288 rows)
      const uint32_t r32 = static_cast<uint32_t>(r), bs = r32 / static_cast<uint32_t>(Hq), h = r32 - bs * Hq;
      const uint32_t bi = bs / static_cast<uint32_t>(S), row = bs - bi * S;
      const size_t dst = (static_cast<size_t>(bi) * Hq + h) * Lp + row;
      const float l = lse[r];
      delta_t[dst] = -t;
      lse2_t[dst] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
    }
  }
  const int pad = Lp - S;
  for (long long x_ = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; x_ < pad_rows;
       x_ += static_cast<long long>(gridDim.x) * kThreads) {
    const long long dst = (x_ / pad) * Lp + S + x_ % pad;
    delta_t[dst] = 0.f;
    lse2_t[dst] = -INFINITY;
  }
}

template <int D>
cudaError_t launch_d(const WinLaunch& L, const void* out, const float* lse, cudaStream_t stream) {
  const long long rows = static_cast<long long>(L.g.B) * L.g.S * L.g.Hq;
  const long long per_block = kThreads / (D / 8) * kSteps;
  const unsigned blocks = static_cast<unsigned>((rows + per_block - 1) / per_block);
  window_prep_kernel<D><<<blocks, kThreads, 0, stream>>>(
      static_cast<const uint4*>(out), static_cast<const uint4*>(L.dO), lse, L.lse2, L.delta, L.status, rows, L.g.S, L.g.Hq, L.Lp,
      static_cast<long long>(L.g.B) * L.g.Hq * (L.Lp - L.g.S));
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_window_prep(const WinLaunch& L, const void* out, const float* lse, cudaStream_t stream) {
  return L.D == 128 ? launch_d<128>(L, out, lse, stream)
                    : L.D == 64 ? launch_d<64>(L, out, lse, stream) : cudaErrorInvalidValue;
}

}  // namespace usp
