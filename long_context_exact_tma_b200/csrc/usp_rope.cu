// usp_rope.cu -- rotary positions with several axes (time, height, width): every
// frequency f of a head row takes its position from one of the axes,
//   a = position[axis(f)] * inv_freq[f],
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a
// for the pair (x1, x2) = elements (f, f + R/2) or (2f, 2f + 1); elements from R
// on are copied. The inverse (the gradient's map) turns by -a.
//
// The angle of a far position needs more bits than fp32 has (at position 10^5 an
// fp32 product is off by 4e-3 rad). Here it is counted in turns on 64 bits: the
// host gives inv_freq / 2 pi as a 64-bit fraction of a turn, off by less than one
// count, and the wrapping 64-bit product with the position drops whole turns and
// nothing else: the angle is off by less than |position| 2^-64 turns (2^-24 at
// position 2^40). The product's upper 32 bits, as a signed number, are the angle
// within half a turn.
//
// Bound by memory: each element is read and written once. A thread takes one
// 16-byte chunk column (two in the halves form, of the copied rest too) of one token and walks some of its
// heads, four at a time, so that the sines are computed once per walk; the lanes of a warp cover
// neighbouring chunks and heads. Views whose rows are not 16-byte aligned take the
// same kernel with one-element chunks.
// 16384 tokens of 32 + 8 heads, D=128, bf16: 55 us on the device, 6.1 TB/s; 15009
// tokens of 16 + 16 heads, D=64, fp32, pairs side by side: 34 us (L2 holds part).
#include <math.h>

#include "../../include/usp.h"
#include "usp_div.cuh"
#include "usp_internal.h"
#include "usp_ptx.cuh"

namespace usp {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxFreq = USP_ROPE_MAX_R / 2;
constexpr int kHeadsPerThread = 8;

struct Job {
  const void* src;
  void* dst;
  int H, groups, g0;  // heads; threads that share a token's heads; the first of them
  long long s_b, s_t, s_h, d_b, d_t, d_h;
};

struct RopeArgs {
  Job job[USP_MAX_ROPE_JOBS];
  int n_jobs, D, R, pos64, inverse;
  Div chunks, groups, S;   // chunks of a row, threads that share a token's chunk, tokens of a sequence
  uint32_t tokens, slice;  // all tokens; those of one blockIdx.y
  long long axis_step;     // tokens per axis of the position table
  const void* pos;
  unsigned long long turn[kMaxFreq];  // inv_freq / 2 pi as a fraction of 2^64
  unsigned char axis[kMaxFreq];
};

template <class T, int V>
struct Chunk {
  T e[V];
};
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T narrow(float x) {
  if constexpr (sizeof(T) == 4)
    return x;
  else
    return __float2bfloat16_rn(x);  // the one rounding of the output
}
template <class T, int V>
__device__ __forceinline__ Chunk<T, V> load(const T* p) {
  Chunk<T, V> c;
  if constexpr (V * sizeof(T) == 16)
    *reinterpret_cast<uint4*>(&c) = *reinterpret_cast<const uint4*>(p);
  else
    for (int x = 0; x < V; ++x) c.e[x] = p[x];
  return c;
}
template <class T, int V>
__device__ __forceinline__ void store(T* p, const Chunk<T, V>& c) {
  if constexpr (V * sizeof(T) == 16)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&c);
  else
    for (int x = 0; x < V; ++x) p[x] = c.e[x];
}

// The rotated pair, its products and sums spelled out: left to the compiler, the variants contract them
// differently, and a row's result would depend on its alignment.
__device__ __forceinline__ float2 turned(float x1, float x2, float c, float s) {
  return make_float2(__fmaf_rn(x1, c, -__fmul_rn(x2, s)), __fmaf_rn(x2, c, __fmul_rn(x1, s)));
}

// kPaired: a chunk of kV elements holds kV / 2 whole pairs; else it is kV first
// elements, whose partners lie R / 2 on.
template <class T, int kV, bool kPaired>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kF = kPaired ? (kV + 1) / 2 : kV;  // frequencies of a chunk
  constexpr int kW = kPaired ? 2 * kF : kV;        // elements of a chunk
  __shared__ unsigned long long s_turn[kMaxFreq];
  __shared__ unsigned char s_axis[kMaxFreq];
  for (int x = threadIdx.x; x < a.R / 2; x += kThreads) {
    s_turn[x] = a.turn[x];
    s_axis[x] = a.axis[x];
  }
  __syncthreads();
  const uint32_t n_rot = a.R / 2 / kF;
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;  // (token of the slice, group, chunk)
  const uint32_t r = quot(a.chunks, u), chunk = u - r * a.chunks.d;
  const uint32_t tok = quot(a.groups, r), grp_ = r - tok * a.groups.d;
  const uint32_t token = blockIdx.y * a.slice + tok;
  if (tok >= a.slice || token >= a.tokens) return;
  const int grp = static_cast<int>(grp_);
  const uint32_t bq = quot(a.S, token);
  const long long b = bq, t = token - bq * a.S.d;
  int j = 0;
  while (j + 1 < a.n_jobs && grp >= a.job[j + 1].g0) ++j;
  const Job& job = a.job[j];
  const int h0 = grp - job.g0;
  const T* src = static_cast<const T*>(job.src) + b * job.s_b + t * job.s_t;
  T* dst = static_cast<T*>(job.dst) + b * job.d_b + t * job.d_t;
  // a chunk past R is copied (in place: left alone)
  const bool rot = chunk < n_rot;
  if (!rot && src == dst && job.s_h == job.d_h) return;
  const int e1 = rot ? static_cast<int>(chunk) * kW : a.R + static_cast<int>(chunk - n_rot) * kV;
  // the halves form's partner; of a copied chunk the one half of the rest on, if there is one (as many
  // bytes as a rotated column: with one chunk each, half of each row rotated took 72 us against 55)
  const int gap = rot ? a.R / 2 : static_cast<int>(a.chunks.d - n_rot) * kV;
  const bool two = rot || e1 + gap < a.D;
  // the first heads' chunks are on their way while the sines are made
  constexpr int kAhead = 4;
  Chunk<T, kW> x1s[kAhead], x2s[kPaired ? 1 : kAhead];
  auto fetch = [&](int h) {
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int hy = h + y * job.groups;
      if (hy >= job.H) break;
      const T* p = src + hy * job.s_h + e1;
      if constexpr (kW == kV)
        x1s[y] = load<T, kW>(p);
      else if (rot)
        x1s[y] = load<T, kW>(p);
      else  // one element past R
        x1s[y].e[0] = p[0];
      if constexpr (!kPaired)
        if (two) x2s[y] = load<T, kV>(p + gap);
    }
  };
  fetch(h0);
  float c[kF], s[kF];
#pragma unroll
  for (int f = 0; f < kF; ++f) {
    if (!rot) break;
    const int fr = chunk * kF + f;
    const long long at = s_axis[fr] * a.axis_step + token;
    const long long p = a.pos64 ? static_cast<const long long*>(a.pos)[at] : static_cast<const int*>(a.pos)[at];
    const unsigned long long turn = s_turn[fr] * static_cast<unsigned long long>(p);
    const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
    if constexpr (sizeof(T) == 4) {
      sincospif(half_turns, &s[f], &c[f]);
    } else {  // absolute error below 2^-20 in [-pi, pi], far below bf16's rounding
      __sincosf(half_turns * 3.14159265358979f, &s[f], &c[f]);
    }
    if (a.inverse) s[f] = -s[f];
  }
  for (int h = h0; h < job.H; h += kAhead * job.groups) {
    if (h != h0) fetch(h);
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int hy = h + y * job.groups;
      if (hy >= job.H) break;
      Chunk<T, kW>& v1 = x1s[y];
      T* const to = dst + hy * job.d_h + e1;
      if (!rot) {
        if constexpr (kW == kV)
          store<T, kW>(to, v1);
        else
          to[0] = v1.e[0];
        if constexpr (!kPaired)
          if (two) store<T, kV>(to + gap, x2s[y]);
        continue;
      }
      if constexpr (kPaired) {
#pragma unroll
        for (int f = 0; f < kF; ++f) {
          const float2 y = turned(widen(v1.e[2 * f]), widen(v1.e[2 * f + 1]), c[f], s[f]);
          v1.e[2 * f] = narrow<T>(y.x);
          v1.e[2 * f + 1] = narrow<T>(y.y);
        }
        store<T, kW>(to, v1);
      } else {
        Chunk<T, kV>& v2 = x2s[y];
#pragma unroll
        for (int f = 0; f < kF; ++f) {
          const float2 y = turned(widen(v1.e[f]), widen(v2.e[f]), c[f], s[f]);
          v1.e[f] = narrow<T>(y.x);
          v2.e[f] = narrow<T>(y.y);
        }
        store<T, kV>(to, v1);
        store<T, kV>(to + gap, v2);
      }
    }
  }
}

template <class T, int kV, bool kPaired>
cudaError_t launch(RopeArgs& a, long long tokens, cudaStream_t st) {
  constexpr int kF = kPaired ? (kV + 1) / 2 : kV;
  const uint32_t n_copy = (a.D - a.R) / kV;
  const uint32_t n_chunks = a.R / 2 / kF + (kPaired ? n_copy : (n_copy + 1) / 2);
  // Heads per thread: as many as pay the sines back, fewer while the tokens alone do not fill the machine.
  int per = kHeadsPerThread;
  auto groups_at = [&](int hp) {
    uint32_t n = 0;
    for (int j = 0; j < a.n_jobs; ++j) n += (a.job[j].H + hp - 1) / hp;
    return n;
  };
  while (per > 1 && tokens * n_chunks * groups_at(per) < 148LL * 1024) per /= 2;
  int groups = 0;
  for (int j = 0; j < a.n_jobs; ++j) {
    a.job[j].g0 = groups;
    a.job[j].groups = (a.job[j].H + per - 1) / per;
    groups += a.job[j].groups;
  }
  const long long lanes = static_cast<long long>(n_chunks) * groups;  // threads of a token
  if (lanes >= 1LL << 30) return cudaErrorInvalidConfiguration;
  a.chunks = make_div(n_chunks);
  a.groups = make_div(groups);
  a.tokens = static_cast<uint32_t>(tokens);
  // thread numbers of a slice stay below 2^31
  const long long most = ((1LL << 31) - kThreads) / lanes;
  a.slice = static_cast<uint32_t>(tokens < most ? tokens : most);
  const long long blocks = (a.slice * lanes + kThreads - 1) / kThreads, slices = (tokens + a.slice - 1) / a.slice;
  if (slices > 65535) return cudaErrorInvalidConfiguration;
  rope_kernel<T, kV, kPaired><<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(slices)), kThreads, 0, st>>>(a);
  note_launch();
  return cudaGetLastError();
}

// inv_freq / 2 pi modulo 1 as a fraction of 2^64, off by less than one count: the product with
// 1 / 2 pi in two doubles, whole turns per position step dropped. That holds up to kMaxInvFreq: lo is the
// part of a turn that the product's double leaves out, and from 2^43 on its own rounding shows in the
// last count; past 2^52 it is more turns than the counts' 64 bits.
constexpr double kMaxInvFreq = 1099511627776.0;  // 2^40
unsigned long long turn_of(double inv_freq) {
  if (inv_freq < 0) return 0ull - turn_of(-inv_freq);
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / 2 pi and what its double leaves out
  const double hi = inv_freq * kHi, lo = fma(inv_freq, kHi, -hi) + inv_freq * kLo;
  const double frac = hi - floor(hi);           // exact
  const double up = floor(frac * 4294967296.0), rest = frac * 4294967296.0 - up;  // upper 32 bits, and the rest of them
  const long long low = static_cast<long long>((rest + lo * 4294967296.0) * 4294967296.0);  // may be just below 0
  return (static_cast<unsigned long long>(up) << 32) + static_cast<unsigned long long>(low);
}

// Whether rows of D elements at b * sb + t * st + h * sh may share elements: each step, the smallest
// first, must be past the rows within it.
bool rows_overlap(int D, int B, long long sb, int S, long long st, int H, long long sh) {
  long long n[3] = {B, S, H}, s[3] = {sb, st, sh}, extent = D;
  for (int x = 0; x < 3; ++x)
    if (n[x] == 1) s[x] = 0;
  for (int round = 0; round < 3; ++round) {
    int at = -1;
    for (int x = 0; x < 3; ++x)
      if (n[x] > 1 && (at < 0 || s[x] < s[at])) at = x;
    if (at < 0) return false;
    if (s[at] < extent) return true;
    extent += (n[at] - 1) * s[at];
    n[at] = 1;
  }
  return false;
}

}  // namespace
}  // namespace usp

using namespace usp;

extern "C" int usp_rope_axes(const usp_rope_job* jobs, int n_jobs, int B, int S, int D, int R, int dtype,
                             const void* positions, int pos_bits, int n_axes, const double* inv_freq, const int* axis,
                             int paired, int inverse, void* stream) {
  if (!jobs || !positions || !inv_freq || !axis) return record_error(USP_ERR_INVALID_ARG, "null pointer");
  if (n_jobs < 1 || n_jobs > USP_MAX_ROPE_JOBS)
    return record_error(USP_ERR_INVALID_ARG, "n_jobs must be 1..%d", USP_MAX_ROPE_JOBS);
  if (B <= 0 || S <= 0 || D <= 0) return record_error(USP_ERR_INVALID_ARG, "sizes must be positive");
  if (dtype != USP_BF16 && dtype != USP_F32) return record_error(USP_ERR_INVALID_ARG, "dtype must be USP_BF16 or USP_F32");
  if (pos_bits != 32 && pos_bits != 64) return record_error(USP_ERR_INVALID_ARG, "pos_bits must be 32 or 64");
  if (reinterpret_cast<uintptr_t>(positions) % (pos_bits / 8))
    return record_error(USP_ERR_INVALID_ARG, "misaligned positions");
  if ((paired | inverse) & ~1) return record_error(USP_ERR_INVALID_ARG, "paired and inverse must be 0 or 1");
  if (n_axes < 1 || n_axes > 255) return record_error(USP_ERR_INVALID_ARG, "n_axes must be 1..255");
  if (R < 2 || R % 2 || R > D || R > USP_ROPE_MAX_R)
    return record_error(USP_ERR_UNSUPPORTED, "R must be even, 2..min(D, %d) (got %d)", USP_ROPE_MAX_R, R);
  const int es = dtype == USP_BF16 ? 2 : 4;
  RopeArgs a{};
  // whole 16-byte chunks everywhere, or single elements
  const int V = 16 / es;
  bool wide = D % V == 0 && (paired ? R % V == 0 : (R / 2) % V == 0);
  for (int x = 0; x < n_jobs; ++x) {
    usp_rope_job j = jobs[x];
    if (B == 1) j.s_b = j.d_b = 0;  // a stride of one step says nothing
    if (S == 1) j.s_t = j.d_t = 0;
    if (j.H == 1) j.s_h = j.d_h = 0;
    if (!j.src || !j.dst) return record_error(USP_ERR_INVALID_ARG, "job %d: null pointer", x);
    if (j.H <= 0) return record_error(USP_ERR_INVALID_ARG, "job %d: heads must be positive", x);
    const uintptr_t bits = reinterpret_cast<uintptr_t>(j.src) | reinterpret_cast<uintptr_t>(j.dst);
    if (bits % es) return record_error(USP_ERR_INVALID_ARG, "job %d: misaligned pointer", x);
    wide = wide && bits % 16 == 0;
    const long long strides[6] = {j.s_b, j.s_t, j.s_h, j.d_b, j.d_t, j.d_h};
    for (long long v : strides) {
      if (v < 0) return record_error(USP_ERR_INVALID_ARG, "job %d: negative stride", x);
      wide = wide && v % V == 0;
    }
    // two rows of the output must not share elements (an input may be broadcast by stride 0)
    if (rows_overlap(D, B, j.d_b, S, j.d_t, j.H, j.d_h))
      return record_error(USP_ERR_INVALID_ARG, "job %d: the output's rows overlap", x);
    if (j.src == j.dst && (j.s_b != j.d_b || j.s_t != j.d_t || j.s_h != j.d_h))
      return record_error(USP_ERR_INVALID_ARG, "job %d: in place with other strides", x);
    for (int y = 0; y < x; ++y)  // the jobs run side by side
      if (j.dst == a.job[y].dst || j.dst == a.job[y].src || j.src == a.job[y].dst)
        return record_error(USP_ERR_INVALID_ARG, "jobs %d and %d: one writes what the other uses", y, x);
    a.job[x].src = j.src;
    a.job[x].dst = j.dst;
    a.job[x].H = j.H;
    a.job[x].s_b = j.s_b; a.job[x].s_t = j.s_t; a.job[x].s_h = j.s_h;
    a.job[x].d_b = j.d_b; a.job[x].d_t = j.d_t; a.job[x].d_h = j.d_h;
  }
  a.n_jobs = n_jobs;
  const long long tokens = static_cast<long long>(B) * S;
  if (tokens >= 1LL << 31) return record_error(USP_ERR_UNSUPPORTED, "too many rows");
  a.S = make_div(S);
  a.D = D; a.R = R;
  a.pos = positions;
  a.pos64 = pos_bits == 64;
  a.inverse = inverse;
  a.axis_step = tokens;
  for (int f = 0; f < R / 2; ++f) {
    if (!isfinite(inv_freq[f])) return record_error(USP_ERR_INVALID_ARG, "inv_freq[%d] is not finite", f);
    if (fabs(inv_freq[f]) > kMaxInvFreq)
      return record_error(USP_ERR_UNSUPPORTED, "inv_freq[%d] = %g is past 2^40", f, inv_freq[f]);
    if (axis[f] < 0 || axis[f] >= n_axes) return record_error(USP_ERR_INVALID_ARG, "axis[%d] = %d is outside 0..%d", f, axis[f], n_axes - 1);
    a.turn[f] = turn_of(inv_freq[f]);
    a.axis[f] = static_cast<unsigned char>(axis[f]);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == USP_BF16) {
    e = wide ? (paired ? launch<__nv_bfloat16, 8, true>(a, tokens, st) : launch<__nv_bfloat16, 8, false>(a, tokens, st))
             : (paired ? launch<__nv_bfloat16, 1, true>(a, tokens, st) : launch<__nv_bfloat16, 1, false>(a, tokens, st));
  } else {
    e = wide ? (paired ? launch<float, 4, true>(a, tokens, st) : launch<float, 4, false>(a, tokens, st))
             : (paired ? launch<float, 1, true>(a, tokens, st) : launch<float, 1, false>(a, tokens, st));
  }
  return e == cudaSuccess ? USP_OK : record_error(USP_ERR_CUDA, "rotary positions launch: %s", cudaGetErrorString(e));
}
