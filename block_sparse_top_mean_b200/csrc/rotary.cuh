// Per-head RMS norm and rotary positions of packed tokens: the device pieces shared by
// qk_norm_rope.cu (training) and paged_append.cu (serving).
//
// A head row of d elements is held by kLanes = d * sizeof(T) / 32 neighbouring lanes; each
// holds 16 bytes of the row's first half and the 16 bytes of its second half that they
// rotate with, so a rotation needs no shuffle and the row's sums take log2(kLanes).  A warp
// carries 32 / kLanes rows at a time.
//
// Angles.  a_i = pos * base^(-2i/d), formed as turns t = pos * (base^(-2i/d) / 2 pi) in fp64
// (relative error 2^-52: 2e-9 rad at position 2^20).  t - n/4 with n = rint(4 t) lies in
// [-1/8, 1/8] and is rounded to fp32 only there (error <= 2^-28 turns = 2.3e-8 rad);
// sincospif gives its sine and cosine and n mod 4 the quadrant.
#pragma once

#include "common.cuh"

namespace msa {

constexpr int kMaxHalf = 64;          // d / 2

struct Turns {
  double per_pos[kMaxHalf];           // base^(-2i/d) / (2 pi)
};

// Host: the table for one base (long double, rounded once); base <= 0 means no rotation.
Turns make_turns(double base, int d);

template <typename T, int D>
struct RowLayout {
  static constexpr int N = Vec16<T>::N;                     // elements of a 16-byte chunk
  static constexpr int kLanes = D / 2 / N;                  // lanes of one head row
  static constexpr int kRows = 32 / kLanes;                 // head rows of a warp
};

// Index of the last segment whose start is <= t: cu[0..n] are the boundaries; -1 for a t
// outside [cu[0], cu[n]).  One outcome for the warp; 32 probes a round, so up to 1024
// segments take two dependent loads where a binary search takes ten.  Never reads outside
// cu[0..n], whatever it holds.
__device__ __forceinline__ int warp_segment(const int32_t* __restrict__ cu, int n, int64_t t) {
  const int lane = threadIdx.x & 31;
  if ((int64_t)__ldg(cu) > t || (int64_t)__ldg(cu + n) <= t) return -1;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int at = lane * step;
    const bool in = at < len && (lane == 0 || (int64_t)__ldg(cu + lo + at) <= t);
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, in));
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

// cos and sin of this lane's N pairs (pairs c*N .. c*N + N-1 of the head) at position pos.
template <int N>
__device__ __forceinline__ void lane_cos_sin(const Turns& tn, int c, int64_t pos, float* cs,
                                             float* sn) {
  const double p = (double)pos;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const double t = p * tn.per_pos[c * N + e];
    const double n4 = rint(4.0 * t);
    const float r = (float)fma(-0.25, n4, t);
    float s, co;
    sincospif(2.f * r, &s, &co);
    const int quad = (int)((long long)n4 & 3);
    const float a = (quad & 1) ? s : co, b = (quad & 1) ? co : s;
    cs[e] = (quad == 1 || quad == 2) ? -a : a;
    sn[e] = (quad >= 2) ? -b : b;
  }
}

// Sum over the kLanes lanes of a row.
template <int kLanes>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// 1 / sqrt(mean(x^2) + eps) of the row held as (xa, xb) by its lanes.
template <int D, int N, int kLanes>
__device__ __forceinline__ float row_rstd(const float* xa, const float* xb, float eps) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) s = fmaf(xa[e], xa[e], fmaf(xb[e], xb[e], s));
  return __frsqrt_rn(fmaf(row_sum<kLanes>(s), 1.f / D, eps));
}

// 16-byte load of data read once.  Not the read-only path: a caller may rotate in place.
__device__ __forceinline__ uint4 ld16_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
// Loads N elements of T at p into fp32 (the 8 fp32 gradients of a bf16 chunk take two loads).
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float* f) {
  constexpr int M = Vec16<T>::N;
#pragma unroll
  for (int i = 0; i < N; i += M) Vec16<T>::unpack(ld16_once(p + i), f + i);
}
// Rounds N = Vec16<T>::N values to T and stores them as 16 bytes.
template <typename T>
__device__ __forceinline__ void store_n(T* p, const float* f) {
  constexpr int N = Vec16<T>::N;
  alignas(16) T y[N];
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = from_f32<T>(f[e]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(y);
}

}  // namespace msa
