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

#include <type_traits>

#include "common.cuh"
#include "fastmath.cuh"

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
// outside [cu[0], cu[n]).  One outcome for the warp, start and end its boundaries.  Every lane
// probes at once: up to 32 segments take one load's latency, up to 1024 three, where a binary
// search takes ten.  Never reads outside cu[0..n], whatever it holds.
__device__ __forceinline__ int warp_segment(const int32_t* __restrict__ cu, int n, int64_t t,
                                            int64_t& start, int64_t& end) {
  const int lane = threadIdx.x & 31;
  if (n <= 32) {
    const int at = min(lane, n - 1);
    const int c0 = __ldg(cu + at), c1 = __ldg(cu + at + 1);
    const unsigned in = __ballot_sync(0xffffffffu, lane < n && (int64_t)c0 <= t);
    const int k = 31 - __clz(in);
    start = __shfl_sync(0xffffffffu, c0, max(k, 0));
    end = __shfl_sync(0xffffffffu, c1, max(k, 0));
    return __shfl_sync(0xffffffffu, c1, n - 1) <= t ? -1 : k;
  }
  const int64_t first = __ldg(cu), last = __ldg(cu + n);
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) >> 5;
    const int at = lane * step;
    const bool in = at < len && (lane == 0 || (int64_t)__ldg(cu + lo + at) <= t);
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, in));
    lo += k * step;
    len = min(step, len - k * step);
  }
  start = __ldg(cu + lo);
  end = __ldg(cu + lo + 1);
  return first > t || last <= t ? -1 : lo;
}

// cos and sin of pair i of a head at position p.
__device__ __forceinline__ void pair_cos_sin(double per_pos, double p, float& c, float& s) {
  const double t = p * per_pos;
  const double n4 = rint(4.0 * t);
  const float r = (float)fma(-0.25, n4, t);
  float s0, c0;
  sincospif(2.f * r, &s0, &c0);
  const int quad = (int)((long long)n4 & 3);
  const float a = (quad & 1) ? s0 : c0, b = (quad & 1) ? c0 : s0;
  c = (quad == 1 || quad == 2) ? -a : a;
  s = (quad >= 2) ? -b : b;
}

// cos and sin of this lane's N pairs (pairs c*N .. c*N + N-1 of the head) at position pos.  The
// kRows lanes that hold the same pairs form N / kRows of them each and pass them round: the
// angles of a token cost the warp N / kRows evaluations, not N.
template <int N, int kLanes>
__device__ __forceinline__ void lane_cos_sin(const Turns& tn, int64_t pos, float (&cs)[N],
                                             float (&sn)[N]) {
  constexpr int kRows = 32 / kLanes, M = N / kRows;
  static_assert(M >= 1 && M * kRows == N, "every lane forms the same number of pairs");
  const int lane = threadIdx.x & 31, c = lane % kLanes, sub = lane / kLanes;
  float co[M], si[M];
#pragma unroll
  for (int e = 0; e < M; ++e)
    pair_cos_sin(tn.per_pos[c * N + sub * M + e], (double)pos, co[e], si[e]);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    cs[e] = __shfl_sync(0xffffffffu, co[e % M], (e / M) * kLanes + c);
    sn[e] = __shfl_sync(0xffffffffu, si[e % M], (e / M) * kLanes + c);
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
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    fastmath::ffma2(s0, s1, xa[e], xa[e + 1], xa[e], xa[e + 1], s0, s1);
    fastmath::ffma2(s0, s1, xb[e], xb[e + 1], xb[e], xb[e + 1], s0, s1);
  }
  return __frsqrt_rn(fmaf(row_sum<kLanes>(s0 + s1), 1.f / D, eps));
}

// Both halves of a lane's weights (ones where there are none).
template <typename T, int D>
__device__ __forceinline__ void load_weights(const T* w, int c, float* wa, float* wb) {
  constexpr int N = Vec16<T>::N;
  if (w != nullptr) {
    Vec16<T>::unpack(ldg16(w + c * N), wa);
    Vec16<T>::unpack(ldg16(w + D / 2 + c * N), wb);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) wa[e] = wb[e] = 1.f;
  }
}

// 16-byte load of data read once.  Not the read-only path: a caller may rotate in place.
__device__ __forceinline__ uint4 ld16_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
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

// Norm and rotation of rows at one position.  The weights are folded into the rotation's factors,
// so an element costs three multiplications: with n = r x, y_a = n_a (w_a cos) - n_b (w_b sin) and
// y_b = n_b (w_b cos) + n_a (w_a sin).
template <typename T, int D>
struct Turn {
  using R = RowLayout<T, D>;
  static constexpr int N = R::N;
  float ac[N], bs[N], bc[N], as[N];   // w_a cos, -w_b sin, w_b cos, w_a sin

  __device__ __forceinline__ void set(const float (&cs)[N], const float (&sn)[N],
                                      const float (&wa)[N], const float (&wb)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      ac[e] = wa[e] * cs[e];
      bs[e] = -wb[e] * sn[e];
      bc[e] = wb[e] * cs[e];
      as[e] = wa[e] * sn[e];
    }
  }
  // One row, held as (ra, rb) by its lanes, to `out` (this lane's 16 bytes of either half) if
  // store.  The whole warp calls it.  Without a rotation an element is no business of its
  // partner's: a product with a sine of 0 would hand on an infinity as NaN, and change zeros' signs.
  // (ROTATE is the compiler's: a branch in here kept rows apart, append of 18K tokens of 8 + 1 heads
  // of 64 20 -> 21.5 us.)
  template <bool ROTATE>
  __device__ __forceinline__ void row(const uint4& ra, const uint4& rb, float eps, bool store,
                                      T* out) const {
    float xa[N], xb[N];
    Vec16<T>::unpack(ra, xa);
    Vec16<T>::unpack(rb, xb);
    const float r = eps > 0.f ? row_rstd<D, N, R::kLanes>(xa, xb, eps) : 1.f;
    if (!store) return;
    float ya[N], yb[N];
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      float p0, p1, q0, q1;
      fastmath::fmul2(p0, p1, xa[e], xa[e + 1], r, r);
      fastmath::fmul2(q0, q1, xb[e], xb[e + 1], r, r);
      fastmath::fmul2(ya[e], ya[e + 1], p0, p1, ac[e], ac[e + 1]);
      fastmath::fmul2(yb[e], yb[e + 1], q0, q1, bc[e], bc[e + 1]);
      if (!ROTATE) continue;
      fastmath::ffma2(ya[e], ya[e + 1], q0, q1, bs[e], bs[e + 1], ya[e], ya[e + 1]);
      fastmath::ffma2(yb[e], yb[e + 1], p0, p1, as[e], as[e + 1], yb[e], yb[e + 1]);
    }
    store_n<T>(out, ya);
    store_n<T>(out + D / 2, yb);
  }
};

// This lane's 16 bytes of either half of a row, zeros when !on.
template <typename T, int D>
__device__ __forceinline__ void load_row(const T* p, bool on, uint4& ra, uint4& rb) {
  ra = rb = make_uint4(0, 0, 0, 0);
  if (on) {
    ra = ld16_once(p);
    rb = ld16_once(p + D / 2);
  }
}

// One token's heads of one tensor, normalised (eps > 0) and rotated: row groups g0, g0 + step, ..
// below `groups` (kRows heads each) of src (heads D apart) to dst (heads `pitch` apart).
// U groups' loads are issued before the first is used.  place() is called between the first
// loads and their use: it finds the token's angles, and says whether to store.
template <typename T, int D, int U, typename Place>
__device__ __forceinline__ void turn_heads(const T* src, T* dst, int64_t pitch, int heads,
                                           const T* w, float eps, bool rotate, int g0, int step,
                                           int groups, Place place) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  const int lane = threadIdx.x & 31, c = lane % R::kLanes, sub = lane / R::kLanes;
  Turn<T, D> turn;
  bool first = true, store = true;
  for (int g = g0; g < groups; g += step * U) {
    uint4 ra[U], rb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (g + u * step) * R::kRows + sub;
      load_row<T, D>(src + (int64_t)h * D + c * N, h < heads, ra[u], rb[u]);
    }
    if (first) {
      float cs[N], sn[N], wa[N], wb[N];
      load_weights<T, D>(w, c, wa, wb);
      store = place(cs, sn);
      turn.set(cs, sn, wa, wb);
      first = false;
    }
    auto rows = [&](auto rot) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = (g + u * step) * R::kRows + sub;
        turn.template row<rot.value>(ra[u], rb[u], eps, h < heads && store,
                                     dst + (int64_t)h * pitch + c * N);
      }
    };
    if (rotate) rows(std::true_type{});
    else rows(std::false_type{});
  }
}

// Warps a token's row groups are dealt to: one, unless the tokens alone leave the SMs without
// enough warps; never more than there are groups.  Every warp looks the token's place up and
// forms its angles (500 / 1000 / 2000 tokens of 32 + 8 heads, norm and rotation: 32 warps an SM
// 8.2 / 13.2 / 15 us, 8 5.4 / 6.4 / 8.7, 2 5.5 / 6.4 / 8.5, but append of 64 tokens 4.8 with 8, 5.7
// with 2).
inline int head_split(int64_t n_tok, int groups) {
  const int64_t want = (int64_t)sm_count() * 8;
  int s = 1;
  while (s < groups && n_tok * s < want) s *= 2;
  return s < groups ? s : groups;
}
// First group at or after `from` that part `part` of `split` takes.
__device__ __forceinline__ int first_group(int from, int part, int split) {
  return from + (part - from % split + split) % split;
}

}  // namespace msa
