// Per-head RMS norm of queries and keys with the document-wise rotation in the same pass,
// and its gradient ("100 Millionen Token: Gedaechtnis oder Trugbild?", aitalk.it, section
// "Das Gehirn mit zwei Geschwindigkeiten": positions restart at every document).
//
//   r = (mean(x^2) + eps)^(-1/2),  n = r x w,  y = R(pos) n          (per head of d elements)
//   g = R(pos)^T dy,  dw = sum g r x,  u = g w,  dx = r (u - r^2 x mean(u x))
//
// Both directions read every element once and write it once: HBM bound.  A warp takes one
// token (or a part of its heads when there are few tokens), so the token's angles are
// formed once, in registers, for all its heads; rows are laid out as in rotary.cuh.  Four
// rows' loads are issued before the first is used, the token's position is looked up while
// they are under way.
//
// dw sums T * heads terms.  A lane adds up the heads of one token first, then the tokens it
// meets, then lanes, warps and CTAs are joined, each in a fixed order: the sum is the same
// in every run, and no chain of additions is longer than the tokens of one warp.
#include <math.h>

#include "paged.cuh"
#include "rotary.cuh"

namespace msa {

Turns make_turns(double base, int d) {
  // one power and d/2 products: 64 roundings of 2^-64 stay below the one to double, and a
  // call per head dimension and base costs under a microsecond (64 powers: 15 us measured)
  Turns t{};
  if (base <= 0) return t;
  const long double step = powl((long double)base, -2.0L / d);
  long double x = 1.0L / 6.283185307179586476925286766559005768L;
  for (int i = 0; i < d / 2; ++i, x *= step) t.per_pos[i] = (double)x;
  return t;
}

namespace {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;            // rows in flight per lane

struct NormArgs {
  Turns tn;
  int64_t n_tok, qs, ks;              // packed tokens; token strides of q and k (elements)
  int hq, hkv, n_docs, split;         // split: warps a token's heads are dealt to
  float eps;
};

// The token's position in its document (0 for a token no document holds).
__device__ __forceinline__ int64_t token_pos(const int32_t* cu, int n_docs, int64_t t) {
  const int s = warp_segment(cu, n_docs, t);
  return s < 0 ? 0 : t - (int64_t)__ldg(cu + s);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
qk_norm_rope_kernel(const T* q, const T* k, const int32_t* __restrict__ cu,
                    const T* __restrict__ wq, const T* __restrict__ wk, T* qo, T* ko,
                    const __grid_constant__ NormArgs a) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  const int lane = threadIdx.x & 31, c = lane % R::kLanes, sub = lane / R::kLanes;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / a.split;
  if (t >= a.n_tok) return;                               // whole warp
  const int part = (int)(unit - t * a.split);
  const int heads = a.hq + a.hkv;
  const T* qt = q + t * a.qs;
  const T* kt = k + t * a.ks;
  float cs[N], sn[N];
  bool placed = false;
  for (int h0 = part * R::kRows; h0 < heads; h0 += a.split * R::kRows * kUnroll) {
    uint4 ra[kUnroll], rb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * a.split * R::kRows + sub;
      if (h >= heads) continue;
      const T* row = h < a.hq ? qt + (int64_t)h * D : kt + (int64_t)(h - a.hq) * D;
      ra[u] = ld16_once(row + c * N);
      rb[u] = ld16_once(row + D / 2 + c * N);
    }
    if (!placed) {
      lane_cos_sin<N>(a.tn, c, token_pos(cu, a.n_docs, t), cs, sn);
      placed = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * a.split * R::kRows + sub;
      float xa[N], xb[N], wa[N], wb[N];
      const bool on = h < heads;
      Vec16<T>::unpack(on ? ra[u] : make_uint4(0, 0, 0, 0), xa);
      Vec16<T>::unpack(on ? rb[u] : make_uint4(0, 0, 0, 0), xb);
      const float r = row_rstd<D, N, R::kLanes>(xa, xb, a.eps);
      if (!on) continue;
      const T* w = h < a.hq ? wq : wk;
      if (w != nullptr) {
        Vec16<T>::unpack(ldg16(w + c * N), wa);
        Vec16<T>::unpack(ldg16(w + D / 2 + c * N), wb);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) wa[e] = wb[e] = 1.f;
      }
      T* out = h < a.hq ? qo + (t * a.hq + h) * D : ko + (t * a.hkv + (h - a.hq)) * D;
      float ya[N], yb[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float na = xa[e] * r * wa[e], nb = xb[e] * r * wb[e];
        ya[e] = na * cs[e] - nb * sn[e];
        yb[e] = nb * cs[e] + na * sn[e];
      }
      store_n<T>(out + c * N, ya);
      store_n<T>(out + D / 2 + c * N, yb);
    }
  }
}

// ------------------------------------------------------------------ backward
// Persistent warps, one token each at a time.  part[cta][2][D]: the CTA's sums for wq, wk.
template <typename T, typename TG, int D>
__global__ void __launch_bounds__(kWarps * 32)
qk_norm_rope_bwd_kernel(const TG* __restrict__ dq, const TG* __restrict__ dk,
                        const T* __restrict__ q, const T* __restrict__ k,
                        const int32_t* __restrict__ cu, const T* __restrict__ wq,
                        const T* __restrict__ wk, T* __restrict__ dqi, T* __restrict__ dki,
                        float* __restrict__ part, const __grid_constant__ NormArgs a) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  __shared__ float s_dw[kWarps][2][D];
  const int lane = threadIdx.x & 31, c = lane % R::kLanes, sub = lane / R::kLanes;
  const int warp = threadIdx.x >> 5;
  float acc[2][2][N];                                     // [q, k][half][pair]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < N; ++e) acc[i][0][e] = acc[i][1][e] = 0.f;

  const int64_t units = a.n_tok * a.split;
  for (int64_t unit = (int64_t)blockIdx.x * kWarps + warp; unit < units;
       unit += (int64_t)gridDim.x * kWarps) {
    const int64_t t = unit / a.split;
    const int part_i = (int)(unit - t * a.split);
    float cs[N], sn[N];
    lane_cos_sin<N>(a.tn, c, token_pos(cu, a.n_docs, t), cs, sn);
#pragma unroll
    for (int i = 0; i < 2; ++i) {                         // queries, then keys
      const int heads = i ? a.hkv : a.hq;
      const T* xt = i ? k + t * a.ks : q + t * a.qs;
      const TG* gt = (i ? dk : dq) + t * heads * D;
      T* ot = (i ? dki : dqi) + t * heads * D;
      const T* w = i ? wk : wq;
      float wa[N], wb[N];
      if (w != nullptr) {
        Vec16<T>::unpack(ldg16(w + c * N), wa);
        Vec16<T>::unpack(ldg16(w + D / 2 + c * N), wb);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) wa[e] = wb[e] = 1.f;
      }
      float ta[N], tb[N];                                 // this token's heads
#pragma unroll
      for (int e = 0; e < N; ++e) ta[e] = tb[e] = 0.f;
#pragma unroll 2
      for (int h0 = part_i * R::kRows; h0 < heads; h0 += a.split * R::kRows) {
        const int h = h0 + sub;
        const bool on = h < heads;
        float xa[N], xb[N], ga[N], gb[N];
        if (on) {
          load_n<T, N>(xt + (int64_t)h * D + c * N, xa);
          load_n<T, N>(xt + (int64_t)h * D + D / 2 + c * N, xb);
          load_n<TG, N>(gt + (int64_t)h * D + c * N, ga);
          load_n<TG, N>(gt + (int64_t)h * D + D / 2 + c * N, gb);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) xa[e] = xb[e] = ga[e] = gb[e] = 0.f;
        }
        const float r = row_rstd<D, N, R::kLanes>(xa, xb, a.eps);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float y0 = ga[e], y1 = gb[e];
          xa[e] *= r;
          xb[e] *= r;
          const float g0 = y0 * cs[e] + y1 * sn[e], g1 = y1 * cs[e] - y0 * sn[e];
          ta[e] = fmaf(g0, xa[e], ta[e]);
          tb[e] = fmaf(g1, xb[e], tb[e]);
          ga[e] = g0 * wa[e];
          gb[e] = g1 * wb[e];
          dot = fmaf(ga[e], xa[e], fmaf(gb[e], xb[e], dot));
        }
        dot = row_sum<R::kLanes>(dot) * (1.f / D);
        if (!on) continue;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          ga[e] = r * fmaf(-xa[e], dot, ga[e]);
          gb[e] = r * fmaf(-xb[e], dot, gb[e]);
        }
        store_n<T>(ot + (int64_t)h * D + c * N, ga);
        store_n<T>(ot + (int64_t)h * D + D / 2 + c * N, gb);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        acc[i][0][e] += ta[e];
        acc[i][1][e] += tb[e];
      }
    }
  }
  if (part == nullptr) return;
  // rows of the warp (lanes with the same c), then the warps of the CTA in order
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float x = acc[i][h][e];
#pragma unroll
        for (int o = 16; o >= R::kLanes; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (sub == 0) s_dw[warp][i][h * (D / 2) + c * N + e] = x;
      }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += (&s_dw[w][0][0])[i];
    part[(int64_t)blockIdx.x * 2 * D + i] = s;
  }
}

// dw[i] = sum over CTAs of part[cta][i]: 32 columns a block, 32 slices of the CTAs.
__global__ void __launch_bounds__(1024)
dw_sum_kernel(const float* __restrict__ part, int n_cta, int d, float* __restrict__ dwq,
              float* __restrict__ dwk) {
  __shared__ float s[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;
  float v = 0.f;
  for (int c = y; c < n_cta; c += 32) v += part[(int64_t)c * 2 * d + col];
  s[y][x] = v;
  __syncthreads();
  if (y != 0) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += s[i][x];
  float* dst = col < d ? dwq : dwk;
  if (dst != nullptr) dst[col < d ? col : col - d] = v;
}

// Warps a token's heads are dealt to: one, unless the tokens alone leave the SMs without
// enough warps; never more than there are row groups.
int head_split(int64_t n_tok, int heads, int rows) {
  const int64_t want = (int64_t)sm_count() * 32;
  const int groups = (heads + rows - 1) / rows;
  int s = 1;
  while (s < groups && n_tok * s < want) s *= 2;
  return s < groups ? s : groups;
}

template <typename T, int D>
cudaError_t run_fwd(NormArgs& a, const void* q, const void* k, const int32_t* cu, const void* wq,
                    const void* wk, void* qo, void* ko, cudaStream_t st) {
  a.split = head_split(a.n_tok, a.hq + a.hkv, RowLayout<T, D>::kRows);
  const int64_t grid = (a.n_tok * a.split + kWarps - 1) / kWarps;
  qk_norm_rope_kernel<T, D><<<(unsigned)grid, kWarps * 32, 0, st>>>(
      (const T*)q, (const T*)k, cu, (const T*)wq, (const T*)wk, (T*)qo, (T*)ko, a);
  return cudaGetLastError();
}

template <typename T, typename TG, int D>
cudaError_t run_bwd(NormArgs& a, const void* dq, const void* dk, const void* q, const void* k,
                    const int32_t* cu, const void* wq, const void* wk, void* dqi, void* dki,
                    float* dwq, float* dwk, float* part, cudaStream_t st) {
  a.split = head_split(a.n_tok, a.hq, RowLayout<T, D>::kRows);
  int64_t grid = (a.n_tok * a.split + kWarps - 1) / kWarps;
  const int64_t cap = qk_norm_rope_bwd_ctas();
  if (grid > cap) grid = cap;
  const bool dw = dwq != nullptr || dwk != nullptr;
  qk_norm_rope_bwd_kernel<T, TG, D><<<(unsigned)grid, kWarps * 32, 0, st>>>(
      (const TG*)dq, (const TG*)dk, (const T*)q, (const T*)k, cu, (const T*)wq, (const T*)wk,
      (T*)dqi, (T*)dki, dw ? part : nullptr, a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dw) return e;
  dw_sum_kernel<<<2 * D / 32, 1024, 0, st>>>(part, (int)grid, D, dwq, dwk);
  return cudaGetLastError();
}

NormArgs make_args(const HeadShape& s, int64_t n_docs, int64_t qs, int64_t ks, double base,
                   float eps) {
  NormArgs a{};
  a.tn = make_turns(base, (int)s.d);
  a.n_tok = s.n_tok;
  a.qs = qs;
  a.ks = ks;
  a.hq = (int)s.hq;
  a.hkv = (int)s.hkv;
  a.n_docs = (int)n_docs;
  a.eps = eps;
  return a;
}

}  // namespace

int64_t qk_norm_rope_bwd_ctas() { return 148 * 4; }

cudaError_t launch_qk_norm_rope(const HeadShape& s, const int32_t* cu, int64_t n_docs,
                                const void* q, int64_t qs, const void* k, int64_t ks,
                                const void* wq, const void* wk, double base, float eps, void* qo,
                                void* ko, cudaStream_t st) {
  NormArgs a = make_args(s, n_docs, qs, ks, base, eps);
  if (s.dtype == MSA_BF16)
    return s.d == 128 ? run_fwd<__nv_bfloat16, 128>(a, q, k, cu, wq, wk, qo, ko, st)
                      : run_fwd<__nv_bfloat16, 64>(a, q, k, cu, wq, wk, qo, ko, st);
  return s.d == 128 ? run_fwd<float, 128>(a, q, k, cu, wq, wk, qo, ko, st)
                    : run_fwd<float, 64>(a, q, k, cu, wq, wk, qo, ko, st);
}

cudaError_t launch_qk_norm_rope_bwd(const HeadShape& s, const int32_t* cu, int64_t n_docs,
                                    const void* dq, const void* dk, int grad_dtype, const void* q,
                                    int64_t qs, const void* k, int64_t ks, const void* wq,
                                    const void* wk, double base, float eps, void* dqi, void* dki,
                                    float* dwq, float* dwk, float* part, cudaStream_t st) {
  NormArgs a = make_args(s, n_docs, qs, ks, base, eps);
  using B = __nv_bfloat16;
#define MSA_BWD(T, TG, D) \
  run_bwd<T, TG, D>(a, dq, dk, q, k, cu, wq, wk, dqi, dki, dwq, dwk, part, st)
  if (s.dtype == MSA_F32) return s.d == 128 ? MSA_BWD(float, float, 128) : MSA_BWD(float, float, 64);
  if (grad_dtype == MSA_F32) return s.d == 128 ? MSA_BWD(B, float, 128) : MSA_BWD(B, float, 64);
  return s.d == 128 ? MSA_BWD(B, B, 128) : MSA_BWD(B, B, 64);
#undef MSA_BWD
}

}  // namespace msa
