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
// they are under way, and the token's other rows are asked for to L2 at the warp's start: what
// a warp has in flight does not end at its registers (32K tokens of 32 + 8 heads of 128, bf16:
// forward 116 -> 106 us, and 103, 6.5 TB/s, with CTAs of one warp; gradient 235 -> 214 us, 6.3
// TB/s.  With the rows of the warp's next token asked for as well: 278).
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

constexpr int kWarps = 8;              // of a CTA of the gradient
constexpr int kUnroll = 4;            // row groups in flight per warp
constexpr int kFwdCtas = 16;          // forward: warps of an SM, a CTA each (8 a CTA: 4% slower)
constexpr int kFewWarps = 2;          // of a CTA with tokens of few heads
constexpr int kBwdCtas = 2;           // of the backward kernel on an SM

struct NormArgs {
  Turns tn;
  int64_t n_tok, qs, ks;              // packed tokens; token strides of q and k (elements)
  int hq, hkv, n_docs, split;         // split: warps a token's heads are dealt to
  float eps;
};

// The token's position in its document (0 for a token no document holds).
__device__ __forceinline__ int64_t token_pos(const int32_t* cu, int n_docs, int64_t t) {
  int64_t start, end;
  return warp_segment(cu, n_docs, t, start, end) < 0 ? 0 : t - start;
}

template <typename T, int D>
__global__ void __launch_bounds__(32, kFwdCtas)
qk_norm_rope_kernel(const T* q, const T* k, const int32_t* __restrict__ cu,
                    const T* __restrict__ wq, const T* __restrict__ wk, T* qo, T* ko,
                    const __grid_constant__ NormArgs a) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  const int64_t t = blockIdx.x / a.split;
  const int part = (int)(blockIdx.x - t * a.split);
  if (a.split == 1 && threadIdx.x == 0) {
    prefetch_l2(q + t * a.qs, a.hq * (int64_t)(D * sizeof(T)));
    prefetch_l2(k + t * a.ks, a.hkv * (int64_t)(D * sizeof(T)));
  }
  const int gq = (a.hq + R::kRows - 1) / R::kRows, gk = (a.hkv + R::kRows - 1) / R::kRows;
  float cs0[N], sn0[N];
  bool placed = false;
  auto place = [&](float (&cs)[N], float (&sn)[N]) {
    if (!placed) {
      lane_cos_sin<N, R::kLanes>(a.tn, token_pos(cu, a.n_docs, t), cs0, sn0);
      placed = true;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) { cs[e] = cs0[e]; sn[e] = sn0[e]; }
    return true;
  };
  turn_heads<T, D, kUnroll>(q + t * a.qs, qo + t * a.hq * D, D, a.hq, wq, a.eps, true, part,
                            a.split, gq, place);
  turn_heads<T, D, 2>(k + t * a.ks, ko + t * a.hkv * D, D, a.hkv, wk, a.eps, true,
                      first_group(gq, part, a.split) - gq, a.split, gk, place);
}

// Tokens of few heads (up to GQ row groups of queries and GK of keys): all of a token's rows are
// loaded before its position is looked up, and with fewer registers and CTAs of two warps more
// tokens are in flight (8 + 1 heads of 64, 32K tokens: 51 -> 22 us; 16 + 4 of 128, 20K: 47 -> 37;
// two to eight tokens a warp: slower than one).  It also beats a token's heads dealt to
// several warps (16 + 4 heads, 500 tokens: 3.9 us, 5.9), but for four groups and fewer
// tokens than SMs (100: 3.8, 3.6).
template <typename T, int D, int GQ, int GK>
__global__ void __launch_bounds__(kFewWarps * 32)
qk_norm_rope_few_kernel(const T* q, const T* k, const int32_t* __restrict__ cu,
                        const T* __restrict__ wq, const T* __restrict__ wk, T* qo, T* ko,
                        const __grid_constant__ NormArgs a) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  const int lane = threadIdx.x & 31, c = lane % R::kLanes, sub = lane / R::kLanes;
  const int64_t t = (int64_t)blockIdx.x * kFewWarps + (threadIdx.x >> 5);
  if (t >= a.n_tok) return;                               // whole warp
  uint4 qa[GQ], qb[GQ], ka[GK], kb[GK];
#pragma unroll
  for (int g = 0; g < GQ; ++g) {
    const int h = g * R::kRows + sub;
    load_row<T, D>(q + t * a.qs + (int64_t)h * D + c * N, h < a.hq, qa[g], qb[g]);
  }
#pragma unroll
  for (int g = 0; g < GK; ++g) {
    const int h = g * R::kRows + sub;
    load_row<T, D>(k + t * a.ks + (int64_t)h * D + c * N, h < a.hkv, ka[g], kb[g]);
  }
  float cs[N], sn[N], wa[N], wb[N];
  lane_cos_sin<N, R::kLanes>(a.tn, token_pos(cu, a.n_docs, t), cs, sn);
  Turn<T, D> turn;
  load_weights<T, D>(wq, c, wa, wb);
  turn.set(cs, sn, wa, wb);
#pragma unroll
  for (int g = 0; g < GQ; ++g) {
    const int h = g * R::kRows + sub;
    turn.template row<true>(qa[g], qb[g], a.eps, h < a.hq, qo + (t * a.hq + h) * D + c * N);
  }
  load_weights<T, D>(wk, c, wa, wb);
  turn.set(cs, sn, wa, wb);
#pragma unroll
  for (int g = 0; g < GK; ++g) {
    const int h = g * R::kRows + sub;
    turn.template row<true>(ka[g], kb[g], a.eps, h < a.hkv, ko + (t * a.hkv + h) * D + c * N);
  }
}

// ------------------------------------------------------------------ backward
// CTAs below nq take the queries, the others the keys (so a lane keeps one set of sums and
// enough warps fit); persistent warps, one token (or part of its heads) each at a time.
// part[cta][D]: the CTA's sums.
struct BwdArgs {
  NormArgs n;
  int nq, split_k;                    // n.split: of the queries
};

// A lane's part of a row and of its upstream gradient, as loaded.
template <typename T, typename TG>
struct GradRow {
  static constexpr int N = Vec16<T>::N, M = N / Vec16<TG>::N;   // 16-byte loads of a gradient
  uint4 xa, xb, ga[M], gb[M];

  __device__ __forceinline__ void load(const T* x, const TG* g, int half, bool on) {
    xa = xb = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < M; ++i) ga[i] = gb[i] = xa;
    if (!on) return;
    xa = ld16_once(x);
    xb = ld16_once(x + half);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      ga[i] = ld16_once(g + i * (N / M));
      gb[i] = ld16_once(g + half + i * (N / M));
    }
  }
};

// ONE: a token is one row group (split is 1); its next one's loads are issued before it is worked
// on (32K tokens of 8 + 1 heads of 64: 58 -> 51 us; 16K of 4 + 4 of 128: 44 -> 33).
template <typename T, typename TG, int D, bool ONE>
__global__ void __launch_bounds__(kWarps * 32, kBwdCtas)
qk_norm_rope_bwd_kernel(const TG* __restrict__ dq, const TG* __restrict__ dk,
                        const T* __restrict__ q, const T* __restrict__ k,
                        const int32_t* __restrict__ cu, const T* __restrict__ wq,
                        const T* __restrict__ wk, T* __restrict__ dqi, T* __restrict__ dki,
                        float* __restrict__ part, const __grid_constant__ BwdArgs b) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  __shared__ float s_dw[kWarps][D];
  const NormArgs& a = b.n;
  const int lane = threadIdx.x & 31, c = lane % R::kLanes, sub = lane / R::kLanes;
  const int warp = threadIdx.x >> 5;
  const bool keys = (int)blockIdx.x >= b.nq;
  const int cta = keys ? blockIdx.x - b.nq : blockIdx.x;
  const int n_cta = keys ? gridDim.x - b.nq : b.nq;
  const int heads = keys ? a.hkv : a.hq, split = keys ? b.split_k : a.split;
  const int64_t stride = keys ? a.ks : a.qs;
  const T* x0 = (keys ? k : q) + c * N;
  const TG* y0 = (keys ? dk : dq) + c * N;
  T* o0 = (keys ? dki : dqi) + c * N;
  const int groups = (heads + R::kRows - 1) / R::kRows;
  float wa[N], wb[N], acc_a[N], acc_b[N];
  load_weights<T, D>(keys ? wk : wq, c, wa, wb);
#pragma unroll
  for (int e = 0; e < N; ++e) acc_a[e] = acc_b[e] = 0.f;

  // one row: dx to out, the products for dw added to (ta, tb)
  auto row = [&](const GradRow<T, TG>& in, bool on, const float (&cs)[N], const float (&sn)[N],
                 float (&ta)[N], float (&tb)[N], T* out) {
    float xa[N], xb[N], ga[N], gb[N];
    Vec16<T>::unpack(in.xa, xa);
    Vec16<T>::unpack(in.xb, xb);
#pragma unroll
    for (int i = 0; i < GradRow<T, TG>::M; ++i) {
      Vec16<TG>::unpack(in.ga[i], ga + i * Vec16<TG>::N);
      Vec16<TG>::unpack(in.gb[i], gb + i * Vec16<TG>::N);
    }
    const float r = row_rstd<D, N, R::kLanes>(xa, xb, a.eps);
    float d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float g0 = fmaf(ga[e], cs[e], gb[e] * sn[e]);         // R^T dy of both halves
      const float g1 = fmaf(gb[e], cs[e], -(ga[e] * sn[e]));
      xa[e] *= r;
      xb[e] *= r;
      ta[e] = fmaf(g0, xa[e], ta[e]);
      tb[e] = fmaf(g1, xb[e], tb[e]);
      ga[e] = g0 * wa[e];
      gb[e] = g1 * wb[e];
      d0 = fmaf(ga[e], xa[e], d0);
      d1 = fmaf(gb[e], xb[e], d1);
    }
    const float dot = row_sum<R::kLanes>(d0 + d1) * (-1.f / D);
    if (!on) return;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      ga[e] = r * fmaf(xa[e], dot, ga[e]);
      gb[e] = r * fmaf(xb[e], dot, gb[e]);
    }
    store_n<T>(out, ga);
    store_n<T>(out + D / 2, gb);
  };

  const int64_t units = a.n_tok * split, step = (int64_t)n_cta * kWarps;
  int64_t unit = (int64_t)cta * kWarps + warp;
  if (ONE) {
    const bool there = sub < heads;
    auto load = [&](int64_t t) {
      GradRow<T, TG> x;
      x.load(x0 + t * stride + sub * D, y0 + (t * heads + sub) * D, D / 2, there && t < units);
      return x;
    };
    GradRow<T, TG> cur = load(unit);
    for (; unit < units; unit += step) {
      const GradRow<T, TG> next = load(unit + step);
      float cs[N], sn[N];
      lane_cos_sin<N, R::kLanes>(a.tn, token_pos(cu, a.n_docs, unit), cs, sn);
      row(cur, there, cs, sn, acc_a, acc_b, o0 + (unit * heads + sub) * D);
      cur = next;
    }
  } else {
    for (; unit < units; unit += step) {
      const int64_t t = unit / split;
      if (split == 1 && lane == 0) {
        prefetch_l2(x0 + t * stride, heads * (int64_t)(D * sizeof(T)));
        prefetch_l2(y0 + t * heads * D, heads * (int64_t)(D * sizeof(TG)));
      }
      float cs[N], sn[N];
      lane_cos_sin<N, R::kLanes>(a.tn, token_pos(cu, a.n_docs, t), cs, sn);
      float ta[N], tb[N];                                 // this token's heads
#pragma unroll
      for (int e = 0; e < N; ++e) ta[e] = tb[e] = 0.f;
      for (int g = (int)(unit - t * split); g < groups; g += split) {
        const int h = g * R::kRows + sub;
        GradRow<T, TG> x;
        x.load(x0 + t * stride + h * D, y0 + (t * heads + h) * D, D / 2, h < heads);
        row(x, h < heads, cs, sn, ta, tb, o0 + (t * heads + h) * D);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        acc_a[e] += ta[e];
        acc_b[e] += tb[e];
      }
    }
  }
  if (part == nullptr) return;
  // rows of the warp (lanes with the same c), then the warps of the CTA in order
#pragma unroll
  for (int e = 0; e < N; ++e) {
#pragma unroll
    for (int o = 16; o >= R::kLanes; o >>= 1) {
      acc_a[e] += __shfl_xor_sync(0xffffffffu, acc_a[e], o);
      acc_b[e] += __shfl_xor_sync(0xffffffffu, acc_b[e], o);
    }
    if (sub == 0) {
      s_dw[warp][c * N + e] = acc_a[e];
      s_dw[warp][D / 2 + c * N + e] = acc_b[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += s_dw[w][i];
    part[(int64_t)blockIdx.x * D + i] = s;
  }
}

// dw[i] = sum over CTAs of part[cta][i]: 32 columns a block, 32 slices of the CTAs.  Blocks below
// d / 32 sum the first nq CTAs (the queries'), the others the rest.
__global__ void __launch_bounds__(1024)
dw_sum_kernel(const float* __restrict__ part, int nq, int n_cta, int d, float* __restrict__ dwq,
              float* __restrict__ dwk) {
  __shared__ float s[32][33];
  // (launched programmatically: it is set up beside the kernel above, which lets it start when it
  // has ended)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const bool keys = (int)blockIdx.x >= d / 32;
  const int col = (blockIdx.x - (keys ? d / 32 : 0)) * 32 + x;
  float v = 0.f;
  const int end = keys ? n_cta : nq;
#pragma unroll 4
  for (int c = (keys ? nq : 0) + y; c < end; c += 32) v += part[(int64_t)c * d + col];
  s[y][x] = v;
  __syncthreads();
  if (y != 0) return;
  v = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += s[i][x];
  float* dst = keys ? dwk : dwq;
  if (dst != nullptr) dst[col] = v;
}

template <typename T, int D>
cudaError_t run_fwd(NormArgs& a, const void* q, const void* k, const int32_t* cu, const void* wq,
                    const void* wk, void* qo, void* ko, cudaStream_t st) {
  constexpr int kR = RowLayout<T, D>::kRows;
  a.split = head_split(a.n_tok, (a.hq + kR - 1) / kR + (a.hkv + kR - 1) / kR);
  const int gq = (a.hq + kR - 1) / kR, gk = (a.hkv + kR - 1) / kR;
  if (gk <= 2 && (gq <= 2 || (gq <= 4 && a.n_tok >= sm_count()))) {
    const unsigned few = (unsigned)((a.n_tok + kFewWarps - 1) / kFewWarps);
    auto launch = [&](auto* kernel) {
      kernel<<<few, kFewWarps * 32, 0, st>>>((const T*)q, (const T*)k, cu, (const T*)wq,
                                             (const T*)wk, (T*)qo, (T*)ko, a);
      return cudaGetLastError();
    };
    if (gq == 1) return launch(qk_norm_rope_few_kernel<T, D, 1, 1>);   // (gk <= gq)
    if (gq == 2)
      return gk == 1 ? launch(qk_norm_rope_few_kernel<T, D, 2, 1>)
                     : launch(qk_norm_rope_few_kernel<T, D, 2, 2>);
    return gk == 1 ? launch(qk_norm_rope_few_kernel<T, D, 4, 1>)
                   : launch(qk_norm_rope_few_kernel<T, D, 4, 2>);
  }
  qk_norm_rope_kernel<T, D><<<(unsigned)(a.n_tok * a.split), 32, 0, st>>>(
      (const T*)q, (const T*)k, cu, (const T*)wq, (const T*)wk, (T*)qo, (T*)ko, a);
  return cudaGetLastError();
}

template <typename T, typename TG, int D>
cudaError_t run_bwd(NormArgs& a, const void* dq, const void* dk, const void* q, const void* k,
                    const int32_t* cu, const void* wq, const void* wk, void* dqi, void* dki,
                    float* dwq, float* dwk, float* part, cudaStream_t st) {
  constexpr int kR = RowLayout<T, D>::kRows;
  BwdArgs b{};
  a.split = head_split(a.n_tok, (a.hq + kR - 1) / kR);
  b.split_k = head_split(a.n_tok, (a.hkv + kR - 1) / kR);
  // The CTAs that fit the GPU, dealt out by row groups plus one for a token's position and
  // angles (32768 tokens of 32 / 8 heads: 234 us; by rows alone 258); fewer where there is less
  // work.
  const int64_t cap = qk_norm_rope_bwd_ctas();
  const int64_t want_q = (a.n_tok * a.split + kWarps - 1) / kWarps;
  const int64_t want_k = (a.n_tok * b.split_k + kWarps - 1) / kWarps;
  const int gq = (a.hq + kR - 1) / kR + 1, gk = (a.hkv + kR - 1) / kR + 1;
  int64_t cap_q = cap * gq / (gq + gk);
  if (cap_q > cap - 1) cap_q = cap - 1;
  b.nq = (int)(want_q < cap_q ? want_q : cap_q);
  const int64_t nk = want_k < cap - cap_q ? want_k : cap - cap_q;
  b.n = a;
  const bool dw = dwq != nullptr || dwk != nullptr;
  const int grid = b.nq + (int)nk;
  const bool one = a.hq <= kR && a.split == 1;            // (hkv <= hq; then split_k is 1 as well)
  auto* kernel =
      one ? qk_norm_rope_bwd_kernel<T, TG, D, true> : qk_norm_rope_bwd_kernel<T, TG, D, false>;
  kernel<<<grid, kWarps * 32, 0, st>>>(
      (const TG*)dq, (const TG*)dk, (const T*)q, (const T*)k, cu, (const T*)wq, (const T*)wk,
      (T*)dqi, (T*)dki, dw ? part : nullptr, b);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dw) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = 2 * D / 32;
  cfg.blockDim = 1024;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dw_sum_kernel, (const float*)part, b.nq, grid, D, dwq, dwk);
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

int64_t qk_norm_rope_bwd_ctas() { return 148 * kBwdCtas; }

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
  if (s.dtype == MSA_F32)
    return s.d == 128 ? MSA_BWD(float, float, 128) : MSA_BWD(float, float, 64);
  if (grad_dtype == MSA_F32) return s.d == 128 ? MSA_BWD(B, float, 128) : MSA_BWD(B, float, 64);
  return s.d == 128 ? MSA_BWD(B, B, 128) : MSA_BWD(B, B, 64);
#undef MSA_BWD
}

}  // namespace msa
