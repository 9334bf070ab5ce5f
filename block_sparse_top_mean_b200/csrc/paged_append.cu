// Append of new tokens to a paged key/value cache, with the norm and the rotation on the way.
//
// Token i of sequence s sits at position pos = kv_lens[s] - n_s + i (kv_lens counts the n_s
// new tokens) and goes to slot pos % page of page page_table[s][pos / page]:
//   k_pages[slot] = R(pos) norm(k),  v_pages[slot] = v,  q_out = R(pos) norm(q).
// Norm and rotation are those of qk_norm_rope.cu; either can be left out.
//
// Single tokens (64 sequences: 1.6 MB) are bound by the launch and by the chain cu_seqlens
// -> kv_lens -> page_table -> store; chunks by HBM (each element read and written once).  A
// warp takes a token's heads, or a part of them when there are few tokens, with the rows'
// loads under way while that chain is walked.
#include "paged.cuh"
#include "rotary.cuh"

namespace msa {
namespace {

constexpr int kWarps = 4;
constexpr int kUnroll = 4;            // rows in flight per lane

struct AppendArgs {
  Turns tn;
  int64_t n_tok, qs, ks, vs;          // packed tokens; token strides (elements)
  PagedShape g;
  int hq, hkv, split, rotate;
  float eps;                          // 0: no norm
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
paged_append_kernel(const T* q, const T* k, const T* v, const T* __restrict__ wq,
                    const T* __restrict__ wk, T* __restrict__ kp, T* __restrict__ vp, T* qo,
                    int* err, const __grid_constant__ AppendArgs a) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  const int lane = threadIdx.x & 31, c = lane % R::kLanes, sub = lane / R::kLanes;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit / a.split;
  if (t >= a.n_tok) return;                               // whole warp
  const int part = (int)(unit - t * a.split);
  const int hk = a.hq + a.hkv, heads = hk + a.hkv;        // rows: queries, keys, values
  float cs[N], sn[N];
  bool placed = false;
  int64_t slot = -1;                                      // row of head 0 in the pools
  for (int h0 = part * R::kRows; h0 < heads; h0 += a.split * R::kRows * kUnroll) {
    uint4 ra[kUnroll], rb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * a.split * R::kRows + sub;
      if (h >= heads) continue;
      const T* row = h < a.hq   ? q + t * a.qs + (int64_t)h * D
                     : h < hk ? k + t * a.ks + (int64_t)(h - a.hq) * D
                              : v + t * a.vs + (int64_t)(h - hk) * D;
      ra[u] = ld16_once(row + c * N);
      rb[u] = ld16_once(row + D / 2 + c * N);
    }
    if (!placed) {
      const int s = warp_segment(a.g.cu, (int)a.g.n_seqs, t);
      if (s < 0) return;                                  // behind the last sequence
      const int64_t c0 = __ldg(a.g.cu + s), c1 = __ldg(a.g.cu + s + 1);
      const int64_t pos = (int64_t)__ldg(a.g.kv_lens + s) - (c1 - c0) + (t - c0);
      if (pos >= 0 && pos < a.g.max_pages * a.g.page) {
        const int64_t pg = __ldg(a.g.table + (int64_t)s * a.g.max_pages + pos / a.g.page);
        if (pg >= 0 && pg < a.g.n_pages)
          slot = pg * a.hkv * a.g.page + pos % a.g.page;
      }
      if (slot < 0 && lane == 0) set_device_error(err, MSA_DEVERR_PAGE_RANGE);
      if (a.rotate) {
        lane_cos_sin<N>(a.tn, c, pos, cs, sn);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) { cs[e] = 1.f; sn[e] = 0.f; }
      }
      placed = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * a.split * R::kRows + sub;
      float xa[N], xb[N];
      const bool on = h < heads;
      Vec16<T>::unpack(on ? ra[u] : make_uint4(0, 0, 0, 0), xa);
      Vec16<T>::unpack(on ? rb[u] : make_uint4(0, 0, 0, 0), xb);
      const float r = a.eps > 0.f ? row_rstd<D, N, R::kLanes>(xa, xb, a.eps) : 1.f;
      if (!on || (h >= a.hq && slot < 0)) continue;
      if (h >= hk) {                                      // values are copied
        T* out = vp + (slot + (int64_t)(h - hk) * a.g.page) * D;
        *reinterpret_cast<uint4*>(out + c * N) = ra[u];
        *reinterpret_cast<uint4*>(out + D / 2 + c * N) = rb[u];
        continue;
      }
      const T* w = h < a.hq ? wq : wk;
      if (a.eps > 0.f) {
        float wa[N], wb[N];
        if (w != nullptr) {
          Vec16<T>::unpack(ldg16(w + c * N), wa);
          Vec16<T>::unpack(ldg16(w + D / 2 + c * N), wb);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) wa[e] = wb[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < N; ++e) {
          xa[e] = xa[e] * r * wa[e];
          xb[e] = xb[e] * r * wb[e];
        }
      }
      T* out = h < a.hq ? qo + (t * a.hq + h) * D : kp + (slot + (int64_t)(h - a.hq) * a.g.page) * D;
      float ya[N], yb[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        ya[e] = xa[e] * cs[e] - xb[e] * sn[e];
        yb[e] = xb[e] * cs[e] + xa[e] * sn[e];
      }
      store_n<T>(out + c * N, ya);
      store_n<T>(out + D / 2 + c * N, yb);
    }
  }
}

template <typename T, int D>
cudaError_t run(AppendArgs& a, const void* q, const void* k, const void* v, const void* wq,
                const void* wk, void* kp, void* vp, void* qo, int* err, cudaStream_t st) {
  const int rows = RowLayout<T, D>::kRows;
  const int groups = (a.hq + 2 * a.hkv + rows - 1) / rows;
  const int64_t want = (int64_t)sm_count() * 32;
  a.split = 1;
  while (a.split < groups && a.n_tok * a.split < want) a.split *= 2;
  if (a.split > groups) a.split = groups;
  const int64_t grid = (a.n_tok * a.split + kWarps - 1) / kWarps;
  paged_append_kernel<T, D><<<(unsigned)grid, kWarps * 32, 0, st>>>(
      (const T*)q, (const T*)k, (const T*)v, (const T*)wq, (const T*)wk, (T*)kp, (T*)vp, (T*)qo,
      err, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const HeadShape& s, const PagedShape& g, const void* q, int64_t qs,
                                const void* k, int64_t ks, const void* v, int64_t vs,
                                const void* wq, const void* wk, double base, float eps, void* kp,
                                void* vp, void* qo, int* err, cudaStream_t st) {
  AppendArgs a{};
  a.tn = make_turns(base, (int)s.d);
  a.n_tok = s.n_tok;
  a.qs = qs;
  a.ks = ks;
  a.vs = vs;
  a.g = g;
  a.hq = q != nullptr ? (int)s.hq : 0;
  a.hkv = (int)s.hkv;
  a.rotate = base > 0.0;
  a.eps = eps;
  using B = __nv_bfloat16;
  if (s.dtype == MSA_BF16)
    return s.d == 128 ? run<B, 128>(a, q, k, v, wq, wk, kp, vp, qo, err, st)
                      : run<B, 64>(a, q, k, v, wq, wk, kp, vp, qo, err, st);
  return s.d == 128 ? run<float, 128>(a, q, k, v, wq, wk, kp, vp, qo, err, st)
                    : run<float, 64>(a, q, k, v, wq, wk, kp, vp, qo, err, st);
}

}  // namespace msa
