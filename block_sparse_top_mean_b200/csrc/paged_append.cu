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
// loads under way while that chain is walked, and its other rows on their way to L2 (55 -> 52
// us).  32 + 2 x 8 heads of 128, bf16: 11.5K tokens into pages of 16 53 us, 5.4 TB/s; 15K into
// pages of 256 80 us, 5.9 TB/s (a head's rows of a page follow one another, 256 bytes each).  Two
// warps a token look it up twice: 67 us; two tokens a warp: 63.
#include "paged.cuh"
#include "rotary.cuh"

namespace msa {
namespace {

constexpr int kCtas = 16;             // warps of an SM, a CTA each (8 CTAs of 2 warps: 3% slower)
constexpr int kUnroll = 4;            // row groups of the queries in flight per warp
constexpr int kValues = 2;            // and of the values
constexpr int kFewWarps = 2;          // of a CTA with tokens of few heads

struct AppendArgs {
  Turns tn;
  int64_t n_tok, qs, ks, vs;          // packed tokens; token strides (elements)
  PagedShape g;
  int hq, hkv, split, rotate;
  float eps;                          // 0: no norm
};

// Where token t goes.  The whole warp calls it.
struct Place {
  bool mine;                          // a sequence holds the token
  int64_t slot, pos;                  // row of KV head 0 in the pools (-1: none), position
};
__device__ __forceinline__ Place find_place(const AppendArgs& a, int64_t t, int* err) {
  const int lane = threadIdx.x & 31, n = (int)a.g.n_seqs;
  Place p{false, -1, 0};
  // (the lengths of up to 32 sequences are fetched beside the search)
  const int kv = n <= 32 ? __ldg(a.g.kv_lens + min(lane, n - 1)) : 0;
  int64_t c0, c1;
  const int s = warp_segment(a.g.cu, n, t, c0, c1);
  if (s < 0) return p;                                    // behind the last sequence
  p.mine = true;
  const int len = n <= 32 ? __shfl_sync(0xffffffffu, kv, s) : __ldg(a.g.kv_lens + s);
  p.pos = (int64_t)len - (c1 - c0) + (t - c0);
  if (p.pos >= 0 && p.pos < a.g.max_pages * a.g.page) {
    const int64_t pg = __ldg(a.g.table + (int64_t)s * a.g.max_pages + p.pos / a.g.page);
    if (pg >= 0 && pg < a.g.n_pages) p.slot = pg * a.hkv * a.g.page + p.pos % a.g.page;
  }
  if (p.slot < 0 && lane == 0) set_device_error(err, MSA_DEVERR_PAGE_RANGE);
  return p;
}

template <typename T, int D>
__global__ void __launch_bounds__(32, kCtas)
paged_append_kernel(const T* q, const T* k, const T* v, const T* __restrict__ wq,
                    const T* __restrict__ wk, T* __restrict__ kp, T* __restrict__ vp, T* qo,
                    int* err, const __grid_constant__ AppendArgs a) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  const int lane = threadIdx.x, c = lane % R::kLanes, sub = lane / R::kLanes;
  const int64_t t = blockIdx.x / a.split;
  const int part = (int)(blockIdx.x - t * a.split);
  if (a.split == 1 && lane < 3) {
    const T* row = lane == 0 ? q + t * a.qs : lane == 1 ? k + t * a.ks : v + t * a.vs;
    const int heads = lane == 0 ? a.hq : a.hkv;
    if (heads > 0) prefetch_l2(row, heads * (int64_t)(D * sizeof(T)));
  }
  const int gq = (a.hq + R::kRows - 1) / R::kRows, gk = (a.hkv + R::kRows - 1) / R::kRows;
  Place at{false, -1, 0};
  bool placed = false, angles = false;
  float cs0[N], sn0[N];
  auto find = [&]() {
    if (!placed) at = find_place(a, t, err);
    placed = true;
  };
  auto place = [&](float (&cs)[N], float (&sn)[N]) {
    find();
    if (!angles && a.rotate) {
      lane_cos_sin<N, R::kLanes>(a.tn, at.pos, cs0, sn0);
      angles = true;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      cs[e] = a.rotate ? cs0[e] : 1.f;
      sn[e] = a.rotate ? sn0[e] : 0.f;
    }
  };
  turn_heads<T, D, kUnroll>(q + t * a.qs, qo + t * a.hq * D, D, a.hq, wq, a.eps, a.rotate, part,
                            a.split, gq, [&](float (&cs)[N], float (&sn)[N]) {
                              place(cs, sn);
                              return at.mine;
                            });
  // The values are copied: their rows are asked for before the keys' turn, kValues groups at a
  // time, and stored behind it.
  const int g0 = first_group(gq, part, a.split) - gq;
  int gv = first_group(gq + gk, part, a.split) - gq - gk;
  uint4 va[kValues], vb[kValues];
  auto load_values = [&]() {
#pragma unroll
    for (int u = 0; u < kValues; ++u) {
      const int h = (gv + u * a.split) * R::kRows + sub;
      if (h >= a.hkv) continue;
      const T* row = v + t * a.vs + (int64_t)h * D;
      va[u] = ld16_once(row + c * N);
      vb[u] = ld16_once(row + D / 2 + c * N);
    }
  };
  load_values();
  // (where the keys go is known only after find(): the rows are placed from the slot)
  if (g0 < gk) {
    find();
    turn_heads<T, D, 2>(k + t * a.ks, kp + max(at.slot, (int64_t)0) * D, a.g.page * D, a.hkv, wk,
                        a.eps, a.rotate, g0, a.split, gk, [&](float (&cs)[N], float (&sn)[N]) {
                          place(cs, sn);
                          return at.slot >= 0;
                        });
  }
  while (gv < gk) {
    find();                                               // (all lanes)
#pragma unroll
    for (int u = 0; u < kValues; ++u) {
      const int h = (gv + u * a.split) * R::kRows + sub;
      if (at.slot < 0 || h >= a.hkv) continue;
      T* out = vp + (at.slot + (int64_t)h * a.g.page) * D;
      *reinterpret_cast<uint4*>(out + c * N) = va[u];
      *reinterpret_cast<uint4*>(out + D / 2 + c * N) = vb[u];
    }
    gv += kValues * a.split;
    load_values();
  }
}

// Tokens of few heads (up to GQ row groups of queries and GK of keys): all of a token's rows are
// loaded before its place is looked up, as in qk_norm_rope_few_kernel (24K tokens of 4 + 4 heads of
// 128: 59 -> 36 us; 18K of 8 + 1 of 64: 40 -> 20; 15K of 16 + 4 of 128: 53 -> 47).
template <typename T, int D, int GQ, int GK>
__global__ void __launch_bounds__(kFewWarps * 32)
paged_append_few_kernel(const T* q, const T* k, const T* v, const T* __restrict__ wq,
                        const T* __restrict__ wk, T* __restrict__ kp, T* __restrict__ vp, T* qo,
                        int* err, const __grid_constant__ AppendArgs a) {
  using R = RowLayout<T, D>;
  constexpr int N = R::N;
  const int lane = threadIdx.x & 31, c = lane % R::kLanes, sub = lane / R::kLanes;
  const int64_t t = (int64_t)blockIdx.x * kFewWarps + (threadIdx.x >> 5);
  if (t >= a.n_tok) return;                               // whole warp
  uint4 qa[GQ], qb[GQ], ka[GK], kb[GK], va[GK], vb[GK];
#pragma unroll
  for (int g = 0; g < GQ; ++g) {
    const int h = g * R::kRows + sub;
    load_row<T, D>(q + t * a.qs + (int64_t)h * D + c * N, h < a.hq, qa[g], qb[g]);
  }
#pragma unroll
  for (int g = 0; g < GK; ++g) {
    const int h = g * R::kRows + sub;
    load_row<T, D>(k + t * a.ks + (int64_t)h * D + c * N, h < a.hkv, ka[g], kb[g]);
    load_row<T, D>(v + t * a.vs + (int64_t)h * D + c * N, h < a.hkv, va[g], vb[g]);
  }
  const Place at = find_place(a, t, err);
  if (!at.mine) return;
  float cs[N], sn[N], wa[N], wb[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    cs[e] = 1.f;
    sn[e] = 0.f;
  }
  if (a.rotate) lane_cos_sin<N, R::kLanes>(a.tn, at.pos, cs, sn);
  Turn<T, D> turn;
  auto rows = [&](auto rot) {
    if (a.hq > 0) {
      load_weights<T, D>(wq, c, wa, wb);
      turn.set(cs, sn, wa, wb);
#pragma unroll
      for (int g = 0; g < GQ; ++g) {
        const int h = g * R::kRows + sub;
        turn.template row<rot.value>(qa[g], qb[g], a.eps, h < a.hq,
                                     qo + (t * a.hq + h) * D + c * N);
      }
    }
    if (at.slot < 0) return;
    load_weights<T, D>(wk, c, wa, wb);
    turn.set(cs, sn, wa, wb);
#pragma unroll
    for (int g = 0; g < GK; ++g) {
      const int h = g * R::kRows + sub;
      const int64_t row = (at.slot + (int64_t)h * a.g.page) * D + c * N;
      turn.template row<rot.value>(ka[g], kb[g], a.eps, h < a.hkv, kp + row);
      if (h >= a.hkv) continue;
      *reinterpret_cast<uint4*>(vp + row) = va[g];
      *reinterpret_cast<uint4*>(vp + row + D / 2) = vb[g];
    }
  };
  if (a.rotate) rows(std::true_type{});
  else rows(std::false_type{});
}

template <typename T, int D>
cudaError_t run(AppendArgs& a, const void* q, const void* k, const void* v, const void* wq,
                const void* wk, void* kp, void* vp, void* qo, int* err, cudaStream_t st) {
  constexpr int kR = RowLayout<T, D>::kRows;
  const int gq = (a.hq + kR - 1) / kR, gk = (a.hkv + kR - 1) / kR;
  a.split = head_split(a.n_tok, gq + 2 * gk);
  if (gk <= 2 && (gq <= 2 || (gq <= 4 && a.n_tok >= sm_count()))) {
    const unsigned few = (unsigned)((a.n_tok + kFewWarps - 1) / kFewWarps);
    auto launch = [&](auto* kernel) {
      kernel<<<few, kFewWarps * 32, 0, st>>>((const T*)q, (const T*)k, (const T*)v, (const T*)wq,
                                             (const T*)wk, (T*)kp, (T*)vp, (T*)qo, err, a);
      return cudaGetLastError();
    };
    if (gq <= 1 && gk == 1) return launch(paged_append_few_kernel<T, D, 1, 1>);
    if (gq <= 2)
      return gk == 1 ? launch(paged_append_few_kernel<T, D, 2, 1>)
                     : launch(paged_append_few_kernel<T, D, 2, 2>);
    return gk == 1 ? launch(paged_append_few_kernel<T, D, 4, 1>)
                   : launch(paged_append_few_kernel<T, D, 4, 2>);
  }
  paged_append_kernel<T, D><<<(unsigned)(a.n_tok * a.split), 32, 0, st>>>(
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
