// Attention of new tokens over a paged cache: which kernel takes which sequences, and the
// kernel that joins the parts of items that were cut (see paged.cuh).
#include "paged.cuh"

namespace msa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Joins the parts of the item that CTA blockIdx.x began and did not finish: one warp a row.
template <typename T, int D>
__global__ void __launch_bounds__(128)
paged_combine_kernel(PagedParts parts, int rows, T* __restrict__ o, float* __restrict__ lse,
                     const __grid_constant__ PagedAttn a) {
  const int4 rec = parts.rec[blockIdx.x];
  if (rec.w == 0) return;
  constexpr int E = D / 32;           // columns of a lane
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 4 + (threadIdx.x >> 5);
  const int rt = rec.z & ~(1 << 30);
  const SeqView v = load_seq(a, rec.x);
  const int t_in = rt * a.tt + row / a.G, h = row % a.G;
  if (row >= rows || row >= a.tt * a.G || t_in >= v.n) return;
  const int64_t slot0 = 2 * (int64_t)blockIdx.x + (rec.z >> 30 & 1);
  auto slot = [&](int i) -> int64_t { return i == 0 ? slot0 : 2 * ((int64_t)blockIdx.x + i); };
  float mx = -CUDART_INF_F;
  for (int i = lane; i < rec.w; i += 32) mx = fmaxf(mx, parts.ml[slot(i) * rows + row].x);
  mx = warp_max(mx);
  if (mx == -CUDART_INF_F) mx = 0.f;
  float l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < rec.w; ++i) {
    const float2 ml = parts.ml[slot(i) * rows + row];
    const float w = exp2f(ml.x - mx);
    const float* src = parts.o + (slot(i) * rows + row) * D + lane * E;
    l = fmaf(ml.y, w, l);
    if (E == 4) {
      const float4 y = *reinterpret_cast<const float4*>(src);
      acc[0] = fmaf(y.x, w, acc[0]);
      acc[1] = fmaf(y.y, w, acc[1]);
      acc[E - 2] = fmaf(y.z, w, acc[E - 2]);
      acc[E - 1] = fmaf(y.w, w, acc[E - 1]);
    } else {
      const float2 y = *reinterpret_cast<const float2*>(src);
      acc[0] = fmaf(y.x, w, acc[0]);
      acc[1] = fmaf(y.y, w, acc[1]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const int64_t qrow = (v.tok0 + t_in) * a.hq + rec.y * a.G + h;
#pragma unroll
  for (int e = 0; e < E; ++e) o[qrow * D + lane * E + e] = from_f32<T>(acc[e] * inv);
  if (lane == 0 && lse != nullptr)
    lse[qrow] = l > 0.f ? (mx + log2f(l)) * kLn2 : -CUDART_INF_F;
}

PagedParts parts_of(char* ws) {
  PagedParts p;
  p.rec = reinterpret_cast<int4*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + kPagedCtas * sizeof(int4));
  p.o = reinterpret_cast<float*>(ws + kPagedCtas * sizeof(int4) +
                                 (size_t)2 * kPagedCtas * kPagedMaxRows * sizeof(float2));
  return p;
}

}  // namespace

size_t paged_attn_ws_bytes(const HeadShape& s) {
  return kPagedCtas * sizeof(int4) +
         (size_t)2 * kPagedCtas * kPagedMaxRows * (sizeof(float2) + s.d * sizeof(float));
}

int paged_grid() { return sm_count() < kPagedCtas ? sm_count() : kPagedCtas; }

cudaError_t launch_paged_combine(const HeadShape& s, const PagedAttn& a, int grid, int rows,
                                 const PagedParts& parts, void* o, float* lse, cudaStream_t st) {
  const dim3 g(grid, (a.tt * a.G + 3) / 4);
  using B = __nv_bfloat16;
  if (s.dtype == MSA_BF16) {
    if (s.d == 128) paged_combine_kernel<B, 128><<<g, 128, 0, st>>>(parts, rows, (B*)o, lse, a);
    else paged_combine_kernel<B, 64><<<g, 128, 0, st>>>(parts, rows, (B*)o, lse, a);
  } else {
    if (s.d == 128)
      paged_combine_kernel<float, 128><<<g, 128, 0, st>>>(parts, rows, (float*)o, lse, a);
    else
      paged_combine_kernel<float, 64><<<g, 128, 0, st>>>(parts, rows, (float*)o, lse, a);
  }
  return cudaGetLastError();
}

cudaError_t launch_paged_attn(const HeadShape& s, const PagedShape& g, int64_t max_new,
                              float scale, const void* q, int64_t qs, const void* kp,
                              const void* vp, void* o, float* lse, char* ws, int* err,
                              cudaStream_t st) {
  PagedAttn a{};
  a.g = g;
  a.n_tok = s.n_tok;
  a.qs = qs;
  a.hq = (int)s.hq;
  a.hkv = (int)s.hkv;
  a.G = (int)(s.hq / s.hkv);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.min_new = 1;
  a.max_new = INT32_MAX;
  if (max_new < 1 || max_new > s.n_tok) max_new = s.n_tok;
  const int64_t rows = max_new * a.G;
  const PagedParts parts = parts_of(ws);
  if (s.dtype == MSA_F32)
    return launch_paged_simt(s, a, rows <= 16 ? 16 : 64, q, kp, vp, o, lse, parts, err, st);
  return launch_paged_few(s, a, rows <= 16, q, kp, vp, o, lse, parts, err, st);
}

}  // namespace msa
