// Attention of new tokens over a paged cache: which kernel takes which sequences, and the
// kernel that joins the parts of items that were cut (see paged.cuh).
#include <algorithm>

#include "paged.cuh"

namespace msa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// Join the parts of the item that CTA blockIdx.x began and did not finish, in their order:
// with m the largest of the parts' maxima, o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// The parts come from L2, so what counts is the chain record -> maxima -> outputs, and that it
// starts as the attention kernel ends (programmatic dependent launch: the wait is for that
// kernel's results).
__device__ __forceinline__ int64_t part_slot(const int4& rec, int i) {
  return i == 0 ? 2 * (int64_t)blockIdx.x + (rec.z & 1) : 2 * ((int64_t)blockIdx.x + i);
}

__device__ __forceinline__ int64_t part_qrow(const int4& rec, int row, int G, int hq) {
  return ((int64_t)rec.y << 32 | (uint32_t)rec.x) + (int64_t)(row / G) * hq + row % G;
}

template <typename T, int D>
__device__ __forceinline__ void store_joined(T* o, float* lse, int64_t qrow, int lane,
                                             const float (&acc)[D / 32], float mx, float l) {
  constexpr int E = D / 32;
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[qrow * D + lane * E + e] = from_f32<T>(acc[e] * inv);
  if (lane == 0 && lse != nullptr)
    lse[qrow] = l != 0.f ? (mx + log2f(l)) * kLn2 : -CUDART_INF_F;
}

template <int E>
__device__ __forceinline__ void load_part(float (&y)[E], const float* src) {
  if (E == 4) *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(src);
  else *reinterpret_cast<float2*>(y) = *reinterpret_cast<const float2*>(src);
}

// Few rows: an item may have a part from every CTA.  A block a row, each of its eight warps
// over every eighth part.
template <typename T, int D>
__global__ void __launch_bounds__(256)
paged_combine_parts_kernel(PagedParts parts, int rows, T* __restrict__ o,
                           float* __restrict__ lse, int G, int hq) {
  constexpr int E = D / 32, W = 8;    // columns of a lane, warps
  __shared__ float s_acc[W][D];
  __shared__ float s_l[W];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = parts.rec[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.y, n = rec.w;
  if (n == 0 || row >= (rec.z >> 1) * G) return;          // whole block
  float2 ml = make_float2(-CUDART_INF_F, 0.f);
  float y[E] = {};
  if (warp < n) {                                         // before the maximum is known
    const int64_t at = part_slot(rec, warp) * rows + row;
    ml = parts.ml[at];
    load_part<E>(y, parts.o + at * D + lane * E);
  }
  float mx = -CUDART_INF_F;
  for (int i = lane; i < n; i += 32)
    mx = fmaxf(mx, parts.ml[part_slot(rec, i) * rows + row].x);
  mx = warp_max(mx);
  const float ref = mx == -CUDART_INF_F ? 0.f : mx;
  float w = exp2f(ml.x - ref), l = ml.y * w, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = y[e] * w;
#pragma unroll 4
  for (int i = warp + W; i < n; i += W) {
    const int64_t at = part_slot(rec, i) * rows + row;
    ml = parts.ml[at];
    load_part<E>(y, parts.o + at * D + lane * E);
    w = exp2f(ml.x - ref);
    l = fmaf(ml.y, w, l);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(y[e], w, acc[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][lane * E + e] = acc[e];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < W; ++w) {
    l += s_l[w];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += s_acc[w][lane * E + e];
  }
  store_joined<T, D>(o, lse, part_qrow(rec, row, G, hq), lane, acc, mx, l);
}

// Many rows: a warp a row.  Up to three parts (a cut item has two, and mostly no more) are asked
// for before their maxima are known; of more, lane i holds the maximum and the weight of part i
// and the outputs come four at a time (64 tokens over 30000 keys: 36 us, 53 one by one).
template <typename T, int D>
__global__ void __launch_bounds__(256, 8)
paged_combine_rows_kernel(PagedParts parts, int rows, T* __restrict__ o,
                          float* __restrict__ lse, int G, int hq) {
  constexpr int E = D / 32, B = 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 rec = parts.rec[blockIdx.x];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = rec.w;
  const int row = blockIdx.y * 8 + warp;
  if (n == 0 || row >= (rec.z >> 1) * G) return;
  auto at = [&](int i) -> int64_t { return part_slot(rec, i) * rows + row; };
  auto part = [&](float (&y)[E], int i) { load_part<E>(y, parts.o + at(i) * D + lane * E); };
  float acc[E], y[B][E];
  if (n <= 3) {
    const float2 m0 = parts.ml[at(0)], m1 = parts.ml[at(1)];
    part(acc, 0);
    part(y[0], 1);
    float2 m2 = make_float2(-CUDART_INF_F, 0.f);
    if (n == 3) {
      m2 = parts.ml[at(2)];
      part(y[1], 2);
    }
    const float mx = fmaxf(fmaxf(m0.x, m1.x), m2.x), ref = mx == -CUDART_INF_F ? 0.f : mx;
    const float w0 = exp2f(m0.x - ref), w1 = exp2f(m1.x - ref), w2 = exp2f(m2.x - ref);
    float l = fmaf(m1.y, w1, m0.y * w0);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(y[0][e], w1, acc[e] * w0);
    if (n == 3) {
      l = fmaf(m2.y, w2, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(y[1][e], w2, acc[e]);
    }
    store_joined<T, D>(o, lse, part_qrow(rec, row, G, hq), lane, acc, mx, l);
    return;
  }
  float2 ml = make_float2(-CUDART_INF_F, 0.f);
  if (lane < n) ml = parts.ml[at(lane)];
  part(acc, 0);
  part(y[0], 1);
  float mx = ml.x;
  for (int i = 32 + lane; i < n; i += 32) mx = fmaxf(mx, parts.ml[at(i)].x);
  mx = warp_max(mx);
  const float ref = mx == -CUDART_INF_F ? 0.f : mx;
  float w = exp2f(ml.x - ref), l = ml.y * w;
  const float w0 = __shfl_sync(0xffffffffu, w, 0), w1 = __shfl_sync(0xffffffffu, w, 1);
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = fmaf(y[0][e], w1, acc[e] * w0);
  for (int i0 = 0; i0 < n; i0 += 32) {
    if (i0 > 0) {                                         // the next 32 parts' weights
      ml = i0 + lane < n ? parts.ml[at(i0 + lane)] : make_float2(-CUDART_INF_F, 0.f);
      w = exp2f(ml.x - ref);
      l = fmaf(ml.y, w, l);
    }
    for (int i = i0 == 0 ? 2 : i0; i < min(n, i0 + 32); i += B) {
#pragma unroll
      for (int b = 0; b < B; ++b) part(y[b], min(i + b, n - 1));
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const float f = __shfl_sync(0xffffffffu, w, (i + b) & 31);
        if (i + b < min(n, i0 + 32)) {
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] = fmaf(y[b][e], f, acc[e]);
        }
      }
    }
  }
  l = warp_sum(l);
  store_joined<T, D>(o, lse, part_qrow(rec, row, G, hq), lane, acc, mx, l);
}

template <typename T, int D>
cudaError_t run_combine(const PagedAttn& a, int grid, int rows, const PagedParts& parts, void* o,
                        float* lse, cudaStream_t st) {
  const bool few = rows <= 16;
  const int used = a.tt * a.G;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, few ? used : (used + 7) / 8);
  cfg.blockDim = 256;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, paged_combine_parts_kernel<T, D>, parts, rows, (T*)o,
                                  lse, a.G, a.hq)
             : cudaLaunchKernelEx(&cfg, paged_combine_rows_kernel<T, D>, parts, rows, (T*)o, lse,
                                  a.G, a.hq);
}

PagedParts parts_of(char* ws) {
  PagedParts p;
  p.rec = reinterpret_cast<int4*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + kPagedRecs * sizeof(int4));
  p.o = reinterpret_cast<float*>(ws + kPagedRecs * sizeof(int4) +
                                 (size_t)2 * kPagedCtas * kPagedMaxRows * sizeof(float2));
  return p;
}

}  // namespace

size_t paged_attn_ws_bytes(const HeadShape& s) {
  return kPagedRecs * sizeof(int4) +
         (size_t)2 * kPagedCtas * kPagedMaxRows * (sizeof(float2) + s.d * sizeof(float));
}

cudaError_t raise_smem(const void* kernel, size_t bytes, DeviceOnce* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || done->done(dev)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done->mark(dev);
  return e;
}

int paged_grid() { return sm_count() < kPagedCtas ? sm_count() : kPagedCtas; }

cudaError_t launch_paged_combine(const HeadShape& s, const PagedAttn& a, int grid, int rows,
                                 const PagedParts& parts, void* o, float* lse, cudaStream_t st) {
  using B = __nv_bfloat16;
  if (s.dtype == MSA_BF16)
    return s.d == 128 ? run_combine<B, 128>(a, grid, rows, parts, o, lse, st)
                      : run_combine<B, 64>(a, grid, rows, parts, o, lse, st);
  return s.d == 128 ? run_combine<float, 128>(a, grid, rows, parts, o, lse, st)
                    : run_combine<float, 64>(a, grid, rows, parts, o, lse, st);
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
    return launch_paged_f32(s, a, rows <= 8 ? (int)rows : 64, q, kp, vp, o, lse, parts, err, st);
  // Up to 16 rows the mma.sync kernel keeps up with the cache's stream; above, the tensor cores'
  // 256-row tiles do better even where few of their rows hold a query (8 sequences x 16000 keys,
  // 4 heads a group: 2 tokens 87 us on the first, 109 on the second; 4 tokens 96 and 107; 5 tokens
  // 123 on the second, 202 on mma.sync with 64 rows a tile).
  if (rows <= 16) return launch_paged_step(s, a, (int)rows, q, kp, vp, o, lse, parts, err, st);
  // A chunk among generated tokens (the others' average says so): single tokens would fill a few
  // rows of a 256-row tile each, so they get a launch of their own, where the caches are large
  // enough to pay for it; the host knows what the tables and the pools can hold (48 tokens of 512
  // keys each, 32 / 8 heads of 128, and a chunk of 1024: 115 us, 107 in one launch; of 2048 keys,
  // 400 MB: 162 and 163; of 8192: 334 and 396).
  const int small = a.G <= 8 ? 8 : 16;
  const int64_t table_keys = (g.n_seqs - 1) * std::min<int64_t>(g.max_pages * g.page, INT32_MAX);
  const int64_t keys = std::min(table_keys, g.n_pages * g.page);
  if (g.n_seqs > 1 && a.G <= 16 && (s.n_tok - max_new) * a.G <= 64 * (g.n_seqs - 1) &&
      keys * s.hkv * s.d * 4 >= 400000000) {
    PagedAttn b = a;
    b.max_new = small / a.G;
    a.min_new = b.max_new + 1;
    const cudaError_t e = launch_paged_step(s, b, small, q, kp, vp, o, lse, parts, err, st);
    if (e != cudaSuccess) return e;
  }
  return launch_paged_chunk(s, a, q, kp, vp, o, lse, parts, err, st);
}

}  // namespace msa
