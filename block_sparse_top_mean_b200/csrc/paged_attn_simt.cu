// Attention of new tokens over a paged cache in fp32 arithmetic (see paged.cuh).
//
// One CTA walks its run of (row tile, 32-key tile) pairs.  Eight neighbouring threads hold a
// row: they form its 32 scores (4 each), its running maximum and sum, and D / 8 of its output
// columns, so a row's softmax needs three shuffles.  Keys and values of a tile are in shared
// memory in fp32.
#include "paged.cuh"

namespace msa {
namespace {

constexpr int KT = 32;
constexpr int kLanes = 8;             // threads of a row
constexpr float kLn2 = 0.6931471805599453f;

template <int D, int ROWS>
struct Smem {
  float k[KT][D + 4];                 // +4: 8 rows of a quarter-warp load hit 32 banks
  float v[KT][D];
  float q[ROWS][D];
  float p[ROWS][KT + 1];
  PlanSmem plan;
};

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(ROWS * kLanes)
paged_attn_simt_kernel(const T* __restrict__ q, const T* __restrict__ kp,
                       const T* __restrict__ vp, T* __restrict__ o, float* __restrict__ lse,
                       PagedParts parts, int* err, const __grid_constant__ PagedAttn a) {
  constexpr int THREADS = ROWS * kLanes;
  constexpr int N = Vec16<T>::N, CH = D / N;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D, ROWS>& sm = *reinterpret_cast<Smem<D, ROWS>*>(smem_raw);
  const int tid = threadIdx.x, row = tid / kLanes, l8 = tid % kLanes;
  Run r = paged_plan<KT, THREADS>(a, &sm.plan);
  if (tid == 0) parts.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
  if (r.at >= r.end) return;
  bool first_item = true;
  do {
    const int tile0 = run_first(a, r), nt = run_tiles(a, r);
    if (nt == 0) break;                                   // the run ends in the item's lead
    const int t_in = r.rt * a.tt + row / a.G, h = row % a.G;
    const bool on = row < a.tt * a.G && t_in < r.v.n;
    const int64_t tok = r.v.tok0 + t_in;
    const int64_t qrow = tok * a.hq + r.g * a.G + h;      // row of o and lse
    // keys this row sees; none for a token before the first key
    const int see = on ? (int)max(0LL, min((long long)r.v.past + t_in + 1, (long long)r.v.cap)) : 0;
    const int vis = tile_keys(a, r.v, r.rt);
    __syncthreads();
    if (on) {
      const T* src = q + tok * a.qs + (int64_t)(r.g * a.G + h) * D;
      for (int c = l8; c < CH; c += kLanes) {
        float f[N];
        Vec16<T>::unpack(ldg16(src + c * N), f);
#pragma unroll
        for (int e = 0; e < N; ++e) sm.q[row][c * N + e] = f[e] * a.scale_log2;
      }
    }
    float m = -CUDART_INF_F, l = 0.f;
    float acc[D / kLanes];
#pragma unroll
    for (int i = 0; i < D / kLanes; ++i) acc[i] = 0.f;
    for (int it = 0; it < nt; ++it) {
      const int key0 = (tile0 + it) * KT;
      __syncthreads();
      for (int i = tid; i < 2 * KT * CH; i += THREADS) {
        const int which = i / (KT * CH), j = i % (KT * CH), kr = j / CH, c = j % CH;
        const int key = key0 + kr;
        float f[N];
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (key < vis) {
          const int pg = key_page(a, r.s, key, err);
          if (pg >= 0)
            raw = ldg16((which ? vp : kp) +
                        (((int64_t)pg * a.hkv + r.g) * a.g.page + key % (int)a.g.page) * D + c * N);
        }
        Vec16<T>::unpack(raw, f);
#pragma unroll
        for (int e = 0; e < N; ++e) (which ? sm.v[kr] : sm.k[kr])[c * N + e] = f[e];
      }
      __syncthreads();
      float s[KT / kLanes];
#pragma unroll
      for (int j = 0; j < KT / kLanes; ++j) s[j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.q[row][d]);
#pragma unroll
        for (int j = 0; j < KT / kLanes; ++j) {
          const float4 y = *reinterpret_cast<const float4*>(&sm.k[l8 + j * kLanes][d]);
          s[j] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s[j]))));
        }
      }
      float mx = m;
#pragma unroll
      for (int j = 0; j < KT / kLanes; ++j)
        if (key0 + l8 + j * kLanes < see) mx = fmaxf(mx, s[j]);
#pragma unroll
      for (int w = 1; w < kLanes; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float ref = mx == -CUDART_INF_F ? 0.f : mx;
      const float alpha = exp2f(m - ref);
      float add = 0.f;
#pragma unroll
      for (int j = 0; j < KT / kLanes; ++j) {
        const float e = key0 + l8 + j * kLanes < see ? exp2f(s[j] - ref) : 0.f;
        sm.p[row][l8 + j * kLanes] = e;
        add += e;
      }
#pragma unroll
      for (int w = 1; w < kLanes; w <<= 1) add += __shfl_xor_sync(0xffffffffu, add, w);
      l = l * alpha + add;
      m = mx;
#pragma unroll
      for (int i = 0; i < D / kLanes; ++i) acc[i] *= alpha;
      __syncwarp();
      for (int kk = 0; kk < KT; ++kk) {
        const float e = sm.p[row][kk];
#pragma unroll
        for (int i = 0; i < D / kLanes / 4; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(&sm.v[kk][(i * kLanes + l8) * 4]);
          acc[i * 4 + 0] = fmaf(e, y.x, acc[i * 4 + 0]);
          acc[i * 4 + 1] = fmaf(e, y.y, acc[i * 4 + 1]);
          acc[i * 4 + 2] = fmaf(e, y.z, acc[i * 4 + 2]);
          acc[i * 4 + 3] = fmaf(e, y.w, acc[i * 4 + 3]);
        }
      }
      __syncwarp();
    }
    const bool whole = nt == r.tiles;
    if (whole) {
      if (on) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int i = 0; i < D / kLanes; ++i)
          o[qrow * D + ((i / 4) * kLanes + l8) * 4 + i % 4] = from_f32<T>(acc[i] * inv);
        if (l8 == 0 && lse != nullptr)
          lse[qrow] = l > 0.f ? (m + log2f(l)) * kLn2 : -CUDART_INF_F;
      }
    } else {
      const int64_t slot = 2 * (int64_t)blockIdx.x + (first_item ? 0 : 1);
      if (l8 == 0) parts.ml[slot * ROWS + row] = make_float2(m, l);
#pragma unroll
      for (int i = 0; i < D / kLanes; i += 4)
        *reinterpret_cast<float4*>(&parts.o[(slot * ROWS + row) * D + ((i / 4) * kLanes + l8) * 4]) =
            make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      if (tid == 0 && tile0 == 0)
        parts.rec[blockIdx.x] = item_record(a, r, first_item);
    }
    first_item = false;
  } while (run_next<KT>(a, r));
}

template <typename T, int D, int ROWS>
cudaError_t run(PagedAttn& a, const HeadShape& s, const void* q, const void* kp, const void* vp,
                void* o, float* lse, const PagedParts& parts, int* err, cudaStream_t st) {
  a.tt = ROWS / a.G;
  a.lead = 1;
  const size_t smem = sizeof(Smem<D, ROWS>);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = raise_smem((const void*)paged_attn_simt_kernel<T, D, ROWS>, smem, &done);
  if (e != cudaSuccess) return e;
  const int grid = paged_grid();
  paged_attn_simt_kernel<T, D, ROWS><<<grid, ROWS * kLanes, smem, st>>>(
      (const T*)q, (const T*)kp, (const T*)vp, (T*)o, lse, parts, err, a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_combine(s, a, grid, ROWS, parts, o, lse, st) : e;
}

}  // namespace

cudaError_t launch_paged_simt(const HeadShape& s, PagedAttn a, int rows, const void* q,
                              const void* kp, const void* vp, void* o, float* lse,
                              const PagedParts& parts, int* err, cudaStream_t st) {
  if (s.d == 128)
    return rows <= 16 ? run<float, 128, 16>(a, s, q, kp, vp, o, lse, parts, err, st)
                      : run<float, 128, 64>(a, s, q, kp, vp, o, lse, parts, err, st);
  return rows <= 16 ? run<float, 64, 16>(a, s, q, kp, vp, o, lse, parts, err, st)
                    : run<float, 64, 64>(a, s, q, kp, vp, o, lse, parts, err, st);
}

}  // namespace msa
