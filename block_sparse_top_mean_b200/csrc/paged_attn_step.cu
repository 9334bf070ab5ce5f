// Attention of single new tokens (up to 16 rows) over a paged cache, bf16 (see paged.cuh for the
// schedule and paged_ring.cuh for the stream).
//
// With R = new tokens x G rows against a cache, 4 R flops come with every element of K and V: the
// cache's stream from HBM is the bound, and the kernel is built round it.  Four consumer warps
// run both products on mma.sync m16n8k16 (the tensor pipe is far from its limit, and a tcgen05
// tile would be 128 rows).  A tile belongs to one warp, so four tiles are in work at a time and a
// tile takes one pass of the softmax.  The products are S^T = K Q^T and O^T += V^T P^T: keys and
// dims fill the 16 rows of the instruction and the queries its 8 columns, so up to 8 rows waste
// nothing (queries as the 16 rows took twice the instructions).  The warps' outputs are joined
// in shared memory when the item ends.  Weights go into the product with V as two bf16 terms
// (hi + lo, 2^-17): the second product hides behind HBM, and the output is off by its own
// rounding alone.
//   64 sequences x 8192 keys, 32 / 8 heads of 128: 316 us, 6.8 TB/s; 1 x 131072 keys: 87 us.
// Keys behind the last visible one are not loaded past their page piece; their scores are
// replaced, and their V rows (which may hold anything) masked in the fragments.
#include "paged_ring.cuh"
#include "fastmath.cuh"

namespace msa {
namespace {

using namespace paged;
using fastmath::fast_exp2;

constexpr int kConsumers = 4;         // warps 0-3; warp 4 produces
constexpr int kThreads = 32 * (kConsumers + 1);
// Two CTAs an SM: while one joins an item's warps and starts the next, the other's tiles keep
// coming (256 sequences of up to 256 keys 50 -> 35 us, 48 of 1 to 16384 52 -> 49, 64 x 8192 325
// -> 316, against one CTA of 12 stages, 192 KB; two of 4 stages hold 128 KB).
constexpr int kCtas = 2;
template <int D> constexpr int kStages = 4 * 128 / D;        // 64 KB of tiles a CTA
// What an item costs beside its tiles, in tiles (48 sequences of 1 to 16384 keys, one CTA an SM: 0
// 168 us, 4 71, 7 61, 10 64; two: 3 51, 5 48.5, 6 48.5, 9 49).
constexpr int kLead = 6;
constexpr float kLn2 = 0.6931471805599453f;

// The warps' outputs of an item, joined when it ends.
template <int D, int R>
struct __align__(16) Join {
  float o[kConsumers][R][D + 4];
  float2 ml[kConsumers][R];
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// C[16x8] += A[16x16] B[16x8]; thread (g, t) = (lane / 4, lane % 4) holds C rows g, g + 8 and
// columns 2t, 2t + 1.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Clears the bf16 lanes of a fragment word whose keys (k, k + 1) are not below lim.
__device__ __forceinline__ uint32_t keep_keys(uint32_t w, int k, int lim) {
  return k + 1 < lim ? w : k < lim ? w & 0xffffu : 0u;
}
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Up to 8 * NQ rows.
template <int D, int NQ>
__global__ void __launch_bounds__(kThreads, kCtas)
paged_step_kernel(const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, int box,
                  const __nv_bfloat16* __restrict__ q, __nv_bfloat16* __restrict__ o,
                  float* __restrict__ lse, PagedParts parts, int* err,
                  const __grid_constant__ PagedAttn a) {
  constexpr int R = 8 * NQ, ST = kStages<D>;
  using RingT = Ring<ST, kConsumers>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  RingT& sm = *reinterpret_cast<RingT*>(ring + ST * kStageBytes<D, 2>);
  Join<D, R>& jn =
      *reinterpret_cast<Join<D, R>*>(ring + ST * kStageBytes<D, 2> + sizeof(RingT));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  Run r = begin<kThreads>(tm_k, tm_v, sm, 1, parts, a);
  if (r.at >= r.end) return;
  if (warp == kConsumers) {
    produce<D, 2>(tm_k, tm_v, box, ring, sm, r, err, q, a);
    return;
  }
  // thread (gr, t4) of a warp: scores of keys gr, gr + 8 of a 16-key block and queries 2 t4,
  // 2 t4 + 1 of each 8; outputs of dims gr, gr + 8 of a 16-dim block and the same queries
  const int gr = lane >> 2, t4 = lane & 3, mi = lane >> 3, ri = lane & 7;
  // ldmatrix rows: K block (keys (mi & 1) * 8 + ri, dims chunk mi >> 1), V block (keys
  // (mi >> 1) * 8 + ri, dims chunk mi & 1); chunk c of row r sits at c ^ (r % 8)
  const uint32_t k_row = (uint32_t)((mi & 1) * 8 + ri) * 128u;
  const uint32_t v_row = (uint32_t)((mi >> 1) * 8 + ri) * 128u;
  uint32_t k_off[4], v_off[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    k_off[j] = k_row + (uint32_t)((2 * j + (mi >> 1)) ^ ri) * 16u;
    v_off[j] = v_row + (uint32_t)((2 * j + (mi & 1)) ^ ri) * 16u;
  }
  int turn = warp, st = warp;                             // tiles until this warp's; its stage
  uint32_t phase = 0;
  bool first_item = true, aborted = false;
  do {
    const int tile0 = run_first(a, r), nt = run_tiles(a, r), vis = tile_keys(a, r.v, r.rt);
    if (nt == 0) break;                                   // the run ends in the item's lead
    uint32_t qb[NQ][D / 16][2];
    int see[NQ][2];                                       // keys of queries 2 t4, 2 t4 + 1
    int least = INT32_MAX;                                // of any query of this thread
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int row = n * 8 + gr, t_in = r.rt * a.tt + row / a.G;
      const bool on = row < a.tt * a.G && t_in < r.v.n;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          q + (r.v.tok0 + t_in) * a.qs + (int64_t)(r.g * a.G + row % a.G) * D);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qb[n][ks][0] = on ? __ldg(src + ks * 8 + t4) : 0u;
        qb[n][ks][1] = on ? __ldg(src + ks * 8 + 4 + t4) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = n * 8 + 2 * t4 + e, c_in = r.rt * a.tt + c / a.G;
        const bool there = c < a.tt * a.G && c_in < r.v.n;
        see[n][e] =
            there ? (int)max(0LL, min((long long)r.v.past + c_in + 1, (long long)r.v.cap)) : 0;
        if (there) least = min(least, see[n][e]);
      }
    }
    // (queries that are not there need no mask: their results go nowhere)
    least = __reduce_min_sync(0xffffffffu, least);
    float m[NQ][2], l[NQ][2], acc[NQ][D / 16][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      m[n][0] = m[n][1] = -CUDART_INF_F;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][dt][e] = 0.f;
    }
    int it = turn;
    for (; it < nt; it += kConsumers) {
      if (aborted || !ring_wait(sm, &sm.full[st], phase, err)) {
        aborted = true;
        break;
      }
      const uint32_t sk = smem_u32(ring + st * kStageBytes<D, 2>), sv = sk + kTileBytes<D, 2>;
      const int key0 = (tile0 + it) * KT;
      float s[NQ][2][4];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][kb][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          uint32_t f[4];
          ldsm4(sk + k_off[ks & 3] + (ks >> 2) * kSlice + kb * 2048, f);
#pragma unroll
          for (int n = 0; n < NQ; ++n) mma16816(s[n][kb], f, qb[n][ks][0], qb[n][ks][1]);
        }
      // online softmax over the tile's keys: s[.][kb][e] is key kb * 16 + gr + 8 (e / 2) and
      // query 2 t4 + e % 2
      const bool inside = key0 + KT <= least;
      bool moved = false;
      uint32_t ph[NQ][4], pl[NQ][4];                      // 8-key blocks of P^T, bf16 pairs
      float alpha[NQ][2];
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float mx[2] = {-CUDART_INF_F, -CUDART_INF_F}, add[2] = {0.f, 0.f}, ref[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[n][kb][e] * a.scale_log2;
            if (!inside && key0 + kb * 16 + gr + 8 * (e >> 1) >= see[n][e & 1]) x = -CUDART_INF_F;
            s[n][kb][e] = x;
            mx[e & 1] = fmaxf(mx[e & 1], x);
          }
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], w));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], w));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[n][e], mx[e]);
          ref[e] = mn == -CUDART_INF_F ? 0.f : mn;
          alpha[n][e] = fast_exp2(m[n][e] - ref[e]);
          moved |= alpha[n][e] != 1.f;
          m[n][e] = mn;
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = fast_exp2(s[n][kb][2 * h] - ref[0]);
            const float p1 = fast_exp2(s[n][kb][2 * h + 1] - ref[1]);
            add[0] += p0;
            add[1] += p1;
            const uint32_t hi = pack_bf16x2(p0, p1);
            ph[n][2 * kb + h] = transpose8(hi);
            pl[n][2 * kb + h] =
                transpose8(pack_bf16x2(p0 - bf16lo_to_f32(hi), p1 - bf16hi_to_f32(hi)));
          }
#pragma unroll
        for (int e = 0; e < 2; ++e) l[n][e] = l[n][e] * alpha[n][e] + add[e];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][dt][e] *= alpha[n][e & 1];
      }
      const int lim = vis - key0;                         // keys of the tile that exist
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          uint32_t f[4];                                  // (dims, keys): (0,0) (8,0) (0,8) (8,8)
          ldsm4_t(sv + v_off[dt & 3] + (dt >> 2) * kSlice + kb * 2048, f);
          if (lim < KT) {
#pragma unroll
            for (int w = 0; w < 4; ++w)
              f[w] = keep_keys(f[w], kb * 16 + (w >> 1) * 8 + 2 * t4, lim);
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
            mma16816(acc[n][dt], f, ph[n][2 * kb], ph[n][2 * kb + 1]);
            mma16816(acc[n][dt], f, pl[n][2 * kb], pl[n][2 * kb + 1]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
      if ((st += kConsumers) >= ST) {
        st -= ST;
        phase ^= 1;
      }
    }
    turn = it - nt;
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], w);
        const int row = n * 8 + 2 * t4 + e;
        if (gr == 0) jn.ml[warp][row] = make_float2(m[n][e], l[n][e]);
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) {
          jn.o[warp][row][dt * 16 + gr] = acc[n][dt][e];
          jn.o[warp][row][dt * 16 + gr + 8] = acc[n][dt][2 + e];
        }
      }
    consumers_sync();
    // join the four warps: R rows x D columns over 128 threads, four columns at a time
    const bool whole = nt == r.tiles;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (first_item ? 0 : 1);
#pragma unroll
    for (int i = tid; i < R * D / 4; i += kConsumers * 32) {
      const int row = i / (D / 4), c = i % (D / 4) * 4, t_in = r.rt * a.tt + row / a.G;
      if (row >= a.tt * a.G || t_in >= r.v.n) continue;
      float mx = -CUDART_INF_F, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) mx = fmaxf(mx, jn.ml[w][row].x);
      const float base = mx == -CUDART_INF_F ? 0.f : mx;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kConsumers; ++w) {
        const float f = fast_exp2(jn.ml[w][row].x - base);
        sum = fmaf(jn.ml[w][row].y, f, sum);
        const float4 x = *reinterpret_cast<const float4*>(&jn.o[w][row][c]);
        y.x = fmaf(x.x, f, y.x);
        y.y = fmaf(x.y, f, y.y);
        y.z = fmaf(x.z, f, y.z);
        y.w = fmaf(x.w, f, y.w);
      }
      const int64_t qrow = (r.v.tok0 + t_in) * a.hq + r.g * a.G + row % a.G;
      if (whole) {
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        *reinterpret_cast<uint2*>(o + qrow * D + c) =
            make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
        if (c == 0 && lse != nullptr)
          lse[qrow] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -CUDART_INF_F;
      } else {
        *reinterpret_cast<float4*>(parts.o + (slot * R + row) * D + c) = y;
        if (c == 0) parts.ml[slot * R + row] = make_float2(mx, sum);
      }
    }
    if (!whole && tile0 == 0 && tid == 0)
      parts.rec[blockIdx.x] = item_record(a, r, first_item);
    consumers_sync();
    first_item = false;
  } while (run_next<KT>(a, r));
}

template <int D, int NQ>
cudaError_t run(PagedAttn& a, const HeadShape& s, const void* q, const void* kp, const void* vp,
                void* o, float* lse, const PagedParts& parts, int* err, cudaStream_t st) {
  a.tt = 8 * NQ / a.G;
  a.lead = kLead;
  int box = 0;
  CUtensorMap mk{}, mv{};
  if (!pool_maps(a, s, kp, vp, &mk, &mv, &box)) return cudaErrorInvalidValue;
  constexpr size_t smem = ring_bytes<D, 2, kStages<D>, kConsumers>() + sizeof(Join<D, 8 * NQ>);
  static_assert(kCtas * (smem + 1024) <= 233472, "228 KB an SM");
  static DeviceOnce done;
  cudaError_t e = raise_smem((const void*)paged_step_kernel<D, NQ>, smem, &done);
  if (e != cudaSuccess) return e;
  const int grid = kCtas * paged_grid();
  paged_step_kernel<D, NQ><<<grid, kThreads, smem, st>>>(
      mk, mv, box, (const __nv_bfloat16*)q, (__nv_bfloat16*)o, lse, parts, err, a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_combine(s, a, grid, 8 * NQ, parts, o, lse, st) : e;
}

}  // namespace

cudaError_t launch_paged_step(const HeadShape& s, PagedAttn a, int rows, const void* q,
                              const void* kp, const void* vp, void* o, float* lse,
                              const PagedParts& parts, int* err, cudaStream_t st) {
  if (s.d == 128)
    return rows <= 8 ? run<128, 1>(a, s, q, kp, vp, o, lse, parts, err, st)
                     : run<128, 2>(a, s, q, kp, vp, o, lse, parts, err, st);
  return rows <= 8 ? run<64, 1>(a, s, q, kp, vp, o, lse, parts, err, st)
                   : run<64, 2>(a, s, q, kp, vp, o, lse, parts, err, st);
}

}  // namespace msa
