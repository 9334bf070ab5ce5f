// Attention of new tokens over a paged cache, fp32 (see paged.cuh for the schedule and
// paged_ring.cuh for the stream): all products on the fp32 pipe, as the fp32 calls of this
// library are (a tf32 product would keep 11 bits).
//
//   paged_step32_kernel (up to 8 rows, single tokens): the cache's stream is the bound.  A tile
//     belongs to one of six warps; eight lanes share a key (16 dims each at d = 128), four keys
//     at a time, so scores take three shuffles and K and V are read once from shared memory
//     for four rows of registers.  16 sequences x 8192 keys, 32 / 8 heads of 128: 171 us, 6.3
//     TB/s (three warps of two stages: 186); with 8 heads a KV head 289 us (467): shuffles and
//     exponentials of eight rows, which one lane a key instead made no faster (350).
//   paged_rows32_kernel (64 rows): 4 d flops a row and key against 74 TFLOP/s make the fp32 pipe
//     the bound, if shared memory can feed it: a thread holds four rows, so eight 16-byte reads
//     serve 64 multiply-adds (with two rows the reads were 79% busy and the fp32 pipe 32%), two
//     in an instruction (1330 -> 1130 us).  A row belongs to eight lanes of one warp, so the
//     warps meet only at the ring.  A prompt of 2048 tokens, 32 / 8 heads of 128: 1009 us, 34
//     TFLOP/s; the accumulators leave room for two warps a scheduler.
#include "paged_ring.cuh"
#include "fastmath.cuh"

namespace msa {
namespace {

using namespace paged;
using fastmath::ffma2;

// Cost of an item beside its tiles, in tiles.
constexpr int kStepLead = 4, kRowLead = 1;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float4 lds4(const unsigned char* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ void fma4(float4& d, float s, const float4& v) {
  d.x = fmaf(s, v.x, d.x);
  d.y = fmaf(s, v.y, d.y);
  d.z = fmaf(s, v.z, d.z);
  d.w = fmaf(s, v.w, d.w);
}
__device__ __forceinline__ void fma4_pairs(float4& d, float s, const float4& v) {
  ffma2(d.x, d.y, s, s, v.x, v.y, d.x, d.y);
  ffma2(d.z, d.w, s, s, v.z, v.w, d.z, d.w);
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}
// Keys that row `row` of the item sees, -1 when it holds no query.
__device__ __forceinline__ int row_sees(const PagedAttn& a, const Run& r, int row) {
  const int t_in = r.rt * a.tt + row / a.G;
  if (row >= a.tt * a.G || t_in >= r.v.n) return -1;
  return (int)max(0LL, min((long long)r.v.past + t_in + 1, (long long)r.v.cap));
}
// The row's query, head-packed; only for rows that hold one.
__device__ __forceinline__ const float* row_query(const PagedAttn& a, const Run& r,
                                                  const float* q, int row, int D) {
  return q + (r.v.tok0 + r.rt * a.tt + row / a.G) * a.qs + (int64_t)(r.g * a.G + row % a.G) * D;
}
__device__ __forceinline__ int64_t row_out(const PagedAttn& a, const Run& r, int row) {
  return (r.v.tok0 + r.rt * a.tt + row / a.G) * a.hq + r.g * a.G + row % a.G;
}

// ------------------------------------------------------------------ up to 4 * RG rows
constexpr int kStepWarps = 6;          // a stage each (d = 64: two)
constexpr int kStepThreads = 32 * (kStepWarps + 1);
template <int D> constexpr int kStepStages = 6 * 128 / D;      // 192 KB

template <int D, int R>
struct __align__(16) Join32 {
  float q[R][D];                      // the item's queries, scaled
  float o[kStepWarps][R][D];          // the warps' outputs of an item
  float2 ml[kStepWarps][R];
};

template <int D, int RG>
__global__ void __launch_bounds__(kStepThreads, 1)
paged_step32_kernel(const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, int box,
                    const float* __restrict__ q, float* __restrict__ o, float* __restrict__ lse,
                    PagedParts parts, int* err, const __grid_constant__ PagedAttn a) {
  constexpr int R = 4 * RG, ST = kStepStages<D>, NS = D / 32;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using RingT = Ring<ST, kStepWarps>;
  RingT& sm = *reinterpret_cast<RingT*>(ring + ST * kStageBytes<D, 4>);
  Join32<D, R>& jn =
      *reinterpret_cast<Join32<D, R>*>(ring + ST * kStageBytes<D, 4> + sizeof(RingT));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  Run r = begin<kStepThreads>(tm_k, tm_v, sm, 1, parts, a);
  if (r.at >= r.end) return;
  if (warp == kStepWarps) {
    produce<D, 4>(tm_k, tm_v, box, ring, sm, r, err, q, a);
    return;
  }
  const int kg = lane >> 3, l8 = lane & 7;      // key of each four; dims l8 * 4 of each 32
  int turn = warp, st = warp;                   // tiles until this warp's; its stage
  uint32_t phase = 0;
  bool first_item = true, aborted = false;
  do {
    const int tile0 = run_first(a, r), nt = run_tiles(a, r), vis = tile_keys(a, r.v, r.rt);
    if (nt == 0) break;                                   // the run ends in the item's lead
    for (int i = tid; i < R * D / 4; i += kStepWarps * 32) {
      const int row = i / (D / 4), c = i % (D / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row_sees(a, r, row) >= 0)
        x = __ldg(reinterpret_cast<const float4*>(row_query(a, r, q, row, D) + c));
      *reinterpret_cast<float4*>(&jn.q[row][c]) = make_float4(
          x.x * a.scale_log2, x.y * a.scale_log2, x.z * a.scale_log2, x.w * a.scale_log2);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kStepWarps * 32) : "memory");
    float m[RG][4], l[RG][4];
    float4 acc[RG][4][NS];
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        m[g][x] = -CUDART_INF_F;
        l[g][x] = 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) acc[g][x][i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    int it = turn;
    for (; it < nt; it += kStepWarps) {
      if (aborted || !ring_wait(sm, &sm.full[st], phase, err)) {
        aborted = true;
        break;
      }
      const unsigned char* sk = ring + st * kStageBytes<D, 4>;
      const unsigned char* sv = sk + kTileBytes<D, 4>;
      const int key0 = (tile0 + it) * KT, lim = vis - key0;
      // this lane's chunk of keys kg and kg + 4 of each eight
      const uint32_t at0 = kg * 128u + ((uint32_t)(l8 ^ kg) << 4);
      const uint32_t at1 = (kg + 4) * 128u + ((uint32_t)(l8 ^ (kg + 4)) << 4);
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        float s[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[k][x] = 0.f;
#pragma unroll 1
        for (int i = 0; i < NS; ++i) {
          float4 qr[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            qr[x] = *reinterpret_cast<const float4*>(&jn.q[g * 4 + x][i * 32 + l8 * 4]);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 kv = lds4(sk + i * kSlice + (k >> 1) * 1024 + ((k & 1) ? at1 : at0));
#pragma unroll
            for (int x = 0; x < 4; ++x) s[k][x] = dot4(qr[x], kv, s[k][x]);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int w = 1; w < 8; w <<= 1) s[k][x] += __shfl_xor_sync(0xffffffffu, s[k][x], w);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int see = row_sees(a, r, g * 4 + x);
          float mx = m[g][x];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (key0 + k * 4 + kg >= see) s[k][x] = -CUDART_INF_F;
            mx = fmaxf(mx, s[k][x]);
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float ref = mx == -CUDART_INF_F ? 0.f : mx;
          const float alpha = exp2f(m[g][x] - ref);
          m[g][x] = mx;
          float add = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            s[k][x] = exp2f(s[k][x] - ref);
            add += s[k][x];
          }
          l[g][x] = l[g][x] * alpha + add;
          if (alpha != 1.f) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
              float4& y = acc[g][x][i];
              y = make_float4(y.x * alpha, y.y * alpha, y.z * alpha, y.w * alpha);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k * 4 + kg >= lim) continue;                // rows behind the last key: anything
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const float4 v = lds4(sv + i * kSlice + (k >> 1) * 1024 + ((k & 1) ? at1 : at0));
#pragma unroll
            for (int x = 0; x < 4; ++x) fma4_pairs(acc[g][x][i], s[k][x], v);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
      if ((st += kStepWarps) >= ST) {
        st -= ST;
        phase ^= 1;
      }
    }
    turn = it - nt;
    // the four keys' lanes, then the warps
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
#pragma unroll
        for (int w = 8; w < 32; w <<= 1) {
          l[g][x] += __shfl_xor_sync(0xffffffffu, l[g][x], w);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            float4& y = acc[g][x][i];
            y.x += __shfl_xor_sync(0xffffffffu, y.x, w);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, w);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, w);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, w);
          }
        }
        if (kg == 0) {
#pragma unroll
          for (int i = 0; i < NS; ++i)
            *reinterpret_cast<float4*>(&jn.o[warp][g * 4 + x][i * 32 + l8 * 4]) = acc[g][x][i];
        }
        if (lane == 0) jn.ml[warp][g * 4 + x] = make_float2(m[g][x], l[g][x]);
      }
    asm volatile("bar.sync 1, %0;" ::"n"(kStepWarps * 32) : "memory");
    const bool whole = nt == r.tiles;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (first_item ? 0 : 1);
    for (int i = tid; i < R * D / 4; i += kStepWarps * 32) {
      const int row = i / (D / 4), c = i % (D / 4) * 4;
      if (row_sees(a, r, row) < 0) continue;
      float mx = -CUDART_INF_F, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kStepWarps; ++w) mx = fmaxf(mx, jn.ml[w][row].x);
      const float base = mx == -CUDART_INF_F ? 0.f : mx;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kStepWarps; ++w) {
        const float f = exp2f(jn.ml[w][row].x - base);
        sum = fmaf(jn.ml[w][row].y, f, sum);
        fma4(y, f, *reinterpret_cast<const float4*>(&jn.o[w][row][c]));
      }
      const int64_t qrow = row_out(a, r, row);
      if (whole) {
        const float inv = sum != 0.f ? 1.f / sum : 0.f;
        *reinterpret_cast<float4*>(o + qrow * D + c) =
            make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
        if (c == 0 && lse != nullptr)
          lse[qrow] = sum != 0.f ? (mx + log2f(sum)) * kLn2 : -CUDART_INF_F;
      } else {
        *reinterpret_cast<float4*>(parts.o + (slot * R + row) * D + c) = y;
        if (c == 0) parts.ml[slot * R + row] = make_float2(mx, sum);
      }
    }
    if (!whole && tile0 == 0 && tid == 0)
      parts.rec[blockIdx.x] = item_record(a, r, first_item);
    asm volatile("bar.sync 1, %0;" ::"n"(kStepWarps * 32) : "memory");
    first_item = false;
  } while (run_next<KT>(a, r));
}

// ------------------------------------------------------------------ 64 rows
constexpr int kXR = 4;                // rows of a thread
constexpr int kRowWarps = 64 / kXR / 4;
constexpr int kRowThreads = 32 * (kRowWarps + 1);
template <int D> constexpr int kRowStages = 2 * 128 / D;       // 64 KB: two CTAs an SM

template <int D>
struct __align__(16) Rows32 {
  float q[64][D + 4];                 // +4: the rows of a warp's four threads hit different banks
  float p[64][KT + 4];
};

template <int D>
__global__ void __launch_bounds__(kRowThreads, 2)
paged_rows32_kernel(const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, int box,
                    const float* __restrict__ q, float* __restrict__ o, float* __restrict__ lse,
                    PagedParts parts, int* err, const __grid_constant__ PagedAttn a) {
  constexpr int R = 64, ST = kRowStages<D>, NS = D / 32, X = kXR;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using RingT = Ring<ST, 1>;
  RingT& sm = *reinterpret_cast<RingT*>(ring + ST * kStageBytes<D, 4>);
  Rows32<D>& rs = *reinterpret_cast<Rows32<D>*>(ring + ST * kStageBytes<D, 4> + sizeof(RingT));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  Run r = begin<kRowThreads>(tm_k, tm_v, sm, kRowWarps, parts, a);
  if (r.at >= r.end) return;
  if (warp == kRowWarps) {
    produce<D, 4>(tm_k, tm_v, box, ring, sm, r, err, q, a);
    return;
  }
  // rows row0 + 4 x (a warp's four threads in neighbouring rows); keys tx + 8 j
  const int row0 = warp * 4 * X + lane / 8, tx = lane % 8;
  int st = 0;
  uint32_t phase = 0;
  bool first_item = true, aborted = false;
  do {
    const int tile0 = run_first(a, r), nt = run_tiles(a, r), vis = tile_keys(a, r.v, r.rt);
    if (nt == 0) break;                                   // the run ends in the item's lead
    int see[X];
#pragma unroll
    for (int x = 0; x < X; ++x) {                         // (rows of this warp alone)
      const int row = row0 + 4 * x;
      see[x] = row_sees(a, r, row);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int c = (i * 8 + tx) * 4;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        if (see[x] >= 0) y = __ldg(reinterpret_cast<const float4*>(row_query(a, r, q, row, D) + c));
        *reinterpret_cast<float4*>(&rs.q[row][c]) = make_float4(
            y.x * a.scale_log2, y.y * a.scale_log2, y.z * a.scale_log2, y.w * a.scale_log2);
      }
    }
    __syncwarp();
    float m[X], l[X];
    float4 acc[X][NS];
#pragma unroll
    for (int x = 0; x < X; ++x) {
      m[x] = -CUDART_INF_F;
      l[x] = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) acc[x][i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int it = 0; it < nt; ++it) {
      if (aborted || !ring_wait(sm, &sm.full[st], phase, err)) {
        aborted = true;
        break;
      }
      const unsigned char* sk = ring + st * kStageBytes<D, 4>;
      const unsigned char* sv = sk + kTileBytes<D, 4>;
      const int key0 = (tile0 + it) * KT, lim = vis - key0;
      float s[X][4], s2[X][4];                            // over even and over odd dims
#pragma unroll
      for (int x = 0; x < X; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[x][j] = s2[x][j] = 0.f;
#pragma unroll 1
      for (int i = 0; i < NS; ++i)
#pragma unroll 8
        for (int c = 0; c < 8; ++c) {
          float4 y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            y[j] = lds4(sk + i * kSlice + (j * 8 + tx) * 128 + ((c ^ tx) << 4));
#pragma unroll
          for (int x = 0; x < X; ++x) {
            const float4 qx = *reinterpret_cast<const float4*>(&rs.q[row0 + 4 * x][i * 32 + c * 4]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              ffma2(s[x][j], s2[x][j], qx.x, qx.y, y[j].x, y[j].y, s[x][j], s2[x][j]);
              ffma2(s[x][j], s2[x][j], qx.z, qx.w, y[j].z, y[j].w, s[x][j], s2[x][j]);
            }
          }
        }
#pragma unroll
      for (int x = 0; x < X; ++x) {
        float mx = m[x];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[x][j] += s2[x][j];
          if (key0 + j * 8 + tx >= see[x]) s[x][j] = -CUDART_INF_F;
          mx = fmaxf(mx, s[x][j]);
        }
#pragma unroll
        for (int w = 1; w < 8; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float ref = mx == -CUDART_INF_F ? 0.f : mx;
        const float alpha = exp2f(m[x] - ref);
        m[x] = mx;
        float add = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(s[x][j] - ref);
          rs.p[row0 + 4 * x][j * 8 + tx] = e;
          add += e;
        }
        l[x] = l[x] * alpha + add;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          float4& y = acc[x][i];
          y = make_float4(y.x * alpha, y.y * alpha, y.z * alpha, y.w * alpha);
        }
      }
      __syncwarp();
      // four keys: their weights for the thread's rows, and the V rows
      auto keys4 = [&](int k, int n) {
        float w[X][4];
#pragma unroll
        for (int x = 0; x < X; ++x) {
          const float4 p = *reinterpret_cast<const float4*>(&rs.p[row0 + 4 * x][k]);
          w[x][0] = p.x;
          w[x][1] = p.y;
          w[x][2] = p.z;
          w[x][3] = p.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (e >= n) break;
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const float4 y = lds4(sv + i * kSlice + (k + e) * 128 + ((tx ^ ((k + e) & 7)) << 4));
#pragma unroll
            for (int x = 0; x < X; ++x) fma4_pairs(acc[x][i], w[x][e], y);
          }
        }
      };
      if (lim >= KT) {
#pragma unroll 2
        for (int k = 0; k < KT; k += 4) keys4(k, 4);
      } else {
        // (weights of keys behind the last are zero, but their V rows may hold anything)
#pragma unroll 1
        for (int k = 0; k < lim; k += 4) keys4(k, lim - k);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[st]);
      if (++st == ST) {
        st = 0;
        phase ^= 1;
      }
    }
    const bool whole = nt == r.tiles;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (first_item ? 0 : 1);
#pragma unroll
    for (int x = 0; x < X; ++x) {
#pragma unroll
      for (int w = 1; w < 8; w <<= 1) l[x] += __shfl_xor_sync(0xffffffffu, l[x], w);
      if (see[x] < 0) continue;
      const int row = row0 + 4 * x;
      const int64_t qrow = row_out(a, r, row);
      const float inv = whole ? (l[x] != 0.f ? 1.f / l[x] : 0.f) : 1.f;
      float* dst = whole ? o + qrow * D : parts.o + (slot * R + row) * D;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const float4 y = acc[x][i];
        *reinterpret_cast<float4*>(dst + (i * 8 + tx) * 4) =
            make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      }
      if (tx == 0) {
        if (!whole) parts.ml[slot * R + row] = make_float2(m[x], l[x]);
        else if (lse != nullptr)
          lse[qrow] = l[x] != 0.f ? (m[x] + log2f(l[x])) * kLn2 : -CUDART_INF_F;
      }
    }
    if (!whole && tile0 == 0 && tid == 0)
      parts.rec[blockIdx.x] = item_record(a, r, first_item);
    first_item = false;
  } while (run_next<KT>(a, r));
}

template <typename K>
cudaError_t run(K kernel, DeviceOnce* done, int rows, int threads, int grid,
                size_t smem, PagedAttn& a, const HeadShape& s, const void* q, const void* kp,
                const void* vp, void* o, float* lse, const PagedParts& parts, int* err,
                cudaStream_t st) {
  a.tt = rows / a.G;
  a.lead = rows == 64 ? kRowLead : kStepLead;
  int box = 0;
  CUtensorMap mk{}, mv{};
  if (!pool_maps(a, s, kp, vp, &mk, &mv, &box)) return cudaErrorInvalidValue;
  cudaError_t e = raise_smem((const void*)kernel, smem, done);
  if (e != cudaSuccess) return e;
  kernel<<<grid, threads, smem, st>>>(mk, mv, box, (const float*)q, (float*)o, lse, parts, err, a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_combine(s, a, grid, rows, parts, o, lse, st) : e;
}

template <int D>
cudaError_t run_rows(int rows, PagedAttn& a, const HeadShape& s, const void* q, const void* kp,
                     const void* vp, void* o, float* lse, const PagedParts& parts, int* err,
                     cudaStream_t st) {
  static DeviceOnce done[3];
  constexpr size_t step = ring_bytes<D, 4, kStepStages<D>, kStepWarps>();
  if (rows <= 4)
    return run(paged_step32_kernel<D, 1>, &done[0], 4, kStepThreads, paged_grid(),
               step + sizeof(Join32<D, 4>), a, s, q, kp, vp, o, lse, parts, err, st);
  if (rows <= 8)
    return run(paged_step32_kernel<D, 2>, &done[1], 8, kStepThreads, paged_grid(),
               step + sizeof(Join32<D, 8>), a, s, q, kp, vp, o, lse, parts, err, st);
  return run(paged_rows32_kernel<D>, &done[2], 64, kRowThreads, 2 * paged_grid(),
             ring_bytes<D, 4, kRowStages<D>, 1>() + sizeof(Rows32<D>), a, s, q, kp, vp, o, lse,
             parts, err, st);
}

}  // namespace

cudaError_t launch_paged_f32(const HeadShape& s, PagedAttn a, int rows, const void* q,
                             const void* kp, const void* vp, void* o, float* lse,
                             const PagedParts& parts, int* err, cudaStream_t st) {
  return s.d == 128 ? run_rows<128>(rows, a, s, q, kp, vp, o, lse, parts, err, st)
                    : run_rows<64>(rows, a, s, q, kp, vp, o, lse, parts, err, st);
}

}  // namespace msa
