// Attention of chunks of new tokens over a paged cache on the 5th-generation tensor cores
// (bf16; see paged.cuh for rows, items and the schedule).
//
// An item's row tile is two halves of 128 rows (128 / G tokens each) against 128-key tiles;
// 4 d flops a row and key against 2 x 2 d bytes a key keep the tensor cores the bound from a
// few tens of rows up.  Roles (384 threads, two warps of them spare; one CTA an SM):
//   producer warp   copies K and V tiles by tensor maps over the pools (one box for every run
//                   of keys that a page holds, page numbers fetched 32 pieces ahead) into a ring
//                   of 128-key units, and the item's query rows (a box of G heads x tokens);
//   issuer warp     S_X = Q_X K^T and O_X += P_X V for the halves X = 0, 1 in turn: while one
//                   half's softmax runs, the tensor core works for the other.  MMAs of one
//                   thread run in order, so S_X of the next tile may be issued right behind the
//                   product that reads P_X from the same columns;
//   two warpgroups  the softmax of one half each, one thread a row: scores from TMEM, base-2
//                   exponentials, P back to TMEM as bf16 (rounded once, 2^-8 of each weight: the
//                   tensor core takes no wider left operand beside a bf16 V; a second bf16 term,
//                   2^-17, was measured: the prompt below 455 -> 627 us) in two parts, so the
//                   product with V starts at half of them.  The exponent reference moves only
//                   when a row's maximum outgrows it by 2^8, so O is rarely rescaled.
// What bounds it: softmax and products in turn, 2.0 us a tile of 256 x 128 at d = 128 (1.64 with
// the softmax left out).  2048 tokens over 30K keys, 32 / 8 heads: 852 to 888 us, 1200 to 1250
// TFLOP/s; a prompt of 8192: 455 to 470 us; four ragged chunks over 12000 keys in pages of 16: 84
// us, of which about 4 us an item's start and end and 8 us the join.  Measured slower: four softmax
// warpgroups, 64-key tiles with two sets of scores, exponentials on a polynomial.
// TMEM columns: S_0 / P_0 [0, 128), S_1 / P_1 [128, 256), O_0 [256, ..), O_1 [384, ..).
// Keys behind the last visible one: their scores are replaced, and the issuer clears their V
// rows (which may hold anything) before the product.
#include "paged.cuh"
#include "fastmath.cuh"
#include "sm100.cuh"

namespace msa {
namespace {

using namespace sm100;
using namespace fastmath;

constexpr int KT = 128;               // keys of a tile
constexpr int kHalfRows = 128;
constexpr int kThreads = 384;        // two softmax warpgroups; issuer, producer, two spare warps
constexpr int kIssuer = 8, kProducer = 9;
constexpr uint32_t kHalf = 128 * 128; // 128 rows x 64 dims
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.f;
// Cost of an item beside its tiles, in tiles (ragged chunks / 2048-token prompt / 8192, a slower
// join: 2 101 / 74 / 492 us, 3 89 / 68 / 470, 4 86 / 68 / 475, 6 88 / 69 / 484).
constexpr int kLead = 3;

template <int D> constexpr uint32_t kUnit = KT * D * 2;      // one K or V tile
template <int D> constexpr int kUnits = D == 128 ? 5 : 10;   // 160 KB

template <int D>
struct __align__(16) Shared {
  uint64_t kv_full[kUnits<D>], kv_empty[kUnits<D>];
  uint64_t q_full, q_empty, s_full[2], p_full[2][2], o_full[2], o_empty[2], idle;
  uint32_t tmem;
  int abort;
  PlanSmem plan;
};

template <int D>
__device__ __forceinline__ void give_up(Shared<D>& sm, int* err) {
  set_device_error(err, MSA_DEVERR_TIMEOUT);
  *(volatile int*)&sm.abort = 1;
}
// Waits for a phase, for the whole warp; false when the wait ran out (after ~2 s) or another
// warp's did.
template <int D>
__device__ __forceinline__ bool wait(Shared<D>& sm, uint64_t* bar, uint32_t parity, int* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  const long long t0 = clock64();
  while (!ok && *(volatile int*)&sm.abort == 0 && clock64() - t0 < MSA_WAIT_CLOCKS)
    ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  if (threadIdx.x % 32 == 0) give_up(sm, err);
  return false;
}

// Both halves hold queries when the row tile's tokens reach into the second.
__device__ __forceinline__ int halves(const PagedAttn& a, const Run& r) {
  return r.v.n - r.rt * a.tt > a.tt / 2 ? 2 : 1;
}

// One row's softmax over a tile: scores (TMEM columns s_t ..) to weights (bf16, over them), the
// row's reference and sum brought along.  lim: the tile's keys that the row sees; FULL: all, in
// every row of the warp, and c2 >= 0 (the maximum of unscaled scores serves).  started: O (o_t
// ..) holds earlier tiles.  p_part[0] is arrived at when the first half of the weights is in
// place, p_part[1] when all are.
template <bool FULL, int D>
__device__ __forceinline__ void softmax_tile(uint32_t s_t, uint32_t o_t, float c2, int lim,
                                             bool started, float& mref, float& l,
                                             uint64_t* p_part) {
  uint32_t sv[4][32];
  tmem_ld32(s_t, sv[0]);
  tmem_ld32(s_t + 32, sv[1]);
  tmem_ld_wait();
  tmem_ld32(s_t + 64, sv[2]);
  tmem_ld32(s_t + 96, sv[3]);
  float mx = -CUDART_INF_F;
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
    if (hf == 1) tmem_ld_wait();
    if (FULL) {
      float m8[8];                                        // eight chains of three-input maxima
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t* v = &sv[hf * 2 + (j >> 2)][(j & 3) * 8];
        float m = fmax3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
        m = fmax3(m, __uint_as_float(v[3]), __uint_as_float(v[4]));
        m = fmax3(m, __uint_as_float(v[5]), __uint_as_float(v[6]));
        m8[j] = fmaxf(m, __uint_as_float(v[7]));
      }
      mx = fmax3(mx, fmax3(m8[0], m8[1], m8[2]),
                 fmax3(fmax3(m8[3], m8[4], m8[5]), m8[6], m8[7]));
    } else {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (hf * 64 + w * 32 + k < lim) mx = fmaxf(mx, __uint_as_float(sv[hf * 2 + w][k]));
    }
  }
  if (!FULL && c2 < 0.f) {                                // the scaled maximum is at the minimum
    mx = CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (w * 32 + k < lim) mx = fminf(mx, __uint_as_float(sv[w][k]));
  }
  const float mc = FULL || lim > 0 ? mx * c2 : -CUDART_INF_F;
  const bool need = mc > mref + kRescaleLog2;
  if (__any_sync(0xffffffffu, need)) {
    const float f = need ? fast_exp2(mref - mc) : 1.f;
    if (started) {                    // O holds the earlier tiles (s_full follows their products)
#pragma unroll 1
      for (int q = 0; q < D / 16; ++q) {
        uint32_t ov[16];
        tmem_ld16(o_t + q * 16, ov);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * f);
        tmem_st16(o_t + q * 16, ov);
      }
    }
    l *= f;
    if (need) mref = mc;
  }
  const float mb = mref > -CUDART_INF_F ? mref : 0.f;
  float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t pk[16];
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      float x0, x1, p0, p1;
      ffma2(x0, x1, __uint_as_float(sv[w][k]), __uint_as_float(sv[w][k + 1]), c2, c2, -mb, -mb);
      p0 = fast_exp2(x0);
      p1 = fast_exp2(x1);
      if (!FULL) {
        p0 = w * 32 + k < lim ? p0 : 0.f;
        p1 = w * 32 + k + 1 < lim ? p1 : 0.f;
      }
      if (w & 1) fadd2(a0, a1, a0, a1, p0, p1);
      else fadd2(b0, b1, b0, b1, p0, p1);
      pk[k / 2] = pack_bf16x2(p0, p1);
    }
    tmem_st16(s_t + w * 16, pk);                          // over scores already read
    if (w & 1) {
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_part[w >> 1]);
    }
  }
  l += (a0 + a1) + (b0 + b1);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q,
                   const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, int box,
                   __nv_bfloat16* __restrict__ o, float* __restrict__ lse, PagedParts parts,
                   int* err, const __grid_constant__ PagedAttn a) {
  constexpr int NU = kUnits<D>, DH = D / 64;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* qs = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* ring = qs + 2 * DH * kHalf;
  Shared<D>& sm = *reinterpret_cast<Shared<D>*>(ring + NU * kUnit<D>);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    for (int s = 0; s < NU; ++s) {
      mbar_init(&sm.kv_full[s], 1);
      mbar_init(&sm.kv_empty[s], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.idle, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.s_full[x], 1);
      mbar_init(&sm.p_full[x][0], kHalfRows);
      mbar_init(&sm.p_full[x][1], kHalfRows);
      mbar_init(&sm.o_full[x], 1);
      mbar_init(&sm.o_empty[x], kHalfRows);
    }
    sm.abort = 0;
    fence_mbar_init();
    parts.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  Run r = paged_plan<KT, kThreads>(a, &sm.plan);          // synchronises the CTA
  if (r.at >= r.end) return;                              // the whole CTA
  if (warp == 0) { tmem_alloc(&sm.tmem, 512); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  // Registers: 168 a thread at launch (3 x 128 x 168); the softmax holds a row's 128 scores.
  if (warp >= 8) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
  if (warp == kProducer) {
    // ---------------------------------------------------------------- producer
    const int per = KT / box;                             // page pieces of a tile
    const int rows = (int)(a.g.n_pages * a.hkv * a.g.page);
    const int half_toks = a.tt / 2;
    int units = 0, u = 0, item = 0;                       // units copied; the next one's place
    uint32_t ph = 1;                                      // of its empty barrier
    bool ok = true;
    do {
      const int tile0 = run_first(a, r), nt = run_tiles(a, r), vis = tile_keys(a, r.v, r.rt);
      if (nt == 0) break;                                 // the run ends in the item's lead
      // row of piece i in the pools, `rows` (reads as zeros) for an entry that is no page, -1
      // past the last visible key
      auto piece_row = [&](int i) -> int {
        const int key = tile0 * KT + i * box;
        if (i >= nt * per || key >= vis) return -1;
        const int pg = key_page(a, r.s, key, err);
        return pg < 0 ? rows : (int)(((int64_t)pg * a.hkv + r.g) * a.g.page + key % (int)a.g.page);
      };
      int cur = piece_row(lane), nxt = piece_row(32 + lane);
      for (int it = 0; it < nt && ok; ++it) {
        const int at = it * per;                          // first piece of the tile
        if (at > 0 && at % 32 == 0) {
          cur = nxt;
          nxt = piece_row(at + 32 + lane);
        }
        const int y = __shfl_sync(0xffffffffu, cur, (at & 31) + (lane < per ? lane : 0));
        const bool mine = lane < per && y >= 0;
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
#pragma unroll
        for (int v = 0; v < 2; ++v) {                     // K, then V
          if (!wait(sm, &sm.kv_empty[u], ph, err)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&sm.kv_full[u], (uint32_t)(n * box * D * 2));
          __syncwarp();
          if (mine && units != MSA_LOSE_COPY) {
#pragma unroll
            for (int h = 0; h < DH; ++h)
              tma_load_2d(ring + u * kUnit<D> + h * kHalf + lane * box * 128, v ? &tm_v : &tm_k,
                          &sm.kv_full[u], h * 64, y);
          }
          ++units;
          if (++u == NU) {
            u = 0;
            ph ^= 1;
          }
          if (it == 0 && v == 0) {                        // the item's queries, behind its first K
            if (!wait(sm, &sm.q_empty, (uint32_t)(item & 1) ^ 1, err)) {
              ok = false;
              break;
            }
            const int nx = halves(a, r), t0 = (int)r.v.tok0 + r.rt * a.tt;
            if (lane == 0) {
              mbar_arrive_expect_tx(&sm.q_full, (uint32_t)(nx * half_toks * a.G * D * 2));
              for (int x = 0; x < nx; ++x)
                for (int h = 0; h < DH; ++h)
                  tma_load_3d(qs + (x * DH + h) * kHalf, &tm_q, &sm.q_full, h * 64, r.g * a.G,
                              t0 + x * half_toks);
            }
            __syncwarp();
            ++item;
          }
        }
      }
    } while (ok && run_next<KT>(a, r));
    // No copy may land after the CTA ends, whoever gave up: the last ones are waited for.
    for (int s = units > NU ? units - NU : 0; s < units; ++s)
      mbar_wait_warp(&sm.kv_full[s % NU], (uint32_t)(s / NU) & 1);
    if (item > 0) mbar_wait_warp(&sm.q_full, (uint32_t)(item - 1) & 1);
  } else if (warp == kIssuer) {
    // ---------------------------------------------------------------- issuer
    const uint32_t id_s = idesc_bf16(128, KT, 0, 0), id_o = idesc_bf16(128, D, 0, 1);
    const uint64_t qd0 = sdesc_sw128(smem_u32(qs), 16, 1024);
    const uint64_t kd0 = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t vd0 = sdesc_sw128(smem_u32(ring), kHalf, 1024);
    int u = 0, item = 0;                                  // next unit of the ring; items begun
    uint32_t ph = 0, steps[2] = {0, 0}, done[2] = {0, 0}; // P tiles and items of each half
    bool ok = true;
    auto take = [&]() -> int {                            // waits for the next unit
      if (!wait(sm, &sm.kv_full[u], ph, err)) { ok = false; return 0; }
      const int at = u;
      if (++u == NU) {
        u = 0;
        ph ^= 1;
      }
      return at;
    };
    auto issue_qk = [&](int x, int ku) {
      if (elect_one()) {
        const uint64_t qd = qd0 + (uint64_t)(x * DH) * (kHalf >> 4);
        const uint64_t kd = kd0 + (uint64_t)ku * (kUnit<D> >> 4);
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint64_t off = (uint64_t)((s >> 2) * (kHalf >> 4) + (s & 3) * 2);
          umma_ss(tmem + x * 128, qd + off, kd + off, id_s, s > 0);
        }
        umma_commit(&sm.s_full[x]);
      }
      __syncwarp();
    };
    do {
      const int tile0 = run_first(a, r), nt = run_tiles(a, r), vis = tile_keys(a, r.v, r.rt);
      if (nt == 0) break;
      const int nx = halves(a, r);
      int ku = take();
      if (!ok || !wait(sm, &sm.q_full, (uint32_t)item & 1, err)) break;
      tc_fence_after();
      for (int x = 0; x < nx; ++x) issue_qk(x, ku);
      if (elect_one()) {
        umma_commit(&sm.kv_empty[ku]);
        if (nt == 1) umma_commit(&sm.q_empty);
      }
      for (int i = 0; i < nt && ok; ++i) {
        const int vu = take();
        if (!ok) break;
        const int lim = vis - (tile0 + i) * KT;           // keys of the tile that exist
        if (lim < KT) {
          unsigned char* v = ring + vu * kUnit<D>;
          const int from = max(lim, 0);
          for (int c = lane; c < (KT - from) * 8; c += 32)
#pragma unroll
            for (int h = 0; h < DH; ++h)
              *reinterpret_cast<uint4*>(v + h * kHalf + from * 128 + c * 16) =
                  make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        const bool more = i + 1 < nt;
        if (more) ku = take();
        if (!ok) break;
        for (int x = 0; x < nx && ok; ++x) {
          if (i == 0 && !wait(sm, &sm.o_empty[x], (done[x] & 1) ^ 1, err)) { ok = false; break; }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {                // the weights come in two parts
            if (!wait(sm, &sm.p_full[x][hf], steps[x] & 1, err)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
              const uint64_t vd = vd0 + (uint64_t)vu * (kUnit<D> >> 4);
#pragma unroll
              for (int s = hf * 4; s < hf * 4 + 4; ++s)
                umma_ts(tmem + 256 + x * 128, tmem + x * 128 + s * 8,
                        vd + (uint64_t)(s * (2048 >> 4)), id_o, (i > 0 || s > 0) ? 1u : 0u);
              if (!more && hf == 1) umma_commit(&sm.o_full[x]);
            }
            __syncwarp();
          }
          if (!ok) break;
          ++steps[x];
          if (more) issue_qk(x, ku);
          else ++done[x];
        }
        if (ok && elect_one()) {
          umma_commit(&sm.kv_empty[vu]);
          if (more) umma_commit(&sm.kv_empty[ku]);
          if (i + 2 == nt) umma_commit(&sm.q_empty);
        }
        __syncwarp();
      }
      ++item;
    } while (ok && run_next<KT>(a, r));
    // No product may read shared memory, write TMEM or arrive at a barrier after the CTA ends: when
    // a wait ran out, nobody else has waited for those under way.
    if (elect_one()) umma_commit(&sm.idle);
    __syncwarp();
    mbar_wait_warp(&sm.idle, 0);
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---------------------------------------------------------------- softmax, epilogue
    const int x = warp >> 2, row = tid & 127;             // this warpgroup's half, this row
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_t = lanes + x * 128, o_t = lanes + 256 + x * 128;
    const int half_toks = a.tt / 2, in_half = row / a.G, h = row - in_half * a.G;
    const float c2 = a.scale_log2;
    const bool wide = (reinterpret_cast<uintptr_t>(o) & 31) == 0;
    uint32_t steps = 0, items = 0;
    bool first_item = true, ok = true;
    do {
      const int tile0 = run_first(a, r), nt = run_tiles(a, r);
      if (nt == 0) break;
      const bool whole = nt == r.tiles;
      if (x < halves(a, r)) {
        const int t_in = r.rt * a.tt + x * half_toks + in_half;
        const bool on = in_half < half_toks && t_in < r.v.n;
        // keys this row sees; a row that holds no query takes no mask, its results go nowhere
        const long long see =
            on ? max(0LL, min((long long)r.v.past + t_in + 1, (long long)r.v.cap)) : (1LL << 40);
        float mref = -CUDART_INF_F, l = 0.f;
        for (int i = 0; i < nt; ++i, ++steps) {
          const int lim = (int)max(0LL, min((long long)KT, see - (long long)(tile0 + i) * KT));
          if (!wait(sm, &sm.s_full[x], steps & 1, err)) { ok = false; break; }
          tc_fence_after();
          // (two bodies: with the mask's comparisons in one, every column paid for them)
          if (__all_sync(0xffffffffu, lim == KT && c2 >= 0.f))
            softmax_tile<true, D>(s_t, o_t, c2, lim, i > 0, mref, l, sm.p_full[x]);
          else
            softmax_tile<false, D>(s_t, o_t, c2, lim, i > 0, mref, l, sm.p_full[x]);
        }
        if (!ok || !wait(sm, &sm.o_full[x], items & 1, err)) { ok = false; break; }
        tc_fence_after();
        ++items;
        const int64_t qrow = (r.v.tok0 + t_in) * a.hq + r.g * a.G + h;
        const int prow = x * half_toks * a.G + row;       // = token of the tile * G + head
        const int64_t slot = 2 * (int64_t)blockIdx.x + (first_item ? 0 : 1);
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t ov[32];
          tmem_ld32(o_t + q * 32, ov);
          tmem_ld_wait();
          if (!on) continue;
          // (32 bytes a store: a warp's rows are D elements apart, and each store of 16 would
          // touch the same 32 lines again)
          if (whole) {
            __nv_bfloat16* dst = o + qrow * D + q * 32;
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * inv,
                                 __uint_as_float(ov[2 * e + 1]) * inv);
            if (wide) {
              st_global_v8(dst, w);
              st_global_v8(dst + 16, w + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4*>(dst)[e] =
                    make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
          } else {
            float* dst = parts.o + (slot * kPagedMaxRows + prow) * D + q * 32;
#pragma unroll
            for (int k = 0; k < 4; ++k) st_global_v8(dst + 8 * k, ov + 8 * k);
          }
        }
        tc_fence_before();
        mbar_arrive(&sm.o_empty[x]);
        if (on) {
          if (!whole) parts.ml[slot * kPagedMaxRows + prow] = make_float2(mref, l);
          else if (lse != nullptr)
            lse[qrow] = l != 0.f ? (mref + log2f(l)) * kLn2 : -CUDART_INF_F;
        }
      }
      if (!whole && tile0 == 0 && tid == 0) parts.rec[blockIdx.x] = item_record(a, r, first_item);
      first_item = false;
    } while (ok && run_next<KT>(a, r));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t run(PagedAttn& a, const HeadShape& s, const void* q, const void* kp, const void* vp,
                void* o, float* lse, const PagedParts& parts, int* err, cudaStream_t st) {
  const int half_toks = kHalfRows / a.G;
  a.tt = 2 * half_toks;
  a.lead = kLead;
  int box = 16;                                           // keys of one copy: they share a page
  while (box < KT && a.g.page % (2 * box) == 0) box *= 2;
  const int64_t pool = a.g.n_pages * a.hkv * a.g.page;
  CUtensorMap mq{}, mk{}, mv{};
  if (!make_bf16_heads_map(&mq, q, s.n_tok, s.hq, D, a.qs, a.G, half_toks) ||
      !make_bf16_2d_map(&mk, kp, pool, D, box) || !make_bf16_2d_map(&mv, vp, pool, D, box))
    return cudaErrorInvalidValue;
  const size_t smem = 1024 + 2 * (D / 64) * kHalf + kUnits<D> * kUnit<D> + sizeof(Shared<D>);
  static DeviceOnce done;
  cudaError_t e = raise_smem((const void*)paged_chunk_kernel<D>, smem, &done);
  if (e != cudaSuccess) return e;
  const int grid = paged_grid();
  paged_chunk_kernel<D><<<grid, kThreads, smem, st>>>(mq, mk, mv, box, (__nv_bfloat16*)o, lse,
                                                      parts, err, a);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_paged_combine(s, a, grid, kPagedMaxRows, parts, o, lse, st) : e;
}

}  // namespace

cudaError_t launch_paged_chunk(const HeadShape& s, PagedAttn a, const void* q, const void* kp,
                               const void* vp, void* o, float* lse, const PagedParts& parts,
                               int* err, cudaStream_t st) {
  return s.d == 128 ? run<128>(a, s, q, kp, vp, o, lse, parts, err, st)
                    : run<64>(a, s, q, kp, vp, o, lse, parts, err, st);
}

}  // namespace msa
