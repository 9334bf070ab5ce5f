// The ring that feeds the attention kernels over a paged cache whose bound is the cache's stream:
// a producer warp copies the key and value tiles of a CTA's run, in order, by tensor maps over
// the pools; consumer warps read them.  A tile is KT keys; in shared memory a row of E-byte
// elements lies as D * E / 128 slices of 128 bytes, slice by slice: row r of a slice at r * 128,
// its 16-byte chunk c at c ^ (r % 8) (the 128-byte swizzle).  One box holds the keys that share a
// page; page numbers are fetched 32 boxes ahead.
#pragma once

#include "paged.cuh"
#include "sm100.cuh"

namespace msa {
namespace paged {

using namespace sm100;

constexpr int KT = 32;                // keys of a tile
constexpr uint32_t kSlice = KT * 128; // bytes of 32 keys x 128

template <int D, int E> constexpr int kSlices = D * E / 128;
template <int D, int E> constexpr uint32_t kTileBytes = KT * D * E;
template <int D, int E> constexpr uint32_t kStageBytes = 2 * kTileBytes<D, E>;

// ST stages.  Where a tile belongs to one of W warps, ST is a multiple of W, so that a stage
// always belongs to the same warp: a parity wait tells a phase only from its neighbours, and a
// warp that took over another's stage could be a whole round ahead of a copy that is late.
template <int ST, int W>
struct __align__(16) Ring {
  static_assert(ST % W == 0, "a stage keeps its warp");
  uint64_t full[ST], empty[ST];
  int abort;
  PlanSmem plan;
};

template <int ST, int W>
__device__ __forceinline__ void ring_fail(Ring<ST, W>& sm, int* err) {
  set_device_error(err, MSA_DEVERR_TIMEOUT);
  *(volatile int*)&sm.abort = 1;
}

// Waits for a phase of one of the ring's barriers, for the whole warp; false when the wait ran
// out (after ~2 s) or another warp's did.
template <int ST, int W>
__device__ __forceinline__ bool ring_wait(Ring<ST, W>& sm, uint64_t* bar, uint32_t parity,
                                          int* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  const long long t0 = clock64();
  while (!ok && *(volatile int*)&sm.abort == 0 && clock64() - t0 < MSA_WAIT_CLOCKS)
    ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  if (threadIdx.x % 32 == 0) ring_fail(sm, err);
  return false;
}

// The producer warp: copies every tile of the run, in order.  It is ahead of the consumers, so it
// also asks for an item's queries to L2 (256 short sequences: 52 -> 50 us).
template <int D, int E, int ST, int W>
__device__ __forceinline__ void produce(const CUtensorMap& tm_k, const CUtensorMap& tm_v, int box,
                                        unsigned char* ring, Ring<ST, W>& sm, Run r, int* err,
                                        const void* q, const PagedAttn& a) {
  const int lane = threadIdx.x % 32;
  const int per = KT / box;                               // page pieces of a tile
  const int rows = (int)(a.g.n_pages * a.hkv * a.g.page);
  int step = 0, st = 0;                                   // copies so far; the next one's stage
  uint32_t ph = 1;                                        // of the stage's empty barrier
  bool ok = true;
  do {
    const int tile0 = run_first(a, r), nt = run_tiles(a, r), vis = tile_keys(a, r.v, r.rt);
    if (nt == 0) break;                                   // the run ends in the item's lead
    for (int t = r.rt * a.tt + lane; t < min(r.v.n, (r.rt + 1) * a.tt); t += 32)
      prefetch_l2((const char*)q + ((r.v.tok0 + t) * a.qs + (int64_t)r.g * a.G * D) * E,
                  a.G * D * E);
    // row of piece i of the item's part of this run in the pools, `rows` (reads as zeros)
    // for an entry that is no page, -1 past the last visible key
    auto piece_row = [&](int i) -> int {
      const int key = tile0 * KT + i * box;
      if (i >= nt * per || key >= vis) return -1;
      const int pg = key_page(a, r.s, key, err);
      return pg < 0 ? rows : (int)(((int64_t)pg * a.hkv + r.g) * a.g.page + key % (int)a.g.page);
    };
    int cur = piece_row(lane), nxt = piece_row(32 + lane);
    for (int it = 0; it < nt; ++it, ++step) {
      const int at = it * per;                            // first piece of the tile
      if (at > 0 && at % 32 == 0) {
        cur = nxt;
        nxt = piece_row(at + 32 + lane);
      }
      // (the first pass over the ring waits for the phase before the first: it is over)
      if (!ring_wait(sm, &sm.empty[st], ph, err)) {
        ok = false;
        break;
      }
      const int y = __shfl_sync(0xffffffffu, cur, (at & 31) + (lane < per ? lane : 0));
      const bool mine = lane < per && y >= 0;
      const int n = __popc(__ballot_sync(0xffffffffu, mine));
      if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], (uint32_t)(n * box * D * E * 2));
      __syncwarp();
      if (mine && step != MSA_LOSE_COPY) {
        unsigned char* dst = ring + st * kStageBytes<D, E> + lane * box * 128;
#pragma unroll
        for (int h = 0; h < kSlices<D, E>; ++h) {
          const int x = h * (128 / E);
          tma_load_2d(dst + h * kSlice, &tm_k, &sm.full[st], x, y);
          tma_load_2d(dst + kTileBytes<D, E> + h * kSlice, &tm_v, &sm.full[st], x, y);
        }
      }
      if (++st == ST) {
        st = 0;
        ph ^= 1;
      }
    }
  } while (ok && run_next<KT>(a, r));
  // No copy may land after the CTA ends, whoever gave up (in a run shorter than the ring the
  // consumers alone may): the last one of every stage is waited for.
  for (int s = step > ST ? step - ST : 0; s < step; ++s)
    mbar_wait_warp(&sm.full[s % ST], (uint32_t)(s / ST) & 1);
}

// Set-up: barriers (readers: warps that read a stage), this CTA's record, the run.
template <int THREADS, int ST, int W>
__device__ __forceinline__ Run begin(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                     Ring<ST, W>& sm, int readers, const PagedParts& parts,
                                     const PagedAttn& a) {
  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], readers);
    }
    sm.abort = 0;
    fence_mbar_init();
    parts.rec[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  return paged_plan<KT, THREADS>(a, &sm.plan);           // synchronises the CTA
}

template <int D, int E, int ST, int W>
constexpr size_t ring_bytes() { return 1024 + ST * kStageBytes<D, E> + sizeof(Ring<ST, W>); }

// Tensor maps over both pools, boxes of the keys that are sure to share a page.
inline bool pool_maps(const PagedAttn& a, const HeadShape& s, const void* kp, const void* vp,
                      CUtensorMap* mk, CUtensorMap* mv, int* box) {
  *box = a.g.page % 32 == 0 ? 32 : 16;
  const int64_t rows = a.g.n_pages * a.hkv * a.g.page;
  return make_2d_map(mk, kp, s.dtype, rows, s.d, *box) &&
         make_2d_map(mv, vp, s.dtype, rows, s.d, *box);
}

}  // namespace paged
}  // namespace msa
