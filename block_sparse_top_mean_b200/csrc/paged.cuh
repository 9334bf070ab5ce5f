// Paged key/value caches: the shapes, the schedule of the attention kernels over them, and
// the partial results that their CTAs leave for paged_combine_kernel.
//
// Pools k_pages, v_pages [n_pages, hkv, page, d]; sequence s holds kv_lens[s] tokens, token p
// in slot p % page of page table[s][p / page]; its last n_s = cu[s+1] - cu[s] tokens are the
// new ones, packed tokens cu[s].. of q and o.  A new token at position pos sees keys p <= pos.
//
// Rows.  The G = hq / hkv query heads of a KV head share its keys, so a row tile is TT tokens
// x G heads (row = token * G + head) against tiles of KT keys.  An item is (sequence, KV
// head, row tile); its key tiles are those up to its last token's position (at least one, so
// that rows that see nothing are still written).
//
// Schedule.  An item counts as its key tiles plus `lead` (what starting and finishing an item
// costs, in tiles).  All items, in order, are one line that the CTAs cut into equal runs (a
// run may start and end inside an item), so the work is even whatever the lengths are: one
// long sequence, or many of very different lengths.  Every CTA finds its run itself from cu
// and kv_lens (a scan over the sequences), so the lengths may change between replays of a
// captured graph.  An item that one CTA holds whole is finished there; of one that is cut,
// each CTA leaves its running maximum, sum and unnormalised output (fp32), and the CTA that
// holds the item's first tile a record of how many parts there are.  Parts are joined in
// order: results do not depend on timing.
#pragma once

#include <math_constants.h>

#include "common.cuh"
#include "device_once.cuh"

namespace msa {

struct HeadShape {
  int64_t n_tok, hq, hkv, d;
  int dtype;
};

struct PagedShape {
  const int32_t* table;               // [n_seqs, max_pages]
  const int32_t* kv_lens;             // [n_seqs]
  const int32_t* cu;                  // [n_seqs + 1]
  int64_t n_seqs, max_pages, n_pages, page;
};

// qk_norm_rope.cu.  part: [qk_norm_rope_bwd_ctas()][d] fp32.
int64_t qk_norm_rope_bwd_ctas();
cudaError_t launch_qk_norm_rope(const HeadShape& s, const int32_t* cu, int64_t n_docs,
                                const void* q, int64_t qs, const void* k, int64_t ks,
                                const void* wq, const void* wk, double base, float eps, void* qo,
                                void* ko, cudaStream_t st);
cudaError_t launch_qk_norm_rope_bwd(const HeadShape& s, const int32_t* cu, int64_t n_docs,
                                    const void* dq, const void* dk, int grad_dtype, const void* q,
                                    int64_t qs, const void* k, int64_t ks, const void* wq,
                                    const void* wk, double base, float eps, void* dqi, void* dki,
                                    float* dwq, float* dwk, float* part, cudaStream_t st);
// paged_append.cu.  q may be null; base 0: no rotation; eps 0: no norm.
cudaError_t launch_paged_append(const HeadShape& s, const PagedShape& g, const void* q, int64_t qs,
                                const void* k, int64_t ks, const void* v, int64_t vs,
                                const void* wq, const void* wk, double base, float eps, void* kp,
                                void* vp, void* qo, int* err, cudaStream_t st);

// Attention over a paged cache.
struct PagedAttn {
  PagedShape g;
  int64_t n_tok, qs;                  // packed tokens, q's token stride (elements)
  int hq, hkv, G, tt;                 // tt: tokens of a row tile
  int lead;                           // cost of an item beside its tiles (in tiles)
  int min_new, max_new;               // the launch takes sequences with this many new tokens
  float scale_log2;                   // softmax scale * log2(e)
};

size_t paged_attn_ws_bytes(const HeadShape& s);
int paged_grid();                     // CTAs of a schedule: one an SM
// Raises a kernel's shared memory limit on the current device, once (done: the kernel's own
// record of the devices where that happened).
cudaError_t raise_smem(const void* kernel, size_t bytes, DeviceOnce* done);
// Each kernel takes the sequences with a.min_new .. a.max_new new tokens, whatever their rows.
// rows: the row tile asked for (at least G).  step: bf16, up to 16 rows; f32: fp32; chunk: bf16
// on the tensor cores, row tiles of 2 x 128 rows.
cudaError_t launch_paged_step(const HeadShape& s, PagedAttn a, int rows, const void* q,
                             const void* kp, const void* vp, void* o, float* lse,
                             const struct PagedParts& parts, int* err, cudaStream_t st);
cudaError_t launch_paged_chunk(const HeadShape& s, PagedAttn a, const void* q, const void* kp,
                               const void* vp, void* o, float* lse,
                               const struct PagedParts& parts, int* err, cudaStream_t st);
cudaError_t launch_paged_f32(const HeadShape& s, PagedAttn a, int rows, const void* q,
                              const void* kp, const void* vp, void* o, float* lse,
                              const struct PagedParts& parts, int* err, cudaStream_t st);
cudaError_t launch_paged_combine(const HeadShape& s, const PagedAttn& a, int grid, int rows,
                                 const struct PagedParts& parts, void* o, float* lse,
                                 cudaStream_t st);
cudaError_t launch_paged_attn(const HeadShape& s, const PagedShape& g, int64_t max_new,
                              float scale, const void* q, int64_t qs, const void* kp,
                              const void* vp, void* o, float* lse, char* ws, int* err,
                              cudaStream_t st);

// Workspace of one of these operators (msa_workspace_bytes); 0 for invalid shapes.
size_t layer_ws_bytes(const msa_params* p, int32_t op);

constexpr int kPagedCtas = 160;       // most SMs a schedule uses (a B200 has 148)
constexpr int kPagedRecs = 2 * kPagedCtas;       // most CTAs: two an SM with row tiles of up to 64
constexpr int kPagedMaxRows = 256;    // rows of the largest row tile (one CTA an SM)

// A build that tests how the kernels give up loses this copy of every CTA's stream.
#ifndef MSA_LOSE_COPY
#define MSA_LOSE_COPY -1
#endif

// Workspace body: records, then (maximum, sum) and outputs of the parts.  CTA c's parts: 2c
// (its first item) and 2c + 1 (its last, when that is another).  Sized for one CTA an SM with
// row tiles of kPagedMaxRows; smaller row tiles leave room for more CTAs.
struct PagedParts {
  int4* rec;                          // [kPagedRecs], see item_record
  float2* ml;                         // [2 * CTAs][rows]
  float* o;                           // [2 * CTAs][rows][d]
};

// ------------------------------------------------------------------ device side
struct SeqView {
  int64_t tok0;                       // first packed token
  int n, past, cap, n_rt;             // new tokens, tokens before them, keys there are, tiles
};

__device__ __forceinline__ SeqView load_seq(const PagedAttn& a, int s) {
  SeqView v;
  const int64_t c0 = max((int64_t)0, min((int64_t)__ldg(a.g.cu + s), a.n_tok));
  const int64_t c1 = max(c0, min((int64_t)__ldg(a.g.cu + s + 1), a.n_tok));
  const int len = max(0, __ldg(a.g.kv_lens + s));
  const int64_t room = a.g.max_pages * a.g.page;
  v.tok0 = c0;
  v.n = (int)(c1 - c0);
  v.past = len - v.n;
  v.cap = (int)max((int64_t)0, min((int64_t)len, room));
  v.n_rt = v.n < a.min_new || v.n > a.max_new ? 0 : (v.n + a.tt - 1) / a.tt;
  return v;
}
// Keys that the last token of row tile rt sees.  (32 bits hold it: past + n is the length.)
__device__ __forceinline__ int tile_keys(const PagedAttn& a, const SeqView& v, int rt) {
  const int toks = (int)min((uint32_t)v.n, (uint32_t)(rt + 1) * (uint32_t)a.tt);
  return max(0, min(v.past + toks, v.cap));
}
template <int KT>
__device__ __forceinline__ int key_tiles(const PagedAttn& a, const SeqView& v, int rt) {
  return max(1, (int)(((uint32_t)tile_keys(a, v, rt) + KT - 1) / KT));
}

// sum_{i < n} floor((p i + q) / m) for 0 <= p, q and p (n - 1) + q < 2^31 (the Euclidean
// algorithm on lattice points under a line: Graham, Knuth, Patashnik, Concrete Mathematics, 3.5).
__device__ __forceinline__ int64_t floor_sum(int n, uint32_t m, uint32_t p, uint32_t q) {
  int64_t sum = 0;
  for (;;) {
    if (p >= m) {
      sum += (int64_t)n * (n - 1) / 2 * (p / m);
      p %= m;
    }
    if (q >= m) {
      sum += (int64_t)n * (q / m);
      q %= m;
    }
    const uint64_t y = (uint64_t)p * n + q;               // height of the line's end
    if (y < m) return sum;
    n = (int)((uint32_t)y / m);
    q = (uint32_t)y % m;
    const uint32_t t = m;
    m = p;
    p = t;
  }
}
// Cost of the first k row tiles of one KV head of a sequence: their key tiles and leads.  Row
// tile i ends at key min(past + (i + 1) tt, cap): up to KT keys count as one tile, those that
// reach cap as many as cap fills, the ones between as ceil of an arithmetic progression.
template <int KT>
__device__ __forceinline__ int64_t rows_cost(const PagedAttn& a, const SeqView& v, int k) {
  int64_t t = (int64_t)k * a.lead;
  if (k <= 16) {                      // (cheaper than the closed form's divisions)
    int sum = 0;                      // below 2^31: 16 rows of at most 2^31 / KT tiles
    for (int rt = 0; rt < k; ++rt) sum += key_tiles<KT>(a, v, rt);
    return t + sum;
  }
  if (v.cap <= KT) return t + k;      // every row tile counts one
  // row tiles that end at or before KT, and before cap
  const uint32_t tt = a.tt;
  const int one = min(k, v.past >= KT ? 0 : (int)((uint32_t)(KT - v.past) / tt));
  const int before = v.cap <= v.past ? 0 : (int)(((uint32_t)(v.cap - v.past) + tt - 1) / tt) - 1;
  const int to = min(k, max(one, before));
  t += one + (int64_t)(k - to) * ((v.cap + KT - 1) / KT);
  if (to > one)
    t += floor_sum(to - one, KT, tt, (uint32_t)v.past + (uint32_t)(one + 1) * tt + KT - 1);
  return t;
}
template <int KT>
__device__ __forceinline__ int64_t group_cost(const PagedAttn& a, const SeqView& v) {
  return rows_cost<KT>(a, v, v.n_rt);
}

// A CTA's run [at, end) of the line and the item it is in: `tiles` tiles from `start` + lead on
// the line.
struct Run {
  int64_t at, end, start;
  int64_t share;                      // length of a run
  int s, g, rt, tiles;
  SeqView v;
};

struct PlanSmem {
  int64_t warp_sum[32];
  Run run;
};

// Every thread of the CTA calls this; the result is the same in all of them.
template <int KT, int THREADS>
__device__ __forceinline__ Run paged_plan(const PagedAttn& a, PlanSmem* sm) {
  constexpr int W = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = (int)a.g.n_seqs;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // paged_combine_kernel
  auto tiles_of = [&](int s) -> int64_t {
    return s < n ? group_cost<KT>(a, load_seq(a, s)) * a.hkv : 0;
  };
  // total of all sequences
  int64_t mine = tiles_of(tid);
  int64_t sum = mine;
  for (int s = tid + THREADS; s < n; s += THREADS) sum += tiles_of(s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sm->warp_sum[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) total += sm->warp_sum[w];
  const int64_t share = max((int64_t)1, (total + gridDim.x - 1) / gridDim.x);
  const int64_t w0 = share * blockIdx.x, w1 = min(total, w0 + share);
  if (tid == 0) sm->run.at = sm->run.end = 0;
  // the sequence that holds w0
  int64_t before = 0;
  for (int s0 = 0; s0 < n && w0 < total; s0 += THREADS) {
    if (s0 > 0) mine = tiles_of(s0 + tid);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) sm->warp_sum[warp] = incl;
    __syncthreads();
    int64_t base = before;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) base += sm->warp_sum[w];
      before += sm->warp_sum[w];
    }
    const int64_t lo = base + incl - mine;
    if (w0 >= lo && w0 < lo + mine) {
      Run r;
      r.at = w0;
      r.end = w1;
      r.share = share;
      r.s = s0 + tid;
      r.v = load_seq(a, r.s);
      const int64_t per = mine / a.hkv;
      r.g = (int)((w0 - lo) / per);
      r.start = lo + r.g * per;
      // the last row tile that starts at or before w0
      int rt = 0, n_rt = r.v.n_rt;
      while (n_rt > 1) {
        const int half = n_rt / 2;
        if (r.start + rows_cost<KT>(a, r.v, rt + half) <= w0) {
          rt += half;
          n_rt -= half;
        } else {
          n_rt = half;
        }
      }
      r.start += rows_cost<KT>(a, r.v, rt);
      r.rt = rt;
      r.tiles = key_tiles<KT>(a, r.v, rt);
      sm->run = r;
    }
    if (before > w0) break;
  }
  __syncthreads();
  return sm->run;
}

// First tile of the current item that belongs to the run, and how many do (none when the run
// ends in the item's lead).
__device__ __forceinline__ int run_first(const PagedAttn& a, const Run& r) {
  return (int)max((int64_t)0, r.at - r.start - a.lead);
}
__device__ __forceinline__ int run_tiles(const PagedAttn& a, const Run& r) {
  const int64_t to = min((int64_t)r.tiles, r.end - r.start - a.lead);
  return (int)max((int64_t)0, to - run_first(a, r));
}
// Steps to the next item.  Returns false when the run is over.
template <int KT>
__device__ __forceinline__ bool run_next(const PagedAttn& a, Run& r) {
  r.start += a.lead + r.tiles;
  if (r.start >= r.end) return false;
  r.at = r.start;
  if (++r.rt >= r.v.n_rt) {
    r.rt = 0;
    if (++r.g >= a.hkv) {
      r.g = 0;
      do {
        if (++r.s >= (int)a.g.n_seqs) return false;       // (lengths that changed meanwhile)
        r.v = load_seq(a, r.s);
      } while (r.v.n_rt == 0);
    }
  }
  r.tiles = key_tiles<KT>(a, r.v, r.rt);
  return true;
}

// Runs that the current item's tiles reach into.
__device__ __forceinline__ int item_parts(const PagedAttn& a, const Run& r) {
  const int64_t first = r.start + a.lead;
  return (int)((first + r.tiles - 1) / r.share - first / r.share) + 1;
}

// The record of a cut item: row of its first query in o and lse (low and high word), its
// tokens << 1 | which of the CTA's two parts it is, and the number of parts.
__device__ __forceinline__ int4 item_record(const PagedAttn& a, const Run& r, bool first_item) {
  const int64_t row = (r.v.tok0 + (int64_t)r.rt * a.tt) * a.hq + r.g * a.G;
  const int toks = min(a.tt, r.v.n - r.rt * a.tt);
  return make_int4((int)(row & 0xffffffff), (int)(row >> 32), toks << 1 | (first_item ? 0 : 1),
                   item_parts(a, r));
}

// The page of key `key` of a sequence, -1 (and the error bit) when the table holds none.
__device__ __forceinline__ int key_page(const PagedAttn& a, int s, int key, int* err) {
  const int pg = __ldg(a.g.table + (int64_t)s * a.g.max_pages + key / (int)a.g.page);
  if (pg >= 0 && pg < a.g.n_pages) return pg;
  set_device_error(err, MSA_DEVERR_PAGE_RANGE);
  return -1;
}

}  // namespace msa
