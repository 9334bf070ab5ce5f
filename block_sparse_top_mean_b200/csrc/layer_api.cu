// C entries of the dense-layer operators (include/msa.h): per-head norm with rotation and
// its backward, the append to a paged cache, and the attention of new tokens over it.
// Every check runs on the host before anything is launched.
#include <math.h>

#include "paged.cuh"

namespace {

using msa::HeadShape;
using msa::PagedShape;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
msa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

constexpr int64_t kMaxTokens = INT32_MAX;
constexpr int64_t kAhead = 1 << 14;   // 64 pieces of at most 128 keys, and a tile
constexpr int64_t kMaxGroup = 64;     // query heads of a KV head

msa_status check_heads(const msa_params* p, HeadShape* s) {
  if (p == nullptr) return MSA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->seq < 0 || p->hq < 1 || p->hkv < 1 || p->d < 1 || p->hq % p->hkv != 0)
    return MSA_ERR_INVALID_ARG;
  if (p->dtype != MSA_F32 && p->dtype != MSA_BF16) return MSA_ERR_INVALID_ARG;
  if (p->d != 64 && p->d != 128) return MSA_ERR_UNSUPPORTED;
  if (p->hq > 65535 || p->hq / p->hkv > kMaxGroup) return MSA_ERR_UNSUPPORTED;
  s->hq = p->hq;
  s->hkv = p->hkv;
  s->d = p->d;
  s->dtype = p->dtype;
  s->n_tok = p->seq;
  return MSA_OK;
}

// Packed tokens of a norm call: batch * seq.
msa_status check_packed(const msa_params* p, HeadShape* s) {
  msa_status st = check_heads(p, s);
  if (st != MSA_OK) return st;
  if (p->batch > kMaxTokens || p->seq > kMaxTokens || p->batch * p->seq > kMaxTokens)
    return MSA_ERR_UNSUPPORTED;
  s->n_tok = p->batch * p->seq;
  return MSA_OK;
}

// A token stride (elements; 0 = heads * d): 16-byte steps, at least one token's heads.
bool stride_ok(const HeadShape& s, int64_t heads, int64_t* stride) {
  if (*stride == 0) *stride = heads * s.d;
  const int64_t es = s.dtype == MSA_BF16 ? 2 : 4;
  return *stride >= heads * s.d && *stride * es % 16 == 0 && *stride < ((int64_t)1 << 32);
}

msa_status check_norm(const HeadShape& s, const int32_t* cu, int64_t n_docs, const void* q,
                      int64_t* qs, const void* k, int64_t* ks, const void* wq, const void* wk,
                      double base, float eps) {
  if (n_docs < 1 || !(base > 1.0) || !isfinite(base) || !(eps > 0.f) || !isfinite(eps))
    return MSA_ERR_INVALID_ARG;
  if (!stride_ok(s, s.hq, qs) || !stride_ok(s, s.hkv, ks)) return MSA_ERR_INVALID_ARG;
  if (n_docs >= INT32_MAX) return MSA_ERR_UNSUPPORTED;
  if (s.n_tok == 0) return MSA_OK;
  if (cu == nullptr || q == nullptr || k == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned(cu, 4) || !aligned(q, 16) || !aligned(k, 16) || !aligned(wq, 16) ||
      !aligned(wk, 16))
    return MSA_ERR_INVALID_ARG;
  return MSA_OK;
}

// Shapes of a paged call: batch sequences, seq packed new tokens, block tokens a page.
msa_status check_paged(const msa_params* p, const msa_paged_cache* c, HeadShape* s,
                       PagedShape* g) {
  msa_status st = check_heads(p, s);
  if (st != MSA_OK) return st;
  if (c == nullptr || p->block < 1 || c->n_pages < 0 || c->max_pages < 0)
    return MSA_ERR_INVALID_ARG;
  if (p->block % 16 != 0 || p->block > (1 << 20)) return MSA_ERR_UNSUPPORTED;
  if (p->batch >= INT32_MAX || p->seq > kMaxTokens) return MSA_ERR_UNSUPPORTED;
  // rows of a pool and keys of a table row are counted in 32 bits, and the kernels look up to
  // kAhead keys past the last one
  if (c->n_pages > INT32_MAX / (p->hkv * p->block) ||
      c->max_pages > (INT32_MAX - kAhead) / p->block)
    return MSA_ERR_UNSUPPORTED;
  g->table = c->page_table;
  g->kv_lens = c->kv_lens;
  g->cu = c->cu_seqlens;
  g->n_seqs = p->batch;
  g->max_pages = c->max_pages;
  g->n_pages = c->n_pages;
  g->page = p->block;
  if (p->batch == 0 || p->seq == 0) return MSA_OK;
  if (c->cu_seqlens == nullptr || c->kv_lens == nullptr || !aligned(c->cu_seqlens, 4) ||
      !aligned(c->kv_lens, 4) || !aligned(c->page_table, 4))
    return MSA_ERR_INVALID_ARG;
  if (c->max_pages > 0 && c->page_table == nullptr) return MSA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->k_pages == nullptr || c->v_pages == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16)) return MSA_ERR_INVALID_ARG;
  return MSA_OK;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

msa_status check_ws(const void* ws, size_t bytes, size_t need) {
  return ws == nullptr || bytes < need || !aligned(ws, 256) ? MSA_ERR_WORKSPACE : MSA_OK;
}

}  // namespace

namespace msa {

size_t layer_ws_bytes(const msa_params* p, int32_t op) {
  HeadShape s;
  if (check_heads(p, &s) != MSA_OK) return 0;
  switch (op) {
    case MSA_OP_QK_NORM_ROPE_BWD:
      return kWsHeader + (size_t)qk_norm_rope_bwd_ctas() * s.d * sizeof(float);
    case MSA_OP_PAGED_APPEND:
      return kWsHeader;
    case MSA_OP_PAGED_ATTN:
      return kWsHeader + round256(paged_attn_ws_bytes(s));
    default:
      return 0;
  }
}

}  // namespace msa

extern "C" {

msa_status msa_qk_norm_rope(const msa_params* p, const int32_t* cu_seqlens, int64_t n_docs,
                            const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                            const void* wq, const void* wk, double base, float eps, void* q_out,
                            void* k_out, msa_stream_t stream) {
  HeadShape s;
  msa_status st = check_packed(p, &s);
  if (st != MSA_OK) return st;
  st = check_norm(s, cu_seqlens, n_docs, q, &q_stride, k, &k_stride, wq, wk, base, eps);
  if (st != MSA_OK || s.n_tok == 0) return st;
  if (q_out == nullptr || k_out == nullptr || !aligned(q_out, 16) || !aligned(k_out, 16))
    return MSA_ERR_INVALID_ARG;
  // in place only row on row
  if ((q_out == q && q_stride != s.hq * s.d) || (k_out == k && k_stride != s.hkv * s.d))
    return MSA_ERR_INVALID_ARG;
  return cuda_status(msa::launch_qk_norm_rope(s, cu_seqlens, n_docs, q, q_stride, k, k_stride, wq,
                                              wk, base, eps, q_out, k_out, (cudaStream_t)stream));
}

msa_status msa_qk_norm_rope_bwd(const msa_params* p, const int32_t* cu_seqlens, int64_t n_docs,
                                const void* dq_out, const void* dk_out, int32_t grad_dtype,
                                const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                const void* wq, const void* wk, double base, float eps, void* dq,
                                void* dk, float* dwq, float* dwk, void* ws, size_t ws_bytes,
                                msa_stream_t stream) {
  HeadShape s;
  msa_status st = check_packed(p, &s);
  if (st != MSA_OK) return st;
  if (grad_dtype != MSA_F32 && grad_dtype != p->dtype) return MSA_ERR_INVALID_ARG;
  st = check_norm(s, cu_seqlens, n_docs, q, &q_stride, k, &k_stride, wq, wk, base, eps);
  if (st != MSA_OK) return st;
  cudaStream_t cs = (cudaStream_t)stream;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return MSA_ERR_INVALID_ARG;
  if (s.n_tok == 0) {                  // no token: the weights' gradients are zero
    cudaError_t e = cudaSuccess;
    if (dwq != nullptr) e = cudaMemsetAsync(dwq, 0, s.d * sizeof(float), cs);
    if (e == cudaSuccess && dwk != nullptr) e = cudaMemsetAsync(dwk, 0, s.d * sizeof(float), cs);
    return cuda_status(e);
  }
  if (dq_out == nullptr || dk_out == nullptr || dq == nullptr || dk == nullptr ||
      !aligned(dq_out, 16) || !aligned(dk_out, 16) || !aligned(dq, 16) || !aligned(dk, 16))
    return MSA_ERR_INVALID_ARG;
  float* part = nullptr;
  if (dwq != nullptr || dwk != nullptr) {
    st = check_ws(ws, ws_bytes, msa::layer_ws_bytes(p, MSA_OP_QK_NORM_ROPE_BWD));
    if (st != MSA_OK) return st;
    part = reinterpret_cast<float*>((char*)ws + msa::kWsHeader);
  }
  return cuda_status(msa::launch_qk_norm_rope_bwd(s, cu_seqlens, n_docs, dq_out, dk_out,
                                                  grad_dtype, q, q_stride, k, k_stride, wq, wk,
                                                  base, eps, dq, dk, dwq, dwk, part, cs));
}

msa_status msa_paged_append(const msa_params* p, const msa_paged_cache* cache, const void* q,
                            int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, const void* wq, const void* wk, double base,
                            float eps, void* q_out, void* ws, size_t ws_bytes,
                            msa_stream_t stream) {
  HeadShape s;
  PagedShape g;
  msa_status st = check_paged(p, cache, &s, &g);
  if (st != MSA_OK) return st;
  if (!(base == 0.0 || (base > 1.0 && isfinite(base))) || !(eps >= 0.f) || !isfinite(eps))
    return MSA_ERR_INVALID_ARG;
  if (!stride_ok(s, s.hq, &q_stride) || !stride_ok(s, s.hkv, &k_stride) ||
      !stride_ok(s, s.hkv, &v_stride))
    return MSA_ERR_INVALID_ARG;
  if (eps == 0.f && (wq != nullptr || wk != nullptr)) return MSA_ERR_INVALID_ARG;
  if (p->batch == 0 || s.n_tok == 0) return MSA_OK;
  if (k == nullptr || v == nullptr || (q == nullptr) != (q_out == nullptr))
    return MSA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(wq, 16) ||
      !aligned(wk, 16) || !aligned(q_out, 16))
    return MSA_ERR_INVALID_ARG;
  if (q != nullptr && q_out == q && q_stride != s.hq * s.d) return MSA_ERR_INVALID_ARG;
  if (ws != nullptr && (st = check_ws(ws, ws_bytes, msa::kWsHeader)) != MSA_OK) return st;
  return cuda_status(msa::launch_paged_append(s, g, q, q_stride, k, k_stride, v, v_stride, wq, wk,
                                              base, eps, cache->k_pages, cache->v_pages, q_out,
                                              reinterpret_cast<int*>(ws), (cudaStream_t)stream));
}

msa_status msa_paged_attn_fwd(const msa_params* p, const msa_paged_cache* cache, int64_t max_new,
                              const void* q, int64_t q_stride, void* o, float* lse, void* ws,
                              size_t ws_bytes, msa_stream_t stream) {
  HeadShape s;
  PagedShape g;
  msa_status st = check_paged(p, cache, &s, &g);
  if (st != MSA_OK) return st;
  // (the kernels scale to base 2: that factor has to be finite as well)
  if (!isfinite(p->scale * 1.4426950408889634f) || max_new < 0) return MSA_ERR_INVALID_ARG;
  if (!stride_ok(s, s.hq, &q_stride)) return MSA_ERR_INVALID_ARG;
  if (p->batch == 0 || s.n_tok == 0) return MSA_OK;
  if (q == nullptr || o == nullptr || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return MSA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, msa::layer_ws_bytes(p, MSA_OP_PAGED_ATTN))) != MSA_OK)
    return st;
  return cuda_status(msa::launch_paged_attn(
      s, g, max_new, p->scale, q, q_stride, cache->k_pages, cache->v_pages, o, lse,
      (char*)ws + msa::kWsHeader, reinterpret_cast<int*>(ws), (cudaStream_t)stream));
}

}  // extern "C"
