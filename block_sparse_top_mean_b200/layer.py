"""Operators round a full-attention layer: per-head norms of queries and keys with the
rotation (and their gradient), the append of new tokens to a paged key/value cache, and the
attention of new tokens over that cache.  Binding of the msa_qk_norm_rope* and msa_paged_*
entries of include/msa.h; the names here are the package's (`msa.qk_norm_rope`, ...).

Every call runs on the current stream of its tensors' device, whichever device is current,
allocates nothing but its outputs (and the workspace where none is given) and can be
captured into a CUDA graph.  Tensors that live on another stream than the current one are
the caller's to order, as with any torch operation."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MSA_BF16, MSA_F32, MsaError, MsaPagedCache, MsaParams

_DT = {torch.float32: MSA_F32, torch.bfloat16: MSA_BF16}
_byref = ctypes.byref


def _fail(text):
    raise ValueError(text)


def _call(name, device, *args):
    """The library's entry on `device`'s current stream (launches need it to be current)."""
    fn = getattr(_lib.load(), name)
    # the raw handle: building a torch.cuda.Stream object costs 2 us of a 10 us call
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != 0:
        _lib.check(name, st)


def _rows(name, x, d, dtype, device):
    """Checks x [T, heads, d] with packed heads and returns its token stride."""
    if x.dtype != dtype or x.device != device:
        _fail(f"{name} must be {dtype} on {device}")
    if x.dim() != 3 or x.shape[2] != d:
        _fail(f"{name} must be [tokens, heads, {d}]")
    T, h, _ = x.shape
    s0, s1, s2 = x.stride()
    if (s2 != 1 or (s1 != d and h > 1)) and x.numel():
        _fail(f"{name}: the heads of a token must be packed (only the token stride is free)")
    return s0 if T > 1 else h * d


def _ints(name, x, shape, device):
    if x.dtype != torch.int32 or x.device != device or not x.is_contiguous():
        _fail(f"{name} must be a contiguous int32 tensor on {device}")
    if x.dim() != len(shape) or any(b is not None and a != b for a, b in zip(x.shape, shape)):
        _fail(f"{name} must have shape {shape}")


def _weight(name, w, d, dtype, device):
    if w is None:
        return None
    if w.dtype != dtype or w.device != device or w.shape != (d,) or not w.is_contiguous():
        _fail(f"{name} must be a contiguous [{d}] {dtype} tensor on {device}")
    return w.data_ptr()


def _out(name, x, shape, dtype, device):
    if x is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if x.dtype != dtype or x.device != device or tuple(x.shape) != tuple(shape) or \
            not x.is_contiguous():
        _fail(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {device}")
    return x


def _head_shape(q, k):
    if not q.is_cuda:
        _fail("block_sparse_top_mean_b200 takes CUDA tensors only")
    if q.dtype not in _DT:
        _fail("tensors must be float32 or bfloat16")
    if q.dim() != 3 or k.dim() != 3:
        _fail("q and k must be [tokens, heads, d]")
    T, hq, d = q.shape
    if k.shape[0] != T:
        _fail("q and k must hold the same tokens")
    return T, hq, k.shape[1], d


def _workspace(p, op, device):
    n = _lib.load().msa_workspace_bytes(_byref(p), op, 0)
    if n == 0:
        raise MsaError("msa_workspace_bytes", _lib.MSA_ERR_INVALID_ARG, "invalid shapes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _ws_ptr(ws, device):
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        _fail(f"ws must be a contiguous uint8 tensor on {device}")
    return ws.data_ptr(), ws.numel()


def _norm_args(q, k, cu_seqlens, wq, wk):
    T, hq, hkv, d = _head_shape(q, k)
    dt, dev = q.dtype, q.device
    qs, ks = _rows("q", q, d, dt, dev), _rows("k", k, d, dt, dev)
    _ints("cu_seqlens", cu_seqlens, (None,), dev)
    p = MsaParams(1, T, hq, hkv, d, 1, 1, 1.0, _DT[dt])
    return (p, dev, dt, (T, hq, d), (T, hkv, d), qs, ks, _weight("wq", wq, d, dt, dev),
            _weight("wk", wk, d, dt, dev))


def qk_norm_rope(q, k, cu_seqlens, base: float, wq=None, wk=None, eps: float = 1e-6, out=None):
    """RMS norm of every head of packed q [T, hq, d] and k [T, hkv, d] (weights wq, wk [d] or
    None for ones), then the rotation by each token's position in its own document
    (cu_seqlens: int32 CUDA tensor of the n_docs + 1 boundaries).  q and k may be strided in
    the token dimension (views of a fused projection).  Returns (q_out, k_out), packed; `out`
    may pass them, or q and k themselves when those are packed."""
    p, dev, dt, sq, sk, qs, ks, pq, pk = _norm_args(q, k, cu_seqlens, wq, wk)
    qo = _out("q_out", None if out is None else out[0], sq, dt, dev)
    ko = _out("k_out", None if out is None else out[1], sk, dt, dev)
    _call("msa_qk_norm_rope", dev, _byref(p), cu_seqlens.data_ptr(), cu_seqlens.numel() - 1,
          q.data_ptr(), qs, k.data_ptr(), ks, pq, pk, base, eps, qo.data_ptr(), ko.data_ptr())
    return qo, ko


def qk_norm_rope_workspace(q, k):
    """A workspace for qk_norm_rope_bwd (it depends on the head shape alone)."""
    T, hq, hkv, d = _head_shape(q, k)
    return _workspace(MsaParams(1, T, hq, hkv, d, 1, 1, 1.0, _DT[q.dtype]),
                      _lib.OP_QK_NORM_ROPE_BWD, q.device)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, cu_seqlens, base: float, wq=None, wk=None,
                     eps: float = 1e-6, ws=None, out=None):
    """Gradient of qk_norm_rope for the upstream gradients dq_out, dk_out (packed; fp32 or the
    inputs' dtype): (dq, dk, dwq, dwk), dq and dk in the inputs' dtype, the weights' gradients
    in fp32.  `out` may pass the four tensors."""
    p, dev, dt, sq, sk, qs, ks, pq, pk = _norm_args(q, k, cu_seqlens, wq, wk)
    gt = dq_out.dtype
    if gt not in (torch.float32, dt):
        _fail(f"the upstream gradients must be float32 or {dt}")
    _out("dq_out", dq_out, sq, gt, dev)
    _out("dk_out", dk_out, sk, gt, dev)
    o = (None,) * 4 if out is None else out
    d = sq[2]
    dq, dk = _out("dq", o[0], sq, dt, dev), _out("dk", o[1], sk, dt, dev)
    dwq, dwk = (_out(n, x, (d,), torch.float32, dev) for n, x in (("dwq", o[2]), ("dwk", o[3])))
    if ws is None:
        ws = _workspace(p, _lib.OP_QK_NORM_ROPE_BWD, dev)
    wp, wn = _ws_ptr(ws, dev)
    _call("msa_qk_norm_rope_bwd", dev, _byref(p), cu_seqlens.data_ptr(), cu_seqlens.numel() - 1,
          dq_out.data_ptr(), dk_out.data_ptr(), _DT[gt], q.data_ptr(), qs, k.data_ptr(), ks, pq,
          pk, base, eps, dq.data_ptr(), dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr(), wp, wn)
    return dq, dk, dwq, dwk


def _cache(k_pages, v_pages, page_table, kv_lens, cu_seqlens, dtype, device):
    """The checked cache of a step and its shape (n_seqs, hkv, page, d)."""
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
        _fail("k_pages and v_pages must both be [n_pages, hkv, page, d]")
    for name, x in (("k_pages", k_pages), ("v_pages", v_pages)):
        if x.dtype != dtype or x.device != device or not x.is_contiguous():
            _fail(f"{name} must be a contiguous {dtype} tensor on {device}")
    n_pages, hkv, page, d = k_pages.shape
    _ints("kv_lens", kv_lens, (None,), device)
    n = kv_lens.numel()
    _ints("page_table", page_table, (n, None), device)
    _ints("cu_seqlens", cu_seqlens, (n + 1,), device)
    c = MsaPagedCache(k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                      kv_lens.data_ptr(), cu_seqlens.data_ptr(), n_pages, page_table.shape[1])
    return c, n, hkv, page, d


def paged_workspace(q, k_pages, kv_lens):
    """A workspace for paged_attn_fwd and paged_append (it depends on the head shape alone, so
    one serves every step; calls that overlap on the GPU need one each)."""
    if not q.is_cuda or q.dtype not in _DT:
        _fail("q must be a float32 or bfloat16 CUDA tensor")
    T, hq, d = q.shape
    _, hkv, page, _ = k_pages.shape
    p = MsaParams(kv_lens.numel(), T, hq, hkv, d, page, 1, 1.0, _DT[q.dtype])
    return _workspace(p, _lib.OP_PAGED_ATTN, q.device)


def paged_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens, q=None, base=None,
                 wq=None, wk=None, eps=None, ws=None, out=None):
    """Appends packed new tokens k, v [T, hkv, d] to the paged cache k_pages, v_pages
    [n_pages, hkv, page, d], in place: sequence s's new tokens cu_seqlens[s]..cu_seqlens[s+1]
    become its last ones, positions kv_lens[s] - n_s .. kv_lens[s] - 1 (kv_lens counts them),
    in the pages of page_table[s].  With `base`, keys (and q [T, hq, d], when given) are
    rotated to their positions; with `eps`, their heads are normalised first (weights wq, wk
    or None for ones).  Returns the new queries [T, hq, d], or None without q.  Tokens without
    a page are skipped and reported in ws, if given (read_device_error)."""
    if not k.is_cuda or k.dtype not in _DT:
        _fail("k must be a float32 or bfloat16 CUDA tensor")
    dt, dev = k.dtype, k.device
    c, n, hkv, page, d = _cache(k_pages, v_pages, page_table, kv_lens, cu_seqlens, dt, dev)
    ks, vs = _rows("k", k, d, dt, dev), _rows("v", v, d, dt, dev)
    T = k.shape[0]
    if k.shape[1] != hkv or v.shape != k.shape:
        _fail("k and v must be [tokens, hkv, d] with the cache's hkv and d")
    hq, qs, qp, op, qo = hkv, 0, None, None, None
    if q is not None:
        qs = _rows("q", q, d, dt, dev)
        if q.shape[0] != T:
            _fail("q, k and v must hold the same tokens")
        hq = q.shape[1]
        qo = _out("out", out, (T, hq, d), dt, dev)
        qp, op = q.data_ptr(), qo.data_ptr()
    elif out is not None or wq is not None:
        _fail("out and wq are for a call with q")
    if eps is None and (wq is not None or wk is not None):
        _fail("wq and wk need eps")
    if eps is not None and not eps > 0:
        _fail("eps must be positive (None: no norm)")
    if base is not None and not base > 1:
        _fail("base must be above 1 (None: no rotation)")
    wp, wn = (None, 0) if ws is None else _ws_ptr(ws, dev)
    p = MsaParams(n, T, hq, hkv, d, page, 1, 1.0, _DT[dt])
    _call("msa_paged_append", dev, _byref(p), _byref(c), qp, qs, k.data_ptr(), ks, v.data_ptr(),
          vs, _weight("wq", wq, d, dt, dev), _weight("wk", wk, d, dt, dev), base or 0.0,
          eps or 0.0, op, wp, wn)
    return qo


def paged_attn_fwd(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, max_new=None,
                   scale=None, want_lse=True, ws=None, out=None):
    """Causal attention of packed new tokens q [T, hq, d] over the paged cache that already
    holds their keys and values (see paged_append).  max_new: the most new tokens of any
    sequence as the host knows it (None: unknown); it chooses the kernel, not the result's
    meaning.  Returns (o [T, hq, d], lse [T, hq] fp32 or None); a token that sees no key gets
    o = 0, lse = -inf; packed tokens behind the last sequence are left as they are (`out` may
    pass o and lse)."""
    if not q.is_cuda or q.dtype not in _DT or q.dim() != 3:
        _fail("q must be a float32 or bfloat16 CUDA tensor [tokens, hq, d]")
    dt, dev = q.dtype, q.device
    c, n, hkv, page, d = _cache(k_pages, v_pages, page_table, kv_lens, cu_seqlens, dt, dev)
    qs = _rows("q", q, d, dt, dev)
    T, hq, _ = q.shape
    if max_new is not None and max_new < 1 and T:
        _fail("max_new must be positive (None: unknown)")
    o = _out("o", None if out is None else out[0], (T, hq, d), dt, dev)
    lse = None
    if want_lse and (out is None or out[1] is not None):
        lse = _out("lse", None if out is None else out[1], (T, hq), torch.float32, dev)
    p = MsaParams(n, T, hq, hkv, d, page, 1, d ** -0.5 if scale is None else scale, _DT[dt])
    if ws is None:
        ws = _workspace(p, _lib.OP_PAGED_ATTN, dev)
    wp, wn = _ws_ptr(ws, dev)
    _call("msa_paged_attn_fwd", dev, _byref(p), _byref(c), max_new or 0, q.data_ptr(), qs,
          o.data_ptr(), None if lse is None else lse.data_ptr(), wp, wn)
    return o, lse
