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
import struct

import torch

from . import _lib
from ._lib import MSA_BF16, MSA_F32, MsaError, MsaParams

_DT = {torch.float32: MSA_F32, torch.bfloat16: MSA_BF16}
_I32, _F32 = torch.int32, torch.float32
_MIN_EPS = 2.0 ** -126             # the smallest normal fp32 number
_fns = {}
# The images of msa_params and msa_paged_cache, passed by address: packing one takes a quarter of
# the time of a ctypes structure (0.12 us, 0.56).
_params = struct.Struct("@7qfi").pack
_cache_image = struct.Struct("@5P2q").pack


def _fail(text):
    raise ValueError(text)


def _call(name, index, *args):
    """The library's entry on the current stream of device `index` (launches need that device to
    be current).  These calls often take less time on the GPU than on the host, so the host
    side looks names up once and asks for the raw stream handle (a torch.cuda.Stream object
    costs 2 us)."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_lib.load(), name)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != 0:
        _lib.check(name, st)


def _device(name, x):
    """Index of x's CUDA device; x must be float32 or bfloat16."""
    index = x.get_device()
    if index < 0:
        _fail(f"{name}: block_sparse_top_mean_b200 takes CUDA tensors only")
    if x.dtype not in _DT:
        _fail(f"{name} must be float32 or bfloat16")
    return index


def _rows(name, x, T, d, dtype, index):
    """Checks x [T, heads, d] with packed heads and returns its token stride."""
    if x.dtype is not dtype or x.get_device() != index:
        _fail(f"{name} must be {dtype} on cuda:{index}")
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[2] != d or shape[0] != T:
        _fail(f"{name} must be [{T}, heads, {d}]")
    if stride[2] != 1 or stride[1] != d:
        if x.numel() and (stride[2] != 1 or shape[1] > 1):
            _fail(f"{name}: the heads of a token must be packed (only the token stride is free)")
    if T > 1 and stride[0] == 0:                          # (0 stands for packed tokens below)
        _fail(f"{name}: tokens must not share their storage")
    return stride[0] if T > 1 else shape[1] * d


def _ints(name, x, index):
    """Pointer of a contiguous int32 tensor."""
    if x.dtype is not _I32 or x.get_device() != index or not x.is_contiguous():
        _fail(f"{name} must be a contiguous int32 tensor on cuda:{index}")
    return x.data_ptr()


def _weight(name, w, d, dtype, index):
    if w is None:
        return None
    if w.dtype is not dtype or w.get_device() != index or w.shape != (d,) or \
            not w.is_contiguous():
        _fail(f"{name} must be a contiguous [{d}] {dtype} tensor on cuda:{index}")
    return w.data_ptr()


def _packed(name, x, shape, dtype, index):
    if x.dtype is not dtype or x.get_device() != index or x.shape != shape or \
            not x.is_contiguous():
        _fail(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on cuda:{index}")
    return x


def _like(name, x, src, dtype, index):
    """x checked, or a new packed tensor of src's shape."""
    if x is not None:
        return _packed(name, x, src.shape, dtype, index)
    y = torch.empty_like(src)
    return y if y.is_contiguous() else torch.empty_like(src, memory_format=torch.contiguous_format)


def _workspace(p, op, device):
    n = _lib.load().msa_workspace_bytes(ctypes.byref(p), op, 0)
    if n == 0:
        raise MsaError("msa_workspace_bytes", _lib.MSA_ERR_INVALID_ARG, "invalid shapes")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def _ws_ptr(ws, index):
    if ws.dtype is not torch.uint8 or ws.get_device() != index or not ws.is_contiguous():
        _fail(f"ws must be a contiguous uint8 tensor on cuda:{index}")
    return ws.data_ptr(), ws.numel()


def _norm_args(q, k, cu_seqlens, wq, wk):
    index, dt = _device("q", q), q.dtype
    if q.dim() != 3 or k.dim() != 3:
        _fail("q and k must be [tokens, heads, d]")
    T, hq, d = q.shape
    qs, ks = _rows("q", q, T, d, dt, index), _rows("k", k, T, d, dt, index)
    if cu_seqlens.dim() != 1:
        _fail("cu_seqlens must have one dimension")
    cu = _ints("cu_seqlens", cu_seqlens, index)
    p = _params(1, T, hq, k.shape[1], d, 1, 1, 1.0, _DT[dt])
    return (p, index, dt, cu, cu_seqlens.shape[0] - 1, qs, ks, _weight("wq", wq, d, dt, index),
            _weight("wk", wk, d, dt, index))


def qk_norm_rope(q, k, cu_seqlens, base: float, wq=None, wk=None, eps: float = 1e-6, out=None):
    """RMS norm of every head of packed q [T, hq, d] and k [T, hkv, d] (weights wq, wk [d] or
    None for ones), then the rotation by each token's position in its own document
    (cu_seqlens: int32 CUDA tensor of the n_docs + 1 boundaries).  q and k may be strided in
    the token dimension (views of a fused projection).  Returns (q_out, k_out), packed; `out`
    may pass them, or q and k themselves when those are packed."""
    p, index, dt, cu, n, qs, ks, pq, pk = _norm_args(q, k, cu_seqlens, wq, wk)
    qo = _like("q_out", None if out is None else out[0], q, dt, index)
    ko = _like("k_out", None if out is None else out[1], k, dt, index)
    _call("msa_qk_norm_rope", index, p, cu, n, q.data_ptr(), qs, k.data_ptr(), ks, pq, pk,
          base, eps, qo.data_ptr(), ko.data_ptr())
    return qo, ko


def qk_norm_rope_workspace(q, k):
    """A workspace for qk_norm_rope_bwd (it depends on the head shape alone)."""
    _device("q", q)
    T, hq, d = q.shape
    return _workspace(MsaParams(1, T, hq, k.shape[1], d, 1, 1, 1.0, _DT[q.dtype]),
                      _lib.OP_QK_NORM_ROPE_BWD, q.device)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, cu_seqlens, base: float, wq=None, wk=None,
                     eps: float = 1e-6, ws=None, out=None):
    """Gradient of qk_norm_rope for the upstream gradients dq_out, dk_out (packed; fp32 or the
    inputs' dtype): (dq, dk, dwq, dwk), dq and dk in the inputs' dtype, the weights' gradients
    in fp32.  `out` may pass the four tensors."""
    p, index, dt, cu, n, qs, ks, pq, pk = _norm_args(q, k, cu_seqlens, wq, wk)
    gt = dq_out.dtype
    if gt is not dt and gt is not _F32:
        _fail(f"the upstream gradients must be float32 or {dt}")
    _packed("dq_out", dq_out, q.shape, gt, index)
    _packed("dk_out", dk_out, k.shape, gt, index)
    o = (None,) * 4 if out is None else out
    dq, dk = _like("dq", o[0], q, dt, index), _like("dk", o[1], k, dt, index)
    if out is None:
        d = q.shape[2]
        dwq, dwk = q.new_empty(d, dtype=_F32), q.new_empty(d, dtype=_F32)
    else:
        dwq, dwk = (_packed(name, x, q.shape[2:], _F32, index) for name, x in
                    (("dwq", o[2]), ("dwk", o[3])))
    if ws is None:
        ws = qk_norm_rope_workspace(q, k)
    wp, wn = _ws_ptr(ws, index)
    _call("msa_qk_norm_rope_bwd", index, p, cu, n, dq_out.data_ptr(), dk_out.data_ptr(),
          _DT[gt], q.data_ptr(), qs, k.data_ptr(), ks, pq, pk, base, eps, dq.data_ptr(),
          dk.data_ptr(), dwq.data_ptr(), dwk.data_ptr(), wp, wn)
    return dq, dk, dwq, dwk


def _cache(k_pages, v_pages, page_table, kv_lens, cu_seqlens, dtype, index):
    """The checked cache of a step and its shape (n_seqs, hkv, page, d)."""
    shape = k_pages.shape
    if len(shape) != 4 or shape != v_pages.shape:
        _fail("k_pages and v_pages must both be [n_pages, hkv, page, d]")
    for x in (k_pages, v_pages):
        if x.dtype is not dtype or x.get_device() != index or not x.is_contiguous():
            _fail(f"k_pages and v_pages must be contiguous {dtype} tensors on cuda:{index}")
    n, table = kv_lens.numel(), page_table.shape
    if kv_lens.dim() != 1 or len(table) != 2 or table[0] != n or cu_seqlens.shape != (n + 1,):
        _fail("kv_lens, page_table and cu_seqlens must be [n_seqs], [n_seqs, max_pages] and "
              "[n_seqs + 1]")
    c = _cache_image(k_pages.data_ptr(), v_pages.data_ptr(),
                     _ints("page_table", page_table, index), _ints("kv_lens", kv_lens, index),
                     _ints("cu_seqlens", cu_seqlens, index), shape[0], table[1])
    return c, n, shape[1], shape[2], shape[3]


def paged_workspace(q, k_pages, kv_lens):
    """A workspace for paged_attn_fwd and paged_append (it depends on the head shape alone, so
    one serves every step; calls that overlap on the GPU need one each)."""
    _device("q", q)
    T, hq, d = q.shape
    _, hkv, page, _ = k_pages.shape
    p = MsaParams(kv_lens.numel(), T, hq, hkv, d, page, 1, 1.0, _DT[q.dtype])
    return _workspace(p, _lib.OP_PAGED_ATTN, q.device)


def _append_eps(eps, wq, wk):
    """The C entry's eps: 0 stands for no norm there, so none may round to it."""
    if eps is None:
        if wq is not None or wk is not None:
            _fail("wq and wk need eps")
        return 0.0
    if not eps >= _MIN_EPS:
        _fail("eps must be positive, 2^-126 at least (None: no norm)")
    return eps


def paged_append(k, v, k_pages, v_pages, page_table, kv_lens, cu_seqlens, q=None, base=None,
                 wq=None, wk=None, eps=None, ws=None, out=None):
    """Appends packed new tokens k, v [T, hkv, d] to the paged cache k_pages, v_pages
    [n_pages, hkv, page, d], in place: sequence s's new tokens cu_seqlens[s]..cu_seqlens[s+1]
    become its last ones, positions kv_lens[s] - n_s .. kv_lens[s] - 1 (kv_lens counts them),
    in the pages of page_table[s].  With `base`, keys (and q [T, hq, d], when given) are
    rotated to their positions; with `eps`, their heads are normalised first (weights wq, wk
    or None for ones).  Returns the new queries [T, hq, d], or None without q.  Tokens without
    a page are skipped and reported in ws, if given (read_device_error)."""
    index, dt = _device("k", k), k.dtype
    c, n, hkv, page, d = _cache(k_pages, v_pages, page_table, kv_lens, cu_seqlens, dt, index)
    T = k.shape[0]
    ks, vs = _rows("k", k, T, d, dt, index), _rows("v", v, T, d, dt, index)
    if k.shape[1] != hkv or v.shape[1] != hkv:
        _fail("k and v must be [tokens, hkv, d] with the cache's hkv and d")
    hq, qs, qp, op, qo = hkv, 0, None, None, None
    if q is not None:
        qs = _rows("q", q, T, d, dt, index)
        hq = q.shape[1]
        qo = _like("out", out, q, dt, index)
        qp, op = q.data_ptr(), qo.data_ptr()
    elif out is not None or wq is not None:
        _fail("out and wq are for a call with q")
    eps = _append_eps(eps, wq, wk)
    if base is None:
        base = 0.0
    elif not base > 1:
        _fail("base must be above 1 (None: no rotation)")
    wp, wn = (None, 0) if ws is None else _ws_ptr(ws, index)
    p = _params(n, T, hq, hkv, d, page, 1, 1.0, _DT[dt])
    _call("msa_paged_append", index, p, c, qp, qs, k.data_ptr(), ks, v.data_ptr(),
          vs, _weight("wq", wq, d, dt, index), _weight("wk", wk, d, dt, index), base, eps, op, wp,
          wn)
    return qo


def paged_attn_fwd(q, k_pages, v_pages, page_table, kv_lens, cu_seqlens, max_new=None,
                   scale=None, want_lse=True, ws=None, out=None):
    """Causal attention of packed new tokens q [T, hq, d] over the paged cache that already
    holds their keys and values (see paged_append).  max_new: the most new tokens of any
    sequence as the host knows it (None: unknown); it chooses the kernel, not the result's
    meaning, and with it how bf16 calls round the softmax's weights before the product with the
    values: to 2^-17 of each where max_new * hq / hkv <= 16, to 2^-8 above.  Returns
    (o [T, hq, d], lse [T, hq] fp32 or None); a token that sees no key gets o = 0, lse = -inf;
    packed tokens behind the last sequence are left as they are (`out` may pass o and lse).

    What goes wrong on the device is reported in ws (read_device_error): DEVERR_PAGE_RANGE for a
    table entry that is no page (its keys and values count as zeros), DEVERR_TIMEOUT for a wait
    that ran out (results are then incomplete).  Without ws the call makes itself a workspace
    (43 MB at d = 128) that ends with it, and nothing reports either.

    Pass max_new where all sequences have few new tokens: a batch of single tokens whose hint
    is left out counts as one that may hold a chunk (48 sequences of up to 16384 keys 71 us,
    49 with it; 64 of 512 44 and 32; 32 / 8 heads of 128)."""
    index, dt = _device("q", q), q.dtype
    c, n, hkv, page, d = _cache(k_pages, v_pages, page_table, kv_lens, cu_seqlens, dt, index)
    if q.dim() != 3:
        _fail("q must be [tokens, hq, d]")
    T, hq, _ = q.shape
    qs = _rows("q", q, T, d, dt, index)
    if max_new is None:
        max_new = 0
    elif max_new < 1 and T:
        _fail("max_new must be positive (None: unknown)")
    o = _like("o", None if out is None else out[0], q, dt, index)
    lse = lp = None
    if want_lse:
        if out is None:
            lse = q.new_empty(T, hq, dtype=_F32)
            lp = lse.data_ptr()
        elif out[1] is not None:
            lse = _packed("lse", out[1], (T, hq), _F32, index)
            lp = lse.data_ptr()
    p = _params(n, T, hq, hkv, d, page, 1, d ** -0.5 if scale is None else scale, _DT[dt])
    if ws is None:
        ws = paged_workspace(q, k_pages, kv_lens)
    wp, wn = _ws_ptr(ws, index)
    _call("msa_paged_attn_fwd", index, p, c, max_new, q.data_ptr(), qs,
          o.data_ptr(), lp, wp, wn)
    return o, lse
