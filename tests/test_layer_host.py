"""Refusals of the layer operators on the host: the C entries check every argument before any
CUDA call (these calls need no GPU), and the binding names what is wrong with a tensor."""
import ctypes

import pytest
import torch

from block_sparse_top_mean_b200 import _lib
from block_sparse_top_mean_b200._lib import MsaPagedCache, MsaParams

INVALID, UNSUPPORTED, WORKSPACE, OK = (_lib.MSA_ERR_INVALID_ARG, _lib.MSA_ERR_UNSUPPORTED,
                                       _lib.MSA_ERR_WORKSPACE, _lib.MSA_OK)
F = ctypes.c_void_p(4096)          # non-null, aligned; never dereferenced (checks fail first)
ODD = ctypes.c_void_p(4096 + 8)


@pytest.fixture(scope="module")
def lib():
    from block_sparse_top_mean_b200 import build
    build.build()
    return _lib.load()


def _p(**kw):
    base = dict(batch=1, seq=100, hq=32, hkv=8, d=128, block=64, topk=1, scale=0.088,
                dtype=_lib.MSA_BF16)
    base.update(kw)
    return ctypes.byref(MsaParams(*[base[k] for k in ["batch", "seq", "hq", "hkv", "d", "block",
                                                      "topk", "scale", "dtype"]]))


SHAPES = [(dict(hq=30), INVALID), (dict(seq=-1), INVALID), (dict(dtype=5), INVALID),
          (dict(d=96), UNSUPPORTED), (dict(hq=8 * 65), UNSUPPORTED),
          (dict(seq=1 << 32), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", SHAPES)
def test_shapes_refused_by_every_entry(lib, kw, code):
    p = _p(**kw)
    c = ctypes.byref(MsaPagedCache(4096, 4096, 4096, 4096, 4096, 10, 10))
    assert lib.msa_qk_norm_rope(p, F, 1, F, 0, F, 0, F, F, 1e4, 1e-6, F, F, None) == code
    assert lib.msa_qk_norm_rope_bwd(p, F, 1, F, F, 0, F, 0, F, 0, F, F, 1e4, 1e-6, F, F, None,
                                    None, None, 0, None) == code
    assert lib.msa_paged_append(p, c, F, 0, F, 0, F, 0, None, None, 0.0, 0.0, F, None, 0,
                                None) == code
    assert lib.msa_paged_attn_fwd(p, c, 0, F, 0, F, None, F, 1 << 40, None) == code


def test_null_params_and_workspace_sizes(lib):
    assert lib.msa_qk_norm_rope(None, F, 1, F, 0, F, 0, F, F, 1e4, 1e-6, F, F, None) == INVALID
    for op in (_lib.OP_QK_NORM_ROPE_BWD, _lib.OP_PAGED_APPEND, _lib.OP_PAGED_ATTN):
        assert lib.msa_workspace_bytes(_p(), op, 0) >= 256
        assert lib.msa_workspace_bytes(_p(d=96), op, 0) == 0
        assert lib.msa_workspace_bytes(None, op, 0) == 0
    # one workspace serves the append and the attention
    assert lib.msa_workspace_bytes(_p(), _lib.OP_PAGED_ATTN, 0) >= \
        lib.msa_workspace_bytes(_p(), _lib.OP_PAGED_APPEND, 0)
    # any group size up to 64 is in range
    for hq in (24, 40, 512):
        assert lib.msa_workspace_bytes(_p(hq=hq), _lib.OP_PAGED_ATTN, 0) > 256


def test_norm_rope_refusals(lib):
    good = dict(cu=F, n=1, q=F, qs=0, k=F, ks=0, wq=F, wk=F, base=1e4, eps=1e-6, qo=F, ko=F)

    def call(p=None, **kw):
        a = {**good, **kw}
        return lib.msa_qk_norm_rope(p or _p(), a["cu"], a["n"], a["q"], a["qs"], a["k"], a["ks"],
                                    a["wq"], a["wk"], a["base"], a["eps"], a["qo"], a["ko"], None)

    for kw in (dict(cu=None), dict(n=0), dict(q=None), dict(k=None), dict(q=ODD), dict(wk=ODD),
               dict(qo=None), dict(ko=ODD), dict(base=1.0), dict(base=float("inf")),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(qs=32 * 128 - 8),
               dict(qs=32 * 128 + 4), dict(ks=-8), dict(qo=F, q=F, qs=48 * 128)):
        assert call(**kw) == INVALID, kw
    assert call(n=1 << 31) == UNSUPPORTED
    assert call(p=_p(seq=0), cu=None, q=None, k=None, qo=None, ko=None) == OK
    assert call(p=_p(batch=0), cu=None, q=None, k=None, qo=None, ko=None) == OK


def test_norm_rope_bwd_refusals(lib):
    good = dict(gq=F, gk=F, gt=_lib.MSA_F32, q=F, k=F, dq=F, dk=F, dwq=F, dwk=F, ws=F)
    need = lib.msa_workspace_bytes(_p(), _lib.OP_QK_NORM_ROPE_BWD, 0)

    def call(n=need, p=None, **kw):
        a = {**good, **kw}
        return lib.msa_qk_norm_rope_bwd(p or _p(), F, 1, a["gq"], a["gk"], a["gt"], a["q"], 0,
                                        a["k"], 0, None, None, 1e4, 1e-6, a["dq"], a["dk"],
                                        a["dwq"], a["dwk"], a["ws"], n, None)

    for kw in (dict(gq=None), dict(gk=ODD), dict(gt=7), dict(q=None), dict(dq=None),
               dict(dk=ODD)):
        assert call(**kw) == INVALID, kw
    # fp32 tensors take fp32 gradients alone
    assert call(p=_p(dtype=_lib.MSA_F32), gt=_lib.MSA_BF16) == INVALID
    for kw in (dict(n=need - 1), dict(ws=None), dict(ws=ctypes.c_void_p(4096 + 16))):
        assert call(**kw) == WORKSPACE, kw


def _cache(**kw):
    base = dict(k=4096, v=4096, table=4096, lens=4096, cu=4096, n=10, m=10)
    base.update(kw)
    return ctypes.byref(MsaPagedCache(*[base[k] for k in ["k", "v", "table", "lens", "cu", "n",
                                                          "m"]]))


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=4096 + 8), INVALID), (dict(table=None), INVALID),
              (dict(lens=None), INVALID), (dict(cu=4097), INVALID), (dict(n=-1), INVALID), (dict(n=0), INVALID),
              (dict(m=-1), INVALID), (dict(n=1 << 40), UNSUPPORTED), (dict(m=1 << 40), UNSUPPORTED),
              (dict(m=(2 ** 31 - 1) // 64), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_CACHES)
def test_caches_refused(lib, kw, code):
    c = _cache(**kw)
    assert lib.msa_paged_append(_p(), c, F, 0, F, 0, F, 0, None, None, 0.0, 0.0, F, None, 0,
                                None) == code
    assert lib.msa_paged_attn_fwd(_p(), c, 0, F, 0, F, None, F, 1 << 40, None) == code


def test_paged_refusals(lib):
    c = _cache()
    for block, code in ((0, INVALID), (8, UNSUPPORTED), (24, UNSUPPORTED), (1 << 21, UNSUPPORTED)):
        assert lib.msa_paged_attn_fwd(_p(block=block), c, 0, F, 0, F, None, F, 1 << 40,
                                      None) == code
    good = dict(q=F, qs=0, k=F, ks=0, v=F, vs=0, wq=F, wk=F, base=1e4, eps=1e-6, qo=F, ws=F,
                n=256)

    def append(p=None, cache=c, **kw):
        a = {**good, **kw}
        return lib.msa_paged_append(p or _p(), cache, a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                    a["vs"], a["wq"], a["wk"], a["base"], a["eps"], a["qo"],
                                    a["ws"], a["n"], None)

    for kw in (dict(k=None), dict(v=None), dict(qo=None), dict(q=None), dict(k=ODD),
               dict(wq=ODD), dict(base=1.0), dict(base=-5.0), dict(eps=-1e-6), dict(eps=0.0),
               dict(ks=8), dict(vs=8 * 128 + 2), dict(q=F, qo=F, qs=48 * 128)):
        assert append(**kw) == INVALID, kw
    assert append(n=255) == WORKSPACE
    assert append(ws=ctypes.c_void_p(4096 + 16)) == WORKSPACE
    assert lib.msa_paged_append(None, c, F, 0, F, 0, F, 0, None, None, 0.0, 0.0, F, None, 0,
                                None) == INVALID
    assert append(cache=None) == INVALID
    # nothing to do: no pointer is looked at
    empty = _cache(k=None, v=None, table=None, lens=None, cu=None, n=0, m=0)
    none = dict(q=None, k=None, v=None, wq=None, wk=None, qo=None, eps=0.0, ws=None)
    assert append(p=_p(seq=0), cache=empty, **none) == OK
    assert append(p=_p(batch=0), cache=empty, **none) == OK
    need = lib.msa_workspace_bytes(_p(), _lib.OP_PAGED_ATTN, 0)
    att = lib.msa_paged_attn_fwd
    assert att(_p(), c, 0, None, 0, F, None, F, need, None) == INVALID
    assert att(_p(), c, 0, F, 0, None, None, F, need, None) == INVALID
    assert att(_p(), c, 0, F, 0, F, ctypes.c_void_p(4098), F, need, None) == INVALID
    assert att(_p(), c, -1, F, 0, F, None, F, need, None) == INVALID
    assert att(_p(), c, 0, F, 100, F, None, F, need, None) == INVALID
    for scale in (float("nan"), float("inf"), 3e38):      # 3e38 * log2(e) is no fp32 number
        assert att(_p(scale=scale), c, 0, F, 0, F, None, F, need, None) == INVALID
    assert att(_p(), c, 0, F, 0, F, None, F, need - 1, None) == WORKSPACE
    assert att(_p(), c, 0, F, 0, F, None, None, need, None) == WORKSPACE
    assert att(_p(seq=0), empty, 0, None, 0, None, None, None, 0, None) == OK


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import block_sparse_top_mean_b200 as msa
    q, k = torch.zeros(4, 2, 64), torch.zeros(4, 1, 64)
    cu = torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros(2, 1, 16, 64)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: msa.qk_norm_rope(q, k, cu, 1e4),
                 lambda: msa.qk_norm_rope_bwd(q, k, q, k, cu, 1e4),
                 lambda: msa.paged_append(k, k, pool, pool, table, lens, cu),
                 lambda: msa.paged_attn_fwd(q, pool, pool, table, lens, cu),
                 lambda: msa.paged_workspace(q, pool, lens)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_tokens_that_share_storage():
    """A token stride of 0 stands for packed tokens in the C entries: an expanded tensor, whose
    stride is 0, would be read past its end.  The check needs no GPU (device index -1)."""
    from block_sparse_top_mean_b200.layer import _rows
    one = torch.zeros(1, 2, 64)
    assert _rows("q", one, 1, 64, torch.float32, -1) == 128
    assert _rows("q", torch.zeros(4, 6, 64)[:, 2:4], 4, 64, torch.float32, -1) == 384
    with pytest.raises(ValueError, match="share"):
        _rows("q", one.expand(4, 2, 64), 4, 64, torch.float32, -1)
    with pytest.raises(ValueError, match="packed"):
        _rows("q", torch.zeros(4, 1, 64).expand(4, 2, 64), 4, 64, torch.float32, -1)
    with pytest.raises(ValueError, match="packed"):
        _rows("q", torch.zeros(4, 64, 2).transpose(1, 2), 4, 64, torch.float32, -1)


def test_packed_images_are_the_structures():
    """The binding passes msa_params and msa_paged_cache as packed bytes."""
    from block_sparse_top_mean_b200 import layer
    a = (3, 1 << 40, 32, 8, 128, 64, 1, 0.125, 1)
    assert layer._params(*a) == bytes(MsaParams(*a))
    c = (1 << 47, 2, 3, 4, 5, 1 << 33, 7)
    assert layer._cache_image(*c) == bytes(MsaPagedCache(*c))
