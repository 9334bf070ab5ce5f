"""Paths of the layer operators that tests/test_gpu_layer.py does not tell apart or does not
reach: what the weights of each attention kernel carry, head layouts that take the general norm
and append kernels, wide groups, outputs at odd addresses.  Bounds as derived there (U = 2^-24,
the half step of an fp32 value; HALF, that of an output's type)."""
import numpy as np
import pytest
import torch

import oracle
import test_gpu_layer as base
from test_gpu_layer import HALF, U, Step, _close, _np
from test_gpu_layer import msa  # noqa: F401  (fixture)

gpu = pytest.mark.gpu


# ------------------------------------------------------------------ the weights' precision

def _bf16(x):
    """float64 values rounded to bf16 (nearest, ties to even; by way of fp32)."""
    return torch.tensor(np.asarray(x)).float().bfloat16().double().numpy()


def _cancelling(hq, hkv, d, n_new, kv, seed):
    """One sequence whose outputs cancel: q, k in {-1, 0, 1}, so scores are whole numbers and exact
    in fp32, and v [kv, hkv, d] of bf16 values whose signs keep the running sum of weight * v of
    column c, for row c % rows of its KV head, near zero (weights in falling order)."""
    r = np.random.default_rng(seed)
    G = hq // hkv
    q = r.integers(-1, 2, (n_new, hq, d)).astype(np.float64)
    k = r.integers(-1, 2, (kv, hkv, d)).astype(np.float64)
    size = _bf16(r.uniform(1, 2, (kv, hkv, d)))
    v = size.copy()
    scale = 1.5 / np.sqrt(d)
    for g in range(hkv):
        for c in range(d):
            t, h = divmod(c % (n_new * G), G)
            see = kv - n_new + t + 1
            p = np.exp(scale * k[:see, g] @ q[t, g * G + h])
            total = 0.0
            for i in np.argsort(-p, kind="stable"):
                v[i, g, c] = -size[i, g, c] if total > 0 else size[i, g, c]
                total += p[i] * v[i, g, c]
    return q, k, v, scale


def _attention(q, k, v, scale, round_weights=None):
    """(o, sum of weight * |v|, targeted) in float64; round_weights: what is planted between the
    softmax and the product with v (weights relative to the row's largest)."""
    n, hq, d = q.shape
    kv, hkv = k.shape[:2]
    G = hq // hkv
    o, a = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    target = np.zeros((n, hq, d), bool)
    for t in range(n):
        see = kv - n + t + 1
        for h in range(hq):
            x = scale * (k[:see, h // G] @ q[t, h])
            p = np.exp(x - x.max())
            w = p if round_weights is None else round_weights(p)
            o[t, h] = w @ v[:see, h // G] / p.sum()
            a[t, h] = p @ np.abs(v[:see, h // G]) / p.sum()
            target[t, h] = np.arange(d) % (n * G) == t * G + h % G
    return o, a, target


CANCEL = [  # hq, hkv, d, new tokens, tokens: up to 16 rows a KV head
    (8, 2, 128, 1, 97), (8, 1, 64, 1, 33), (16, 1, 128, 1, 230), (8, 2, 128, 4, 65),
    (2, 2, 64, 1, 120),
]


def _score_error(q, k, scale):
    """The scores are exact; their scaling and the subtraction of the maximum are off by 2 U each."""
    k = np.repeat(k, q.shape[1] // k.shape[1], axis=1)
    return 4 * U * max(1.0, scale * np.abs(np.einsum("thd,khd->tkh", q, k)).max())


def _bound(ref, a, q, k, scale, weights):
    n_keys, e = k.shape[0], _score_error(q, k, scale)
    return 2.0 ** -8 * np.abs(ref) + a * (2 * e + 2.0 ** -19 + weights + 2 * n_keys * U)


@pytest.mark.parametrize("case", CANCEL, ids=range(len(CANCEL)))
def test_cancelling_values_tell_one_term_from_two(case):
    """On the CPU: weights of one bf16 term leave the two-term bound at most of the entries whose
    values cancel; weights of two terms (a rounding of at most 2^-17) stay within it."""
    hq, hkv, d, n, kv = case
    q, k, v, scale = _cancelling(*case, seed=5)
    ref, a, target = _attention(q, k, v, scale)
    bound = _bound(ref, a, q, k, scale, 2.0 ** -17)
    one, _, _ = _attention(q, k, v, scale, _bf16)
    two, _, _ = _attention(q, k, v, scale, lambda p: _bf16(p) + _bf16(p - _bf16(p)))
    assert (np.abs(one - ref) > bound)[target].mean() > 0.5
    assert (np.abs(two - ref) <= bound).all()


def _cancelling_step(case):
    hq, hkv, d, n, kv = case
    q, k, v, scale = _cancelling(*case, seed=5)
    st = Step(torch.bfloat16, d, hq, hkv, 32, [(n, kv)])
    st.q = torch.tensor(q, device="cuda").bfloat16()
    for pool, x in ((st.kp, k), (st.vp, v)):
        pages = torch.tensor(st.table[0], device="cuda").long()
        x = torch.tensor(x, device="cuda").bfloat16()
        for p in range(kv):
            pool[pages[p // 32], :, p % 32] = x[p]
    return st, q, k, v, scale


@gpu
@pytest.mark.parametrize("case", CANCEL, ids=range(len(CANCEL)))
def test_weights_of_few_rows_carry_two_terms(msa, case):  # noqa: F811
    """Up to 16 rows of a KV head: the weights meet V with 2^-17, not with a bf16's 2^-8."""
    hq, hkv, d, n, kv = case
    st, q, k, v, scale = _cancelling_step(case)
    ref, a, _ = _attention(q, k, v, scale)
    o, _ = st.attn(msa, scale=scale, max_new=n)
    _close(o, ref, _bound(ref, a, q, k, scale, 2.0 ** -17))


@gpu
@pytest.mark.parametrize("case", [(8, 1, 128, 40, 97), (16, 4, 64, 9, 230), (32, 1, 128, 1, 65)])
def test_weights_of_many_rows_are_rounded_once(msa, case):  # noqa: F811
    """Above 16 rows: weights of one bf16 term, 2^-8 of each, while the sum they are divided by,
    and lse, keep the unrounded ones."""
    hq, hkv, d, n, kv = case
    st, q, k, v, scale = _cancelling_step(case)
    ref, a, _ = _attention(q, k, v, scale)
    o, lse = st.attn(msa, scale=scale, max_new=n)
    _close(o, ref, _bound(ref, a, q, k, scale, 2.0 ** -8))
    rl = oracle.paged_attention(q, _np(st.kp), _np(st.vp), st.table, st.kv, st.cu, 32, scale)[1]
    _close(lse, rl, _score_error(q, k, scale) + 2.0 ** -20 + kv * U + 4 * U * np.abs(rl))


# ------------------------------------------------------------------ append without a rotation

@gpu
@pytest.mark.parametrize("dtype,hq,hkv", [
    (torch.bfloat16, 4, 2), (torch.bfloat16, 32, 8), (torch.float32, 2, 1), (torch.float32, 16, 4)])
@pytest.mark.parametrize("tokens", [5, 1300])
def test_append_without_rotation_keeps_elements_apart(msa, dtype, hq, hkv, tokens):  # noqa: F811
    """Neither norm nor rotation: a copy, infinities, NaN and zeros' signs included.  A norm alone: an
    infinite element makes the others of its row zero, and none of them NaN."""
    st = Step(dtype, 128, hq, hkv, 32, [(tokens, tokens)])
    for x in (st.q, st.k):
        x[1, :, 3], x[2, :, 70], x[3, :, 5] = float("inf"), -float("inf"), float("nan")
        x[4, :, :70] = -0.0
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32

    def rows(pool):
        pages = torch.tensor(st.table[0], device="cuda").long()
        return pool[pages[pages >= 0]].transpose(1, 2).reshape(-1, hkv, 128)[:tokens]

    q = msa.paged_append(st.k, st.v, st.kp, st.vp, *st.dev, q=st.q)
    for got, want in ((q, st.q), (rows(st.kp), st.k), (rows(st.vp), st.v)):
        nan = want.isnan()
        assert torch.equal(got.isnan(), nan)
        assert torch.equal(got.contiguous().view(bits)[~nan], want.contiguous().view(bits)[~nan])
    q = msa.paged_append(st.k, st.v, st.kp, st.vp, *st.dev, q=st.q, eps=1e-6)
    for got in (q, rows(st.kp)):
        for t, c in ((1, 3), (2, 70)):
            assert got[t, :, c].isnan().all()
            assert (got[t, :, :c] == 0).all() and (got[t, :, c + 1:] == 0).all()
        assert (got[4, :, :70] == 0).all() and got[4].isfinite().all()


# ------------------------------------------------------------------ the general kernels

# The norm and the append give tokens of few row groups (a group: 32 / (d sizeof / 32) heads) kernels
# of their own; these layouts have more than four groups of queries or more than two of keys.
GENERAL = [  # dtype, d, hq, hkv
    (torch.float32, 128, 32, 8), (torch.float32, 128, 6, 6), (torch.float32, 128, 16, 2),
    (torch.float32, 64, 32, 8), (torch.float32, 64, 17, 17), (torch.bfloat16, 64, 64, 8),
    (torch.bfloat16, 64, 24, 24), (torch.bfloat16, 64, 33, 11),
]


@gpu
@pytest.mark.parametrize("cu", [[0, 3, 3, 50], base.LONG], ids=["several_warps", "one_warp"])
@pytest.mark.parametrize("heads", GENERAL, ids=range(len(GENERAL)))
def test_norm_rope_general_kernel(msa, heads, cu):  # noqa: F811
    """Forward and gradient, a token's heads dealt to several warps or all one warp's."""
    base.test_norm_rope_vs_oracle(msa, (*heads, cu, 1e6, True, True))
    base.test_norm_rope_vs_oracle(msa, (*heads, cu, 1e4, False, False))
    base.test_norm_rope_bwd_vs_oracle(msa, (*heads, cu, 1e6, True, True), "same")
    base.test_norm_rope_bwd_vs_oracle(msa, (*heads, cu, 1e4, False, False), "f32")


@gpu
@pytest.mark.parametrize("seqs", ["chunks", "steps", "empties", "many"])
@pytest.mark.parametrize("heads", GENERAL, ids=range(len(GENERAL)))
def test_append_general_kernel(msa, monkeypatch, heads, seqs):  # noqa: F811
    monkeypatch.setitem(base.HEADS, "x", (*heads, 48))
    monkeypatch.setitem(base.SEQS, "many", [(700, 700), (600, 900), (1, 5)])
    base.test_paged_append_vs_oracle(msa, "x", seqs, 1e6, True, True, True)
    base.test_paged_append_vs_oracle(msa, "x", seqs, 1e4, False, False, True)


@gpu
@pytest.mark.parametrize("heads", GENERAL, ids=range(len(GENERAL)))
def test_append_general_kernel_of_many_tokens_is_that_of_a_few(msa, heads):  # noqa: F811
    base.test_append_of_many_tokens_is_that_of_a_few(msa, *heads, True)


# ------------------------------------------------------------------ wide groups, odd addresses

WIDE = {   # dtype, d, hq, hkv, page: up to 64 query heads of a KV head
    "bf16_g64": (torch.bfloat16, 128, 64, 1, 64),
    "bf16_g64_d64": (torch.bfloat16, 64, 128, 2, 16),
    "bf16_g17": (torch.bfloat16, 128, 34, 2, 48),
    "bf16_g33_d64": (torch.bfloat16, 64, 33, 1, 128),
    "bf16_g63": (torch.bfloat16, 128, 63, 1, 80),
    "f32_g64": (torch.float32, 128, 64, 1, 64),
    "f32_g33_d64": (torch.float32, 64, 33, 1, 32),
    "f32_g16": (torch.float32, 128, 16, 1, 16),
}


@gpu
@pytest.mark.parametrize("seqs", base.SEQS)
@pytest.mark.parametrize("heads", WIDE)
def test_paged_attn_wide_groups(msa, monkeypatch, heads, seqs):  # noqa: F811
    monkeypatch.setitem(base.HEADS, heads, WIDE[heads])
    base.test_paged_attn_vs_oracle(msa, heads, seqs)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,hint", [(64, None), (128, None), (128, 1), (64, 2)])
def test_paged_attn_output_at_any_16_bytes(msa, dtype, d, hint):  # noqa: F811
    """Outputs that start 16 bytes behind a 32-byte boundary: the same bits, nothing around them
    touched."""
    st = Step(dtype, d, 8, 2, 64, [(70, 150), (1, 40), (3, 9)])
    want, wl = st.attn(msa, max_new=hint)
    step, n = 16 // want.element_size(), want.numel()
    room = torch.full((n + 4 * step,), 7.0, dtype=dtype, device="cuda")
    lroom = torch.full((wl.numel() + 2,), 7.0, device="cuda")
    o, lse = room[step:step + n].view(want.shape), lroom[1:-1].view(wl.shape)
    assert o.data_ptr() % 32 == 16
    st.attn(msa, out=(o, lse), max_new=hint)
    assert torch.equal(o, want) and torch.equal(lse, wl)
    assert (room[:step] == 7).all() and (room[step + n:] == 7).all()
    assert lroom[0] == 7 and lroom[-1] == 7
    with pytest.raises(msa.MsaError):
        st.attn(msa, out=(room[1:1 + n].view(want.shape), lse), max_new=hint)
