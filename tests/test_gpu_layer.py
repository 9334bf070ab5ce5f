"""Per-head norms with the rotation and their gradient, the append to a paged cache and the
attention over it, on the GPU against the fp64 oracle (oracle/msa_layer.py).

Bounds (u = 2^-24, the fp32 half step; h = the output type's half step, 2^-8 for bf16):
* norm + rotation: one rounding h |ref| plus fp32 arithmetic.  The mean of squares is a chain of
  at most 16 fused additions and 4 shuffles (20 u, halved by the root), its root and the two
  products add 4 u, the cosine and sine are off by at most 5 u, the rotation's products by 3 u:
  under 32 u of the pair |n_i| + |n_{i+d/2}|.
* dx: the same, twice over (the rotation back, the mean of u x, the last products): under 64 u of
  r (pair of |u| + |x r| mean |u x r|).
* dw: every term is off by at most 32 u of its pair; a sum's chain holds the heads of a lane, its
  tokens, 5 shuffles, 8 warps, up to 19 CTAs a slice and 32 slices: under 96 u more.
* attention: scores are fp32 dot products of d terms (d u of sum |q k|; 2 u for the scaling), so
  a weight is off by e = 4 d u s relative, s the row's largest scale * sum |q k|, its
  exponential by 2^-20 and, where it is rounded to bf16 before the product with V, by 2^-8; the
  sums over n keys by n u.  o: h |ref| + a (2 e + 2^-19 + [bf16] 2^-8 + 2 n u), a = sum of
  weight * |v|.  lse: e + 2^-20 + n u + 4 u |lse|."""
import numpy as np
import pytest
import torch

import oracle
import msa_inputs as mi

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module")
def msa():
    import block_sparse_top_mean_b200 as m
    from block_sparse_top_mean_b200 import build
    build.build()
    return m


def _np(x):
    return x.double().cpu().numpy()


def _pair(x):
    x = np.abs(x)
    return x + np.roll(x, x.shape[-1] // 2, axis=-1)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _close(got, ref, bound):
    got = _np(got)
    assert got.shape == ref.shape and np.isfinite(got).all()
    bad = np.abs(got - ref) > bound + 1e-37
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - ref).max()))


def _qkv(T, hq, hkv, d, dtype, seed, fused=False):
    x = mi.normal((T, hq + 2 * hkv, d), seed, mi.STREAM_Q, "cuda", dtype)
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return parts if fused else tuple(t.contiguous() for t in parts)


def _weights(d, dtype, seed):
    w = 1 + 0.2 * mi.normal((2, d), seed, mi.STREAM_V, "cuda", torch.float32)
    return w[0].to(dtype), w[1].to(dtype)


# ------------------------------------------------------------------ norm + rotation

NORM = [  # dtype, d, hq, hkv, cu, base, fused, weighted
    (torch.bfloat16, 128, 32, 8, [0, 700, 700, 1500], 1e6, True, True),
    (torch.bfloat16, 128, 3, 1, [0, 1], 1e4, False, True),
    (torch.bfloat16, 64, 5, 5, [0, 2, 3, 77], 500.0, True, False),
    (torch.float32, 64, 4, 2, [0, 1, 2, 1029], 1e4, False, True),
    (torch.float32, 128, 7, 1, [0, 17, 300], 1e4, True, True),
    (torch.float32, 128, 1, 1, [0, 9, 100_033], 1e6, False, True),    # far positions
]


# tokens enough for a warp each: every head count's own path, up to and above 32 documents
LONG = [0, 1, 1, 2500, 4999, 5003]
MANY = [0, *range(3, 153, 3), 4801]
NORM += [
    (torch.bfloat16, 128, 4, 4, LONG, 1e6, True, True),
    (torch.bfloat16, 128, 8, 1, MANY, 1e6, False, True),
    (torch.bfloat16, 128, 8, 8, LONG, 1e4, True, True),
    (torch.bfloat16, 128, 16, 4, MANY, 1e4, True, True),
    (torch.bfloat16, 128, 12, 6, LONG, 1e4, False, False),
    (torch.bfloat16, 128, 20, 5, MANY, 1e6, True, True),
    (torch.bfloat16, 64, 8, 1, MANY, 1e6, True, True),
    (torch.bfloat16, 64, 24, 12, LONG, 1e6, True, True),
    (torch.float32, 64, 2, 2, LONG, 1e4, False, True),
    (torch.float32, 64, 3, 1, MANY, 1e4, True, True),
    (torch.float32, 128, 8, 4, LONG, 1e4, True, True),
    (torch.float32, 128, 2, 1, LONG, 1e4, True, True),
]


def _norm_inputs(case, seed):
    dtype, d, hq, hkv, cu, base, fused, weighted = case
    q, k, _ = _qkv(cu[-1], hq, hkv, d, dtype, seed, fused)
    wq, wk = _weights(d, dtype, seed) if weighted else (None, None)
    return q, k, wq, wk


@pytest.mark.parametrize("case", NORM, ids=range(len(NORM)))
def test_norm_rope_vs_oracle(msa, case):
    dtype, d, hq, hkv, cu, base, fused, weighted = case
    q, k, wq, wk = _norm_inputs(case, 3)
    qo, ko = msa.qk_norm_rope(q, k, _i32(cu), base, wq=wq, wk=wk, eps=1e-5)
    pos = oracle.doc_positions(cu)
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        assert y.dtype == dtype and y.is_contiguous()
        wn = None if w is None else _np(w)
        ref = oracle.norm_rope(_np(x), wn, pos, base, 1e-5)
        n = oracle.msa_layer.norm_heads(_np(x), wn, 1e-5)
        _close(y, ref, HALF[dtype] * np.abs(ref) + 32 * U * _pair(n))


@pytest.mark.parametrize("grad", ["same", "f32"])
@pytest.mark.parametrize("case", NORM, ids=range(len(NORM)))
def test_norm_rope_bwd_vs_oracle(msa, case, grad):
    dtype, d, hq, hkv, cu, base, fused, weighted = case
    if cu[-1] > 50000:
        cu = [0, 9, 1033]
        case = (dtype, d, hq, hkv, cu, base, fused, weighted)
    gt = torch.float32 if grad == "f32" else dtype
    q, k, wq, wk = _norm_inputs(case, 4)
    T = cu[-1]
    gq = mi.normal((T, hq, d), 5, mi.STREAM_K, "cuda", gt)
    gk = mi.normal((T, hkv, d), 6, mi.STREAM_K, "cuda", gt)
    args = (gq, gk, q, k, _i32(cu), base)
    out = msa.qk_norm_rope_bwd(*args, wq=wq, wk=wk, eps=1e-5)
    pos = oracle.doc_positions(cu)
    for x, w, g, dx, dw in ((q, wq, gq, out[0], out[2]), (k, wk, gk, out[1], out[3])):
        assert dx.dtype == dtype and dw.dtype == torch.float32
        xn, gn = _np(x), _np(g)
        wn = np.ones(d) if w is None else _np(w)
        rx, rw = oracle.norm_rope_backward(gn, xn, wn, pos, base, 1e-5)
        r = 1 / np.sqrt((xn ** 2).mean(-1, keepdims=True) + 1e-5)
        pu = _pair(gn) * np.abs(wn)
        mag = r * (pu + np.abs(xn * r) * (pu * np.abs(xn * r)).mean(-1, keepdims=True))
        _close(dx, rx, HALF[dtype] * np.abs(rx) + 64 * U * mag)
        _close(dw, rw, 128 * U * (_pair(gn) * np.abs(xn * r)).sum((0, 1)))
    again = msa.qk_norm_rope_bwd(*args, wq=wq, wk=wk, eps=1e-5)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_norm_rope_bwd_against_differences(msa):
    """Directional differences of the forward kernel itself (fp32, step 2^-7: the truncation is
    of order step^2 = 6e-5 of the third derivative, the forward's rounding 32 u / step)."""
    case = (torch.float32, 64, 3, 1, [0, 5, 11], 100.0, False, True)
    q, k, wq, wk = _norm_inputs(case, 8)
    cu, step = _i32(case[4]), 2.0 ** -7
    gq, gk = (mi.normal(x.shape, 9 + i, mi.STREAM_K, "cuda", torch.float32)
              for i, x in enumerate((q, k)))
    dq, dk, dwq, dwk = msa.qk_norm_rope_bwd(gq, gk, q, k, cu, 100.0, wq=wq, wk=wk, eps=1e-3)

    def f(q, wq):
        return float((msa.qk_norm_rope(q, k, cu, 100.0, wq=wq, wk=wk, eps=1e-3)[0].double()
                      * gq.double()).sum())
    v = mi.normal(q.shape, 20, mi.STREAM_V, "cuda", torch.float32)
    v = v / v.norm()
    num = (f(q + step * v, wq) - f(q - step * v, wq)) / (2 * step)
    assert abs(num - float((dq.double() * v.double()).sum())) < 2e-2
    e = torch.zeros_like(wq)
    e[7] = 1.0
    num = (f(q, wq + step * e) - f(q, wq - step * e)) / (2 * step)
    assert abs(num - float(dwq[7])) < 2e-2


@pytest.mark.parametrize("heads", [(4, 4), (8, 4), (16, 8), (32, 8)])
def test_norm_rope_tokens_outside_documents_and_in_place(msa, heads):
    """Tokens before the first and behind the last document sit at position 0, in every path; in
    place as out of place."""
    T = 5000
    q, k, _ = _qkv(T, *heads, 128, torch.bfloat16, 9)
    cu = _i32([7, 2000, 4990])
    a = msa.qk_norm_rope(q, k, cu, 1e4)
    edge = torch.tensor([*range(7), *range(4990, T)], device="cuda")
    z = msa.qk_norm_rope(q[edge], k[edge], _i32(list(range(len(edge) + 1))), 1e4)
    assert torch.equal(a[0][edge], z[0]) and torch.equal(a[1][edge], z[1])
    mid = msa.qk_norm_rope(q[7:4990], k[7:4990], _i32([0, 1993, 4983]), 1e4)
    assert torch.equal(a[0][7:4990], mid[0]) and torch.equal(a[1][7:4990], mid[1])
    msa.qk_norm_rope(q, k, cu, 1e4, out=(q, k))
    assert torch.equal(q, a[0]) and torch.equal(k, a[1])


def test_norm_rope_edges(msa):
    """In place, no tokens, zero rows, tokens no document holds, another stream, repeats."""
    q, k, _ = _qkv(9, 4, 2, 64, torch.float32, 1)
    q[3] = 0
    cu = _i32([0, 4, 9])
    a = msa.qk_norm_rope(q, k, cu, 1e4)
    assert (a[0][3] == 0).all()
    q2, k2 = q.clone(), k.clone()
    b = msa.qk_norm_rope(q2, k2, cu, 1e4, out=(q2, k2))
    assert b[0] is q2 and torch.equal(a[0], q2) and torch.equal(a[1], k2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = msa.qk_norm_rope(q, k, cu, 1e4)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a[0], c[0])
    e = msa.qk_norm_rope(q[:0], k[:0], cu, 1e4)
    assert e[0].shape == (0, 4, 64)
    g = msa.qk_norm_rope_bwd(q[:0], k[:0], q[:0], k[:0], cu, 1e4)
    assert (g[2] == 0).all() and (g[3] == 0).all()
    # tokens behind the last document sit at position 0: the norm alone
    f = msa.qk_norm_rope(q, k, _i32([0, 4]), 1e4)
    z = msa.qk_norm_rope(q[4:], k[4:], _i32(list(range(6))), 1e4)
    assert torch.equal(f[0][4:], z[0])
    with pytest.raises(ValueError):
        msa.qk_norm_rope(q.transpose(0, 1), k, cu, 1e4)
    with pytest.raises(ValueError):
        msa.qk_norm_rope(q, k.bfloat16(), cu, 1e4)
    with pytest.raises(ValueError):
        msa.qk_norm_rope(q, k, cu.long(), 1e4)


# ------------------------------------------------------------------ paged cache

class Step:
    """A paged cache filled with seeded values (NaN in every slot no token holds) and the new
    tokens of one step: seqs = [(new, kv_len)]."""

    def __init__(self, dtype, d, hq, hkv, page, seqs, seed=1, pad=0, spare=2, fused=False):
        self.dtype, self.d, self.hq, self.hkv, self.page = dtype, d, hq, hkv, page
        self.new, self.kv = [a for a, _ in seqs], [b for _, b in seqs]
        self.cu = [0] + list(np.cumsum(self.new))
        need = [-(-b // page) for b in self.kv]
        total = sum(need) + 1
        order = np.random.default_rng(seed).permutation(total)
        self.table = np.full((len(seqs), max(need + [0]) + spare), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        shape = (total, hkv, page, d)
        self.kp = mi.normal(shape, seed, mi.STREAM_K, "cuda", dtype)
        self.vp = mi.normal(shape, seed, mi.STREAM_V, "cuda", dtype)
        held = np.zeros((total, page), bool)
        for s, L in enumerate(self.kv):
            for p in range(L):
                held[self.table[s, p // page], p % page] = True
        self.free = torch.tensor(~held, device="cuda")
        for pool in (self.kp, self.vp):
            pool.transpose(1, 2)[self.free] = float("nan")
        self.T = self.cu[-1] + pad
        self.q, self.k, self.v = _qkv(self.T, hq, hkv, d, dtype, seed + 7, fused)
        self.q = self.q * 2
        self.dev = (_i32(self.table), _i32(self.kv), _i32(self.cu))

    def attn(self, msa, **kw):
        return msa.paged_attn_fwd(self.q, self.kp, self.vp, *self.dev, **kw)

    def check(self, o, lse, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        n = self.cu[-1]
        ref, rl, a, s = oracle.paged_attention(
            _np(self.q), _np(self.kp), _np(self.vp), self.table, self.kv, self.cu, self.page, scale)
        e = 4 * self.d * U * np.abs(s[:n])
        keys = np.concatenate([np.zeros(0)] + [np.full(c, L) for c, L in zip(self.new, self.kv)])
        keys = np.maximum(keys, 0)[:, None]
        bf = self.dtype == torch.bfloat16
        b = HALF[self.dtype] * np.abs(ref[:n]) + a[:n] * (
            2 * e + 2.0 ** -19 + (2.0 ** -8 if bf else 0) + 2 * keys * U)[..., None]
        _close(o[:n], ref[:n], b)
        if lse is not None:
            seen = np.isfinite(rl[:n])
            got = _np(lse[:n])
            assert np.array_equal(np.isneginf(got), ~seen)
            bound = (e + 2.0 ** -20 + keys * U + 4 * U * np.abs(np.where(seen, rl[:n], 0)))[seen]
            assert (np.abs(got[seen] - rl[:n][seen]) <= bound).all()


SEQS = {
    "steps": [(1, 1), (1, 15), (1, 64), (1, 65), (1, 700)],
    "one_long_step": [(1, 5000)],
    "chunks": [(40, 40), (3, 200), (130, 131), (1, 333), (65, 900)],
    "empties": [(0, 0), (2, 2), (0, 77), (5, 3), (1, 1), (0, 0)],      # 5 new, 3 in the cache
    "prompt": [(300, 300)],
    "long_chunk": [(257, 1500)],
    "mixed": [(1, 300), (1, 17), (150, 800), (1, 1), (0, 40), (2, 90), (3, 3)],
    "verify": [(4, 260), (4, 9), (4, 64)],
}
HEADS = {   # dtype, d, hq, hkv, page
    "bf16_g4": (torch.bfloat16, 128, 8, 2, 64),
    "bf16_g8_p16": (torch.bfloat16, 128, 16, 2, 16),
    "bf16_g1_p256": (torch.bfloat16, 128, 2, 2, 256),
    "bf16_g3_p48": (torch.bfloat16, 128, 3, 1, 48),
    "bf16_g5_d64": (torch.bfloat16, 64, 10, 2, 32),
    "bf16_g16_d64_p128": (torch.bfloat16, 64, 16, 1, 128),
    "bf16_g24": (torch.bfloat16, 128, 24, 1, 80),
    "f32_g2_d64": (torch.float32, 64, 4, 2, 16),
    "f32_g4": (torch.float32, 128, 4, 1, 64),
    "f32_g7": (torch.float32, 128, 7, 1, 112),
}


@pytest.mark.parametrize("seqs", SEQS)
@pytest.mark.parametrize("heads", HEADS)
def test_paged_attn_vs_oracle(msa, heads, seqs):
    st = Step(*HEADS[heads], SEQS[seqs], pad=3)
    o = torch.full((st.T, st.hq, st.d), 7.0, dtype=st.dtype, device="cuda")
    lse = torch.full((st.T, st.hq), 7.0, device="cuda")
    ws = msa.paged_workspace(st.q, st.kp, st.dev[1])
    st.attn(msa, out=(o, lse), ws=ws, max_new=max(st.new))
    assert msa.read_device_error(ws) == 0
    st.check(o, lse)
    assert (o[st.cu[-1]:] == 7).all() and (lse[st.cu[-1]:] == 7).all()
    # the same call again, on a workspace of other content: the same bits
    ws[256:].fill_(0xFF)
    o2, lse2 = st.attn(msa, ws=ws, max_new=max(st.new))
    n = st.cu[-1]
    assert torch.equal(o[:n], o2[:n]) and torch.equal(lse[:n], lse2[:n])


@pytest.mark.parametrize("hint", [None, 1, 4, 10 ** 6])
def test_paged_attn_any_hint(msa, hint):
    """max_new chooses the kernel: every one of them is right for every length."""
    st = Step(torch.bfloat16, 128, 8, 2, 64, SEQS["chunks"] + SEQS["empties"])
    st.check(*st.attn(msa, max_new=hint))


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 1, 128), (24, 8, 64), (8, 8, 128)])
def test_paged_attn_chunk_among_single_tokens_of_large_caches(msa, hq, hkv, d):
    """Pools of more than 400 MB: single tokens and a chunk go to a launch each."""
    seqs = [(1, 70 * i + 1) for i in range(12)] + [(200, 900), (0, 5), (2, 300),
                                                   (17 // (hq // hkv), 65)]
    st = Step(torch.bfloat16, d, hq, hkv, 64, seqs, spare=4000)
    total = 400000000 // (4 * hkv * d * 64) + 2
    for name in ("kp", "vp"):
        big = torch.empty((total, hkv, 64, d), dtype=torch.bfloat16, device="cuda")
        big[:getattr(st, name).shape[0]] = getattr(st, name)
        setattr(st, name, big)
    o = torch.full((st.T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((st.T, hq), 7.0, device="cuda")
    st.attn(msa, out=(o, lse), max_new=200)
    st.check(o, lse)


def test_paged_attn_strided_queries_scale_and_no_lse(msa):
    st = Step(torch.bfloat16, 128, 8, 2, 32, [(70, 150), (1, 40)])
    wide = torch.empty(st.T, 20, 128, dtype=st.dtype, device="cuda")
    wide[:, 3:11] = st.q
    o, lse = msa.paged_attn_fwd(wide[:, 3:11], st.kp, st.vp, *st.dev, scale=0.05, want_lse=False)
    assert lse is None
    st.check(o, None, 0.05)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
def test_paged_attn_any_scale(msa, scale):
    for dtype in (torch.bfloat16, torch.float32):
        st = Step(dtype, 64, 4, 2, 32, [(70, 150), (1, 40)])
        st.check(*st.attn(msa, scale=scale), scale)


def test_paged_attn_shared_prefix_and_many_sequences(msa):
    """Sequences that share pages, and more sequences than a CTA has threads."""
    st = Step(torch.bfloat16, 128, 4, 1, 16, [(1, 40)] * 700)
    st.table[:, :2] = st.table[0, :2]
    st.dev = (_i32(st.table),) + st.dev[1:]
    st.check(*st.attn(msa, max_new=1))
    st.check(*st.attn(msa))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("new", [1, 100])
def test_paged_attn_bad_pages_are_reported(msa, dtype, new):
    """An entry that is no page reads as zeros and sets the error bit; a length beyond the table
    row ends at the row.  Other sequences are unharmed."""
    st = Step(dtype, 128, 4, 1, 16, [(new, 150), (new, 200), (new, 160)], spare=0)
    st.table[0, 3], st.table[2, 5] = 10 ** 6, -5
    st.kv[1] = 500                                     # the row holds 208 tokens
    st.vp.nan_to_num_(0.5)                             # the row's last slots are keys now
    st.kp.nan_to_num_(0.5)
    st.dev = (_i32(st.table), _i32(st.kv), st.dev[2])
    ws = msa.paged_workspace(st.q, st.kp, st.dev[1])
    st.check(*st.attn(msa, ws=ws, max_new=new))
    assert msa.read_device_error(ws) == msa.DEVERR_PAGE_RANGE


def test_paged_attn_large_scores_and_infinite_lse(msa):
    """Scores of some hundreds: the running maximum moves by more than any exponent range."""
    st = Step(torch.bfloat16, 128, 4, 1, 64, [(1, 700), (200, 700)])
    st.q = st.q * 20
    st.check(*st.attn(msa))
    st.check(*st.attn(msa, max_new=1))


@pytest.mark.parametrize("dtype,new,kv", [
    (torch.bfloat16, 2, 300), (torch.bfloat16, 1, 9000), (torch.bfloat16, 90, 700),
    (torch.float32, 2, 300), (torch.float32, 90, 700)])
def test_paged_attn_nan_query_stays_in_its_row(msa, dtype, new, kv):
    """A query head that is NaN has a NaN output and lse; every other row is as without it."""
    st = Step(dtype, 128, 4, 1, 64, [(new, kv)])
    o, lse = st.attn(msa)
    st.q[new // 2, 1] = float("nan")
    o2, lse2 = st.attn(msa)
    assert o2[new // 2, 1].isnan().all() and lse2[new // 2, 1].isnan()
    o2[new // 2, 1], lse2[new // 2, 1] = o[new // 2, 1], lse[new // 2, 1]
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


APPEND = [   # heads, seqs, base, norm, weighted, queries
    ("bf16_g4", "chunks", 1e6, True, True, True),
    ("bf16_g8_p16", "steps", 1e4, False, False, True),
    ("bf16_g5_d64", "chunks", None, True, True, True),
    ("f32_g2_d64", "chunks", 1e4, True, False, False),
    ("f32_g7", "steps", 1e6, True, True, True),
    ("bf16_g1_p256", "empties", 1e4, False, False, False),
]


@pytest.mark.parametrize("heads,seqs,base,norm,weighted,queries", APPEND)
def test_paged_append_vs_oracle(msa, heads, seqs, base, norm, weighted, queries):
    st = Step(*HEADS[heads], SEQS[seqs], pad=2, fused=True)
    st.kp.nan_to_num_(3.0)
    st.vp.nan_to_num_(3.0)
    eps = 1e-5 if norm else None
    wq, wk = _weights(st.d, st.dtype, 4) if weighted else (None, None)
    kp0, vp0 = _np(st.kp), _np(st.vp)
    q = st.q if queries else None
    ws = msa.paged_workspace(st.q, st.kp, st.dev[1])
    out = torch.full((st.T, st.hq, st.d), 7.0, dtype=st.dtype, device="cuda") if queries else None
    got = msa.paged_append(st.k, st.v, st.kp, st.vp, *st.dev, q=q, base=base, eps=eps,
                           wq=wq if queries else None, wk=wk, ws=ws, out=out)
    short = any(a > b for a, b in SEQS[seqs])          # tokens at negative positions
    assert msa.read_device_error(ws) == (msa.DEVERR_PAGE_RANGE if short else 0)
    kn, vn = _np(st.k), _np(st.v)
    wkn = None if wk is None else _np(wk)
    kp, vp = oracle.paged_append(kp0, vp0, kn, vn, st.table, st.kv, st.cu, st.page, base, wkn, eps)
    assert np.array_equal(_np(st.vp), vp)
    changed = (kp != kp0).any(-1, keepdims=True)
    h = HALF[st.dtype]
    mag = 2 * np.abs(kp).max() + 2 * np.abs(kn).max()  # pair of |n|, bounded over the step
    _close(st.kp, kp, np.where(changed, h * np.abs(kp) + 32 * U * mag, 0.0))
    if not queries:
        assert got is None
        return
    assert got is out and (got[st.cu[-1]:] == 7).all()
    rows = oracle.paged_positions(st.kv, st.cu)
    pos = np.array([p for _, _, p in rows])
    qn = _np(st.q)[:st.cu[-1]]
    n = oracle.msa_layer.norm_heads(qn, None if wq is None else _np(wq), eps) if norm else qn
    ref = n if base is None else oracle.rotate_heads(n, pos, base)
    _close(got[:st.cu[-1]], ref, h * np.abs(ref) + 32 * U * _pair(n))


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype,d,hq,hkv", [
    (torch.bfloat16, 128, 4, 4), (torch.bfloat16, 128, 8, 2), (torch.bfloat16, 128, 8, 8),
    (torch.bfloat16, 128, 12, 3), (torch.bfloat16, 128, 16, 8), (torch.bfloat16, 128, 32, 8),
    (torch.bfloat16, 64, 8, 1), (torch.float32, 64, 4, 2), (torch.float32, 128, 8, 4),
    (torch.float32, 128, 0, 3)])
def test_append_of_many_tokens_is_that_of_a_few(msa, dtype, d, hq, hkv, norm):
    """A warp a token, or several: bitwise the same pages, queries and errors (40 sequences; one
    is shorter than its new tokens, one has an entry that is no page, three tokens belong to
    nobody)."""
    seqs = [(125, 125 + 31 * i % 200) for i in range(38)] + [(20, 5), (0, 9)]
    st = Step(dtype, d, max(hq, hkv), hkv, 32, seqs, pad=3, fused=True)
    st.table[7, 1] = -1
    st.dev = (_i32(st.table),) + st.dev[1:]
    pools = [x.nan_to_num_(3.0) for x in (st.kp, st.vp)]
    wq, wk = _weights(d, dtype, 4) if norm else (None, None)
    kw = dict(base=1e4 if norm else None, eps=1e-5 if norm else None, wk=wk)

    def append(a, b, kp, vp):
        x, y = st.cu[a], st.cu[b] + (3 if b == 40 else 0)
        ws = msa.paged_workspace(st.q, kp, st.dev[1])
        qs = dict(q=st.q[x:y], wq=wq, out=torch.full((y - x, st.hq, d), 7.0, dtype=dtype,
                                                     device="cuda")) if hq else {}
        out = msa.paged_append(st.k[x:y], st.v[x:y], kp, vp, st.dev[0][a:b].contiguous(),
                               st.dev[1][a:b].contiguous(), st.dev[2][a:b + 1] - x, ws=ws,
                               **kw, **qs)
        return out, msa.read_device_error(ws)

    one = [x.clone() for x in pools]
    out, err = append(0, 40, *one)
    parts = [append(a, a + 5, *pools) for a in range(0, 40, 5)]
    assert torch.equal(one[0], pools[0]) and torch.equal(one[1], pools[1])
    assert err == msa.DEVERR_PAGE_RANGE
    assert [e for _, e in parts] == [0, err, 0, 0, 0, 0, 0, err]
    if hq:
        assert torch.equal(out, torch.cat([o for o, _ in parts]))
        assert (out[-3:] == 7).all()


def test_append_and_norm_rope_agree(msa):
    """The append's keys and queries are bitwise qk_norm_rope's at the same positions."""
    st = Step(torch.bfloat16, 128, 8, 2, 32, [(90, 90), (33, 33)])
    wq, wk = _weights(128, st.dtype, 2)
    qo, ko = msa.qk_norm_rope(st.q, st.k, st.dev[2], 1e6, wq=wq, wk=wk, eps=1e-6)
    qa = msa.paged_append(st.k, st.v, st.kp, st.vp, *st.dev, q=st.q, base=1e6, wq=wq, wk=wk,
                          eps=1e-6)
    assert torch.equal(qa, qo)
    for s in range(2):
        pages = torch.tensor(st.table[s], device="cuda").long()
        rows = st.kp[pages].transpose(1, 2).reshape(-1, 2, 128)[:st.kv[s]]
        assert torch.equal(rows, ko[st.cu[s]:st.cu[s + 1]])


def _serve(msa, st, ws, max_new, wq, wk):
    """One step of a full-attention layer: append with norm and rotation, then attention."""
    q = msa.paged_append(st.k, st.v, st.kp, st.vp, *st.dev, q=st.q, base=1e6, wq=wq, wk=wk,
                         eps=1e-6, ws=ws)
    return msa.paged_attn_fwd(q, st.kp, st.vp, *st.dev, max_new=max_new, ws=ws)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_in_chunks_then_single_tokens(msa, dtype):
    """A prompt served in uneven chunks and then token by token attends as the whole sequence at
    once: norm + rotation by qk_norm_rope and fp64 dense causal attention."""
    d, hq, hkv, page, L = 128, 8, 2, 32, 211
    st = Step(dtype, d, hq, hkv, page, [(0, L)])
    qkv = _qkv(L, hq, hkv, d, dtype, 31)
    wq, wk = _weights(d, dtype, 3)
    qo, ko = msa.qk_norm_rope(qkv[0], qkv[1], _i32([0, L]), 1e6, wq=wq, wk=wk, eps=1e-6)
    ws = msa.paged_workspace(qkv[0], st.kp, st.dev[1])
    outs, at = [], 0
    for n in [100, 1, 64, 40, 1, 1, 1, 1, 1, 1]:
        st.q, st.k, st.v = (x[at:at + n] for x in qkv)
        st.dev = (st.dev[0], _i32([at + n]), _i32([0, n]))
        outs.append(_serve(msa, st, ws, n, wq, wk))
        at += n
    assert at == L and msa.read_device_error(ws) == 0
    st.q, st.new, st.kv, st.cu, st.T = qo, [L], [L], [0, L], L
    st.check(torch.cat([o for o, _ in outs]), torch.cat([x for _, x in outs]))
    rows = st.kp[torch.tensor(st.table[0, :7], device="cuda").long()].transpose(1, 2)
    assert torch.equal(rows.reshape(-1, hkv, d)[:L], ko)


def test_captured_step_replays_with_new_lengths(msa):
    """A captured step reads lengths, table and boundaries when it runs; two graphs share a
    workspace one after the other."""
    st = Step(torch.bfloat16, 128, 8, 2, 16, [(1, 100), (1, 31), (1, 250)])
    wq, wk = _weights(128, st.dtype, 3)
    st.kp.nan_to_num_(0.25)
    st.vp.nan_to_num_(0.25)
    ws = msa.paged_workspace(st.q, st.kp, st.dev[1])
    _serve(msa, st, ws, 1, wq, wk)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _serve(msa, st, ws, 1, wq, wk)
        graphs.append((g, out))
    for kv in ([100, 31, 250], [96, 16, 241], [3, 1, 200]):
        st.dev[1].copy_(_i32(kv))
        for g, _ in graphs:
            g.replay()
        eager = _serve(msa, st, ws, 1, wq, wk)
        for _, out in graphs:
            assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])


def test_calls_on_two_streams_with_a_workspace_each(msa):
    a = Step(torch.bfloat16, 128, 8, 2, 64, [(1, 3000)] * 4, seed=1)
    b = Step(torch.bfloat16, 128, 8, 2, 64, [(300, 900)], seed=2)
    want = [a.attn(msa, max_new=1), b.attn(msa)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s, st, hint in zip(streams, (a, b), (1, None)):
            with torch.cuda.stream(s):
                got.append(st.attn(msa, max_new=hint))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_paged_nothing_to_do(msa):
    st = Step(torch.bfloat16, 64, 2, 1, 16, [(0, 5), (0, 0)])
    o, lse = st.attn(msa)
    assert o.shape == (0, 2, 64) and lse.shape == (0, 2)
    assert msa.paged_append(st.k, st.v, st.kp, st.vp, *st.dev) is None
    pad = Step(torch.bfloat16, 64, 2, 1, 16, [(0, 5), (0, 0)], pad=4)
    o = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 2), 7.0, device="cuda")
    pad.attn(msa, out=(o, lse))
    pad.attn(msa, out=(o, lse), max_new=1)
    assert (o == 7).all() and (lse == 7).all()
    with pytest.raises(ValueError):
        st.attn(msa, ws=torch.empty(4, device="cuda"))
    with pytest.raises(msa.MsaError):
        pad.attn(msa, ws=torch.empty(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        pad.attn(msa, max_new=0)


@pytest.mark.parametrize("dtype,new", [(torch.bfloat16, 1), (torch.bfloat16, 40),
                                       (torch.float32, 1), (torch.float32, 40)])
def test_pools_beyond_32_bits(msa, dtype, new):
    """Pages whose elements lie beyond 2^32 (and bytes beyond 2^33) from the pool's start."""
    st = Step(dtype, 128, 4, 2, 64, [(new, 200), (new, 64)], spare=0)
    kp, vp, n = st.kp, st.vp, st.kp.shape[0]
    total = 2 ** 32 // kp[0].numel() + 2 * n
    st.kp, st.vp = (torch.empty((total, *kp.shape[1:]), dtype=dtype, device="cuda")
                    for _ in "kv")
    st.kp[total - n:], st.vp[total - n:] = kp, vp
    st.table[st.table >= 0] += total - n
    st.dev = (_i32(st.table),) + st.dev[1:]
    ws = msa.paged_workspace(st.q, st.kp, st.dev[1])
    msa.paged_append(st.k, st.v, st.kp, st.vp, *st.dev, ws=ws)
    o, lse = st.attn(msa, max_new=new, ws=ws)
    assert msa.read_device_error(ws) == 0
    for s, at in ((0, 200), (1, 64)):
        page, row = st.table[s, (at - 1) // 64], (at - 1) % 64
        assert torch.equal(st.vp[page, :, row], st.v[st.cu[s + 1] - 1])
    st.kp, st.vp = st.kp[total - n:].clone(), st.vp[total - n:].clone()
    st.table[st.table >= 0] -= total - n
    st.check(o, lse)


@pytest.mark.parametrize("new,hq", [(1, 32), (2, 64), (5, 32)])
def test_paged_attn_long_caches_many_rounds(msa, new, hq):
    """Rings that go round hundreds of times, with copies that arrive late and out of order (a
    pool of 1.2 GB in shuffled small pages): every row against float64 on the GPU, five times."""
    n, hkv, page, d, L = 40, 8, 16, 128, 7000
    G, need = hq // hkv, -(-L // page)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    kp, vp = (torch.randn(n * need, hkv, page, d, generator=g, device="cuda",
                          dtype=torch.bfloat16) for _ in range(2))
    table = torch.randperm(n * need, generator=g, device="cuda").int().view(n, need)
    lens = torch.randint(L - 500, L + 1, (n,), generator=g, device="cuda").int()
    cu = torch.arange(0, (n + 1) * new, new, device="cuda").int()
    q = (2 * torch.randn(n * new, hq, d, generator=g, device="cuda")).bfloat16()
    ws = msa.paged_workspace(q, kp, lens)
    o, lse = msa.paged_attn_fwd(q, kp, vp, table, lens, cu, max_new=new, ws=ws)
    for _ in range(5):
        o2, lse2 = msa.paged_attn_fwd(q, kp, vp, table, lens, cu, max_new=new, ws=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert msa.read_device_error(ws) == 0
    for s in range(n):
        c = int(lens[s])
        K, V = (x[table[s].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :c].double()
                for x in (kp, vp))
        qs = q[s * new:(s + 1) * new].view(new, hkv, G, d).permute(1, 0, 2, 3).double()
        x = (qs.reshape(hkv, new * G, d) @ K.transpose(1, 2)).view(hkv, new, G, c) * d ** -0.5
        pos = torch.arange(c - new, c, device="cuda")
        x.masked_fill_((torch.arange(c, device="cuda")[None] > pos[:, None])[None, :, None],
                       -float("inf"))
        z = x.logsumexp(-1)
        p = torch.exp(x - z[..., None]).reshape(hkv, new * G, c)
        ref, a = (p @ V).view(hkv, new, G, d), (p @ V.abs()).view(hkv, new, G, d)
        big = (qs.abs().reshape(hkv, new * G, d) @ K.abs().transpose(1, 2)).amax(-1)
        e = 4 * d * U * float(big.max()) * d ** -0.5
        got = o[s * new:(s + 1) * new].view(new, hkv, G, d).permute(1, 0, 2, 3).double()
        bound = 2.0 ** -8 * ref.abs() + a * (2 * e + 2.0 ** -19 + 2.0 ** -8 + 2 * c * U)
        assert ((got - ref).abs() <= bound).all()
        gl = lse[s * new:(s + 1) * new].view(new, hkv, G).permute(1, 0, 2).double()
        assert ((gl - z).abs() <= e + 2.0 ** -20 + c * U + 4 * U * z.abs()).all()
