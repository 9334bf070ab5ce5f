"""Measured cases of the operators round a full-attention layer: the per-head norms of queries
and keys with the rotation (forward and backward), the append of new tokens to a paged
key/value cache, and the attention of new tokens over that cache.

`run` computes an operator in plain torch operations, or, where `own` is true, makes the
calls a user makes of this package.  Shapes (ragged lengths included) follow from the case
alone, values from the seed."""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-6


def _msa():
    import block_sparse_top_mean_b200 as msa
    return msa


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a training step's packed documents, a 128-wide head layout of 32 query / 8 KV heads
        dict(name="norm_rope_docs_32k", op="norm_rope", dtype="bf16", tokens=32768, docs=9,
             hq=32, hkv=8, d=128, base=1e6, fused=True, lens_seed=1),
        # one short fp32 document batch, odd token count, the small head layout
        dict(name="norm_rope_short_f32", op="norm_rope", dtype="fp32", tokens=1029, docs=4,
             hq=4, hkv=2, d=64, base=1e4, fused=False, lens_seed=2),
        # its backward: fp32 upstream gradients, as the sparse attention's backward writes them
        dict(name="norm_rope_bwd_32k", op="norm_rope_bwd", dtype="bf16", tokens=32768, docs=9,
             hq=32, hkv=8, d=128, base=1e6, grad="fp32", fused=True, lens_seed=1),
        # backward of a short batch in the tensors' own type
        dict(name="norm_rope_bwd_1k", op="norm_rope_bwd", dtype="bf16", tokens=1500, docs=3,
             hq=8, hkv=2, d=128, base=1e4, grad="bf16", fused=False, lens_seed=3),
        # one generated token for each of 64 running sequences
        dict(name="append_step_64", op="append", dtype="bf16", seqs=64, new=1, past=4096,
             hq=32, hkv=8, d=128, page=64, base=1e6, norm=True, lens_seed=4),
        # ragged prompt chunks of six requests
        dict(name="append_chunks_ragged", op="append", dtype="bf16", seqs=6, new=4096, past=8000,
             hq=32, hkv=8, d=128, page=16, base=1e6, norm=True, lens_seed=5),
        # fp32 small heads, no norm, no queries beyond the rotation
        dict(name="append_f32_small", op="append", dtype="fp32", seqs=3, new=77, past=500,
             hq=4, hkv=2, d=64, page=16, base=1e4, norm=False, lens_seed=6),
        # one generated token for each of 48 sequences of very different lengths
        dict(name="attn_step_48", op="attn", dtype="bf16", seqs=48, new=1, past=16384,
             hq=32, hkv=8, d=128, page=64, lens_seed=7),
        # one generated token of a single long context
        dict(name="attn_step_1_long", op="attn", dtype="bf16", seqs=1, new=1, past=131071,
             hq=32, hkv=8, d=128, page=256, lens_seed=8),
        # a prompt's chunk over what its earlier chunks left in the cache, ragged, small pages
        dict(name="attn_chunk_ragged", op="attn", dtype="bf16", seqs=4, new=1000, past=12000,
             hq=16, hkv=4, d=128, page=16, lens_seed=9),
        # a whole prompt from an empty cache
        dict(name="attn_prompt_8k", op="attn", dtype="bf16", seqs=1, new=8192, past=0,
             hq=32, hkv=8, d=128, page=128, lens_seed=10),
        # fp32, d = 64, a mixed batch of short chunks
        dict(name="attn_f32_mixed", op="attn", dtype="fp32", seqs=5, new=150, past=700,
             hq=4, hkv=2, d=64, page=32, lens_seed=11),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8] if hkv < 8 else [1, 2, 4])
    c = dict(op=op, dtype=dtype, hq=hq, hkv=hkv, d=d, lens_seed=rng.randrange(1 << 20))
    if op in ("norm_rope", "norm_rope_bwd"):
        c.update(tokens=_log_int(rng, 1, 40000), base=rng.choice([1e4, 1e6]),
                 fused=rng.random() < 0.5)
        c["docs"] = min(c["tokens"], _log_int(rng, 1, 64))
        if op == "norm_rope_bwd":
            c["grad"] = "fp32" if dtype == "fp32" else rng.choice(["fp32", "bf16"])
        return c
    c["page"] = rng.choice([16, 32, 48, 64, 128, 256])
    c["seqs"] = _log_int(rng, 1, 64)
    if op == "append":
        c.update(new=1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 8192 // c["seqs"])),
                 past=_log_int(rng, 1, 4096), base=rng.choice([1e4, 1e6]),
                 norm=rng.random() < 0.7)
        return c
    if rng.random() < 0.5:
        c.update(new=1, past=_log_int(rng, 1, 2 ** 19 // c["seqs"]))
    else:
        c.update(new=_log_int(rng, 2, max(2, 4096 // c["seqs"])), past=_log_int(rng, 1, 8192))
    if dtype == "fp32":                     # fp32 serving is for checks, at short lengths
        c.update(new=min(c["new"], 256), past=min(c["past"], 8192))
    return c


def _doc_lens(c):
    """`docs` document lengths that sum to `tokens`: cuts drawn uniformly (ragged, some short)."""
    r = random.Random(c["lens_seed"])
    cuts = sorted(r.randrange(c["tokens"] + 1) for _ in range(c["docs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [c["tokens"]])]


def _seq_lens(c):
    """(new tokens, tokens of the cache with them) of every sequence.  One sequence, or single
    tokens, take `new` as it is; the cached lengths are spread over their logarithm."""
    r = random.Random(c["lens_seed"])
    n = c["seqs"]
    new = [c["new"]] * n if n == 1 or c["new"] == 1 else [r.randint(1, c["new"]) for _ in range(n)]
    if n == 1 or c["past"] == 0:
        past = [c["past"]] * n
    else:
        past = [int(math.exp(r.uniform(0, math.log(c["past"] + 1)))) - 1 for _ in range(n)]
        past[r.randrange(n)] = c["past"]
    return new, [a + b for a, b in zip(new, past)]


# ------------------------------------------------------------------ inputs

def _bounds(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def _qkv(c, T, gen, fused, scale_q=1.0):
    """q, k, v [T, heads, d]; fused: views of one projection's [T, (hq + 2 hkv) d] output."""
    dt, hq, hkv, d = _DT[c["dtype"]], c["hq"], c["hkv"], c["d"]
    x = torch.randn(T, hq + 2 * hkv, d, generator=gen, device="cuda")
    x[:, :hq] *= scale_q
    x = x.to(dt)
    parts = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    return parts if fused else tuple(t.contiguous() for t in parts)


def _weights(c, gen):
    """Norm weights near one, as training leaves them."""
    dt = _DT[c["dtype"]]
    return tuple((1 + 0.1 * torch.randn(c["d"], generator=gen, device="cuda")).to(dt)
                 for _ in range(2))


def _cache(c, kv_lens, gen):
    """Page pools [n_pages, hkv, page, d] and the sequences' page table: pages in shuffled order,
    as a pool that has served earlier requests hands them out; unused entries -1."""
    page, dt = c["page"], _DT[c["dtype"]]
    need = [-(-x // page) for x in kv_lens]
    total = sum(need)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((c["seqs"], max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    shape = (total, c["hkv"], page, c["d"])
    pools = []
    for _ in range(2):
        pool = torch.empty(shape, dtype=dt, device="cuda")
        step = max(1, (1 << 28) // (shape[1] * shape[2] * shape[3]))
        for a in range(0, total, step):
            b = min(total, a + step)
            pool[a:b] = torch.randn((b - a,) + shape[1:], generator=gen, device="cuda").to(dt)
        pools.append(pool)
    return pools[0], pools[1], table


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case=c)
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        q, k, _ = _qkv(c, c["tokens"], gen, c["fused"])
        wq, wk = _weights(c, gen)
        st.update(q=q, k=k, wq=wq, wk=wk, cu=_bounds(_doc_lens(c)))
        if c["op"] == "norm_rope_bwd":
            g = _DT[c["grad"]]
            st["dq"] = torch.randn(q.shape, generator=gen, device="cuda").to(g)
            st["dk"] = torch.randn(k.shape, generator=gen, device="cuda").to(g)
        return st
    new, kv = _seq_lens(c)
    kp, vp, table = _cache(c, kv, gen)
    st.update(k_pages=kp, v_pages=vp, table=table, cu=_bounds(new), max_new=max(new),
              kv_lens=torch.tensor(kv, dtype=torch.int32, device="cuda"))
    if c["op"] == "append":
        q, k, v = _qkv(c, sum(new), gen, True)
        wq, wk = _weights(c, gen) if c["norm"] else (None, None)
        st.update(q=q, k=k, v=v, wq=wq, wk=wk)
    else:
        st["q"] = _qkv(c, sum(new), gen, False, 2.0)[0]
    return st


# ------------------------------------------------------------------ plain forms

def _segment(cu, T):
    """Segment of every packed token and its offset in it."""
    t = torch.arange(T, device=cu.device)
    seg = torch.searchsorted(cu[1:].long(), t, right=True)
    return seg, t - cu.long()[seg]


def _cos_sin(pos, d, base):
    """cos and sin of pos * base^(-2i/d), the angles in 64 bits."""
    i = torch.arange(d // 2, device=pos.device, dtype=torch.float64)
    a = pos.double()[:, None] * torch.pow(float(base), -2.0 * i / d)[None, :]
    return torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]


def _rotate(x, cos, sin):
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _norm(x, w, eps):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _plain_norm_rope(st):
    c = st["case"]
    _, pos = _segment(st["cu"], c["tokens"])
    cos, sin = _cos_sin(pos, c["d"], c["base"])
    return tuple(_rotate(_norm(x.float(), w.float(), _EPS), cos, sin).to(x.dtype)
                 for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])))


def _plain_norm_rope_bwd(st):
    c = st["case"]
    _, pos = _segment(st["cu"], c["tokens"])
    cos, sin = _cos_sin(pos, c["d"], c["base"])
    dxs, dws = [], []
    for x, w, dy in ((st["q"], st["wq"], st["dq"]), (st["k"], st["wk"], st["dk"])):
        xf = x.float()
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + _EPS)
        g = _rotate(dy.float(), cos, -sin)
        xh = xf * r
        dws.append((g * xh).sum((0, 1)))
        u = g * w.float()
        dxs.append((r * (u - xh * (u * xh).mean(-1, keepdim=True))).to(x.dtype))
    return dxs[0], dxs[1], dws[0], dws[1]


def _plain_append(st):
    c = st["case"]
    T = st["q"].shape[0]
    seg, off = _segment(st["cu"], T)
    n_new = (st["cu"][1:] - st["cu"][:-1]).long()
    pos = st["kv_lens"].long()[seg] - n_new[seg] + off
    page = st["table"].long()[seg, pos // c["page"]]
    slot = pos % c["page"]
    cos, sin = _cos_sin(pos, c["d"], c["base"])

    def turned(x, w):
        y = x.float()
        return _rotate(_norm(y, w.float(), _EPS) if c["norm"] else y, cos, sin).to(x.dtype)

    st["k_pages"][page, :, slot] = turned(st["k"], st["wk"])
    st["v_pages"][page, :, slot] = st["v"]
    return turned(st["q"], st["wq"]), st["k_pages"], st["v_pages"]


def _plain_attn(st):
    c = st["case"]
    n, hq, hkv, d, qm = c["seqs"], c["hq"], c["hkv"], c["d"], st["max_new"]
    G, T, dev = hq // hkv, st["q"].shape[0], st["q"].device
    L = st["table"].shape[1] * c["page"]
    seg, off = _segment(st["cu"], T)
    kv = st["kv_lens"].long()
    n_new = (st["cu"][1:] - st["cu"][:-1]).long()
    at = st["table"].long().clamp(min=0)
    kf = st["k_pages"][at].permute(0, 2, 1, 3, 4).reshape(n, hkv, L, d).float()
    vf = st["v_pages"][at].permute(0, 2, 1, 3, 4).reshape(n, hkv, L, d).float()
    key = torch.arange(L, device=dev)
    vf = torch.where((key[None] < kv[:, None])[:, None, :, None], vf, torch.zeros((), device=dev))
    qp = torch.zeros(n, qm, hkv, G, d, device=dev)
    qp[seg, off] = st["q"].float().view(T, hkv, G, d)
    qp = qp.permute(0, 2, 3, 1, 4).reshape(n, hkv, G * qm, d)
    s = torch.matmul(qp, kf.transpose(2, 3)).view(n, hkv, G, qm, L) * d ** -0.5
    pos = (kv - n_new)[:, None] + torch.arange(qm, device=dev)[None]
    hidden = key[None, None] > torch.minimum(pos, kv[:, None] - 1)[:, :, None]
    s.masked_fill_(hidden[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros((), device=dev), m)
    s = torch.exp(s - m)
    l = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(n, hkv, G * qm, L), vf).view(n, hkv, G, qm, d)
    o = o / torch.where(l > 0, l, torch.ones((), device=dev))
    lse = (m + torch.log(l))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(n, qm, hq, d)[seg, off]
    lse = lse.permute(0, 3, 1, 2).reshape(n, qm, hq)[seg, off]
    return o.to(st["q"].dtype), lse


# ------------------------------------------------------------------ the package's calls

def _own(st):
    msa, c = _msa(), st["case"]
    if c["op"] == "norm_rope":
        return msa.qk_norm_rope(st["q"], st["k"], st["cu"], c["base"], wq=st["wq"], wk=st["wk"],
                                eps=_EPS)
    if c["op"] == "norm_rope_bwd":
        if "ws" not in st:                  # a training program keeps it from step to step
            st["ws"] = msa.qk_norm_rope_workspace(st["q"], st["k"])
        return msa.qk_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], st["cu"], c["base"],
                                    wq=st["wq"], wk=st["wk"], eps=_EPS, ws=st["ws"])
    if "ws" not in st:                      # a serving program keeps it from step to step
        st["ws"] = msa.paged_workspace(st["q"], st["k_pages"], st["kv_lens"])
    if c["op"] == "append":
        q = msa.paged_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"],
                             st["kv_lens"], st["cu"], q=st["q"], base=c["base"], wq=st["wq"],
                             wk=st["wk"], eps=_EPS if c["norm"] else None, ws=st["ws"])
        return q, st["k_pages"], st["v_pages"]
    return msa.paged_attn_fwd(st["q"], st["k_pages"], st["v_pages"], st["table"], st["kv_lens"],
                              st["cu"], max_new=st["max_new"], ws=st["ws"])


def run(state):
    if own:
        return _own(state)
    return {"norm_rope": _plain_norm_rope, "norm_rope_bwd": _plain_norm_rope_bwd,
            "append": _plain_append, "attn": _plain_attn}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def _pairs(new, kv):
    """Visible (query, key) pairs of a causal chunk: sum over its tokens of position + 1."""
    return sum(n * (x - n) + n * (n + 1) // 2 for n, x in zip(new, kv))


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        n = c["tokens"] * (c["hq"] + c["hkv"]) * c["d"]
        w = 2 * c["d"]
        if c["op"] == "norm_rope":
            return {"bytes": 2 * n * es + w * es, "flops": 8 * n}
        gs = 2 if c["grad"] == "bf16" else 4
        return {"bytes": n * (2 * es + gs) + w * (es + 4), "flops": 16 * n}
    new, kv = _seq_lens(c)
    T = sum(new)
    if c["op"] == "append":
        n = T * (c["hq"] + 2 * c["hkv"]) * c["d"]
        return {"bytes": 2 * n * es, "flops": (8 if c["norm"] else 3) * n}
    return {"bytes": es * c["d"] * (2 * T * c["hq"] + 2 * sum(kv) * c["hkv"]) + 4 * T * c["hq"],
            "flops": 4 * c["d"] * c["hq"] * _pairs(new, kv)}


# ------------------------------------------------------------------ 64-bit values

def _turn64(x, pos, base, inverse=False):
    """Pair (i, i + d/2) as a complex number, times exp(+-1j pos base^(-2i/d))."""
    d = x.shape[-1]
    theta = torch.tensor([float(base) ** (-2.0 * i / d) for i in range(d // 2)],
                         dtype=torch.float64, device=x.device)
    a = pos.double()[:, None] * theta
    turn = torch.polar(torch.ones_like(a), -a if inverse else a)[:, None, :]
    z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn
    return torch.cat([z.real, z.imag], -1)


def _unit64(x):
    return (x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS) ** -0.5


def _positions(starts_lens):
    return torch.cat([torch.arange(a, a + n, device="cuda") for a, n in starts_lens])


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] in ("norm_rope", "norm_rope_bwd"):
        pos = _positions([(0, n) for n in _doc_lens(c)])
        out, dws = [], []
        for x, w, dy in ((st["q"], st["wq"], st.get("dq")), (st["k"], st["wk"], st.get("dk"))):
            x, w = x.double(), w.double()
            r = _unit64(x)
            if dy is None:
                out.append(_turn64(x * r * w, pos, c["base"]))
                continue
            g = _turn64(dy.double(), pos, c["base"], inverse=True)
            dws.append((g * x * r).sum((0, 1)))
            gw = g * w
            # d/dx of r(x) x: r on the diagonal, minus r^3 x x^T / d
            out.append(r * gw - r ** 3 * x * (gw * x).sum(-1, keepdim=True) / c["d"])
        return tuple(out + dws)
    new, kv = _seq_lens(c)
    if c["op"] == "append":
        pos = _positions([(b - a, a) for a, b in zip(new, kv)])
        done = []
        for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
            x = x.double()
            done.append(_turn64(x * _unit64(x) * w.double() if c["norm"] else x, pos, c["base"]))
        kp, at = st["k_pages"].double(), 0
        for s, (a, b) in enumerate(zip(new, kv)):
            p = torch.arange(b - a, b, device="cuda")
            pg = st["table"][s].long()[p // c["page"]]
            kp[pg, :, p % c["page"]] = done[1][at:at + a]
            at += a
        return done[0], kp, None
    if 4.0 * c["d"] * c["hq"] * _pairs(new, kv) > 5e13:
        return None
    T, hq, hkv, d, G = sum(new), c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    o = torch.zeros(T, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((T, hq), float("-inf"), dtype=torch.float64, device="cuda")
    at = 0
    for s, (a, b) in enumerate(zip(new, kv)):
        pages = st["table"][s, :-(-b // c["page"])].long()
        for g in range(hkv):
            K = st["k_pages"][pages, g].reshape(-1, d)[:b].double()
            V = st["v_pages"][pages, g].reshape(-1, d)[:b].double()
            step = max(1, (1 << 27) // (G * b))
            for t0 in range(0, a, step):
                t1 = min(a, t0 + step)
                q = st["q"][at + t0:at + t1, g * G:(g + 1) * G].double()
                x = torch.einsum("thd,kd->thk", q, K) / math.sqrt(d)
                far = torch.arange(b, device="cuda")[None] > \
                    torch.arange(b - a + t0, b - a + t1, device="cuda")[:, None]
                x = x.masked_fill(far[:, None], float("-inf"))
                z = torch.logsumexp(x, -1)
                lse[at + t0:at + t1, g * G:(g + 1) * G] = z
                o[at + t0:at + t1, g * G:(g + 1) * G] = torch.einsum(
                    "thk,kd->thd", torch.exp(x - z[..., None]), V)
        at += a
    return o, lse
