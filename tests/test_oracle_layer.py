"""Pins of the layer oracle (oracle/msa_layer.py): closed forms, central differences, torch
autograd in float64, and dense causal attention."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import msa_layer


def _rand(shape, seed):
    return np.random.default_rng(seed).standard_normal(shape)


def test_norm_rope_closed_form():
    """x = (3, 4, 0, 0): mean square 25/4; weight 2; position 2 rotates pair 0 by 2 rad."""
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y = oracle.norm_rope(x, np.full(4, 2.0), [2], 10000.0, 0.0)[0, 0]
    n = [3 / 2.5 * 2, 4 / 2.5 * 2]
    want = [n[0] * math.cos(2), n[1] * math.cos(0.02), n[0] * math.sin(2), n[1] * math.sin(0.02)]
    np.testing.assert_allclose(y, want, atol=1e-14)


def test_norm_rope_matches_rope_of_docs_without_norm():
    x, cu = _rand((7, 2, 8), 1), [0, 3, 7]
    pos = oracle.doc_positions(cu)
    np.testing.assert_array_equal(oracle.rotate_heads(x, pos, 500.0),
                                  oracle.rope_docwise(x, cu, 500.0))
    np.testing.assert_allclose(oracle.rotate_heads(oracle.rotate_heads(x, pos, 500.0), pos, 500.0,
                                                   inverse=True), x, atol=1e-14)


@pytest.mark.parametrize("weighted", [True, False])
def test_backward_is_the_gradient(weighted):
    """Against central differences of norm_rope, and torch autograd of the formula."""
    T, h, d, base, eps = 5, 3, 8, 100.0, 1e-3
    x, dy, pos = _rand((T, h, d), 2), _rand((T, h, d), 3), np.array([0, 1, 2, 7, 1000])
    w = 1 + 0.3 * _rand(d, 4) if weighted else None
    dx, dw = oracle.norm_rope_backward(dy, x, w, pos, base, eps)
    f = lambda x, w: (oracle.norm_rope(x, w, pos, base, eps) * dy).sum()  # noqa: E731
    step = 1e-5
    for at in [(0, 0, 0), (3, 1, 5), (4, 2, 7)]:
        a, b = x.copy(), x.copy()
        a[at] += step
        b[at] -= step
        assert abs((f(a, w) - f(b, w)) / (2 * step) - dx[at]) < 1e-8
    ones = np.ones(d) if w is None else w
    for i in range(d):
        a, b = ones.copy(), ones.copy()
        a[i] += step
        b[i] -= step
        assert abs((f(x, a) - f(x, b)) / (2 * step) - dw[i]) < 1e-8
    tx = torch.tensor(x, requires_grad=True)
    tw = torch.tensor(ones, requires_grad=True)
    n = tx * (tx.square().mean(-1, keepdim=True) + eps).rsqrt() * tw
    ang = torch.tensor(oracle.rope_angles(pos, d, base))[:, None]
    p, q = n[..., :d // 2], n[..., d // 2:]
    y = torch.cat([p * ang.cos() - q * ang.sin(), q * ang.cos() + p * ang.sin()], -1)
    (y * torch.tensor(dy)).sum().backward()
    np.testing.assert_allclose(dx, tx.grad.numpy(), atol=1e-12)
    np.testing.assert_allclose(dw, tw.grad.numpy(), atol=1e-12)


def test_append_then_attention_is_dense_causal_attention():
    """Two steps through a shuffled page table, then every row against torch's attention over
    the same sequence."""
    page, hkv, G, d = 16, 2, 3, 8
    lens = [37, 5]
    table = np.array([[4, 0, 2], [1, -1, -1]])
    kp, vp = np.zeros((5, hkv, page, d)), np.zeros((5, hkv, page, d))
    K = [_rand((L, hkv, d), 10 + i) for i, L in enumerate(lens)]
    V = [_rand((L, hkv, d), 20 + i) for i, L in enumerate(lens)]
    Q = [_rand((L, hkv * G, d), 30 + i) for i, L in enumerate(lens)]
    first = [20, 0]
    for a, b in ((([0, 0]), first), (first, lens)):
        new = [y - x for x, y in zip(a, b)]
        cu = [0] + list(np.cumsum(new))
        cat = lambda X: np.concatenate([x[i:j] for x, i, j in zip(X, a, b)])  # noqa: E731
        kp, vp = oracle.paged_append(kp, vp, cat(K), cat(V), table, b, cu, page)
        o, lse, _, _ = oracle.paged_attention(cat(Q), kp, vp, table, b, cu, page, 0.4)
    at = 0
    for i, L in enumerate(lens):
        q, k, v = (torch.tensor(x).transpose(0, 1) for x in (Q[i], K[i], V[i]))
        k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
        ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True, scale=0.4)
        n = L - first[i]
        np.testing.assert_allclose(o[at:at + n], ref.transpose(0, 1)[first[i]:].numpy(), atol=1e-12)
        x = 0.4 * q @ k.transpose(1, 2)
        x = x.masked_fill(torch.ones(L, L).triu(1).bool(), -math.inf)
        np.testing.assert_allclose(lse[at:at + n], x.logsumexp(-1).T[first[i]:].numpy(), atol=1e-12)
        at += n


def test_attention_rows_that_see_nothing():
    kp = _rand((2, 1, 16, 4), 1)
    q = _rand((3, 1, 4), 2)
    o, lse, _, _ = oracle.paged_attention(q, kp, kp, np.array([[0], [1]]), [1, 0], [0, 3, 3], 16, 1.0)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all()      # positions -2, -1
    np.testing.assert_allclose(o[2, 0], kp[0, 0, 0], atol=1e-15)    # sees key 0 alone


def test_append_skips_tokens_without_a_page():
    kp = np.zeros((2, 1, 16, 4))
    k = np.ones((4, 1, 4))
    table = np.array([[0, 7], [1, -1]])
    a, _ = msa_layer.paged_append(kp, kp, k, k, table, [18, 33], [0, 2, 4], 16)
    # sequence 0: positions 16, 17 (page 7 of 2: none); sequence 1: 31 (entry -1), 32 (past the row)
    assert (a == 0).all()
