"""What pins the oracle of a step with drafted trees: closed forms, the causal oracle, and exact probabilities."""
import itertools

import numpy as np
import pytest

from oracle import attention as oa
from oracle import speculative as osp


def test_ancestors_by_hand():
    #      0
    #    1   2
    #   3 4   5      6: a second root
    want = np.array([[1, 0, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0, 0], [1, 1, 0, 1, 0, 0, 0],
                     [1, 1, 0, 0, 1, 0, 0], [1, 0, 1, 0, 0, 1, 0], [0, 0, 0, 0, 0, 0, 1]], dtype=bool)
    np.testing.assert_array_equal(osp.ancestors([-1, 0, 0, 1, 1, 2, -5]), want)
    np.testing.assert_array_equal(osp.ancestors([3, 1]), np.eye(2, dtype=bool))  # not in front of their rows


@pytest.mark.parametrize("n,m", [(1, 1), (5, 5), (4, 9), (6, 3), (3, 0)])
def test_a_chain_is_causal_attention(n, m):
    rng = np.random.default_rng(n + m)
    q, k, v = rng.standard_normal((n, 4, 8)), rng.standard_normal((m, 2, 8)), rng.standard_normal((m, 2, 8))
    got, want = osp.attend_tree(q, k, v, list(range(-1, n - 1)), 0.3), oa.attend(q, k, v, 0.3)
    for a, b in zip(got[:4], want):
        np.testing.assert_allclose(a, b, rtol=1e-13, atol=1e-15)


def test_a_tree_is_causal_attention_along_each_way():
    rng = np.random.default_rng(7)
    parents, m = [-1, 0, 0, 1, 2, 2, 4], 12
    n = len(parents)
    q, k, v = rng.standard_normal((n, 2, 8)), rng.standard_normal((m, 1, 8)), rng.standard_normal((m, 1, 8))
    out, lse = osp.attend_tree(q, k, v, parents, 0.5)[:2]
    for i in range(n):
        way = [i]
        while parents[way[0]] >= 0:
            way.insert(0, parents[way[0]])
        keys = list(range(m - n)) + [m - n + j for j in way]
        o, z = oa.attend(q[i:i + 1], k[keys], v[keys], 0.5)[:2]
        np.testing.assert_allclose(out[i], o[0], rtol=1e-13)
        np.testing.assert_allclose(lse[i], z[0], rtol=1e-13)


def test_residual_by_hand():
    p, q = np.array([0.5, 0.3, 0.2]), np.array([0.2, 0.6, 0.2])
    np.testing.assert_allclose(osp.residual(p, q, [1]), [0.3, 0.0, 0.0], atol=1e-15)
    np.testing.assert_allclose(osp.residual(p, q, [1, 1]), [0.8, 0.0, 0.0], atol=1e-15)  # 0.3 / 0.3 - 0.2
    np.testing.assert_allclose(osp.residual(p, None, [0, 2]), [0.0, 0.3, 0.0])


@pytest.mark.parametrize("children", [1, 2, 3])
@pytest.mark.parametrize("drafted", [True, False])
def test_the_first_token_is_distributed_as_the_target(children, drafted):
    """Over all draws of the children (with their probabilities), exactly: accepted or new, the token has the target's p."""
    rng = np.random.default_rng(children)
    V = 5
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    total = np.zeros(V)
    draws = itertools.product(range(V), repeat=children) if drafted else [(3, 0, 1)[:children]]
    for ys in draws:
        weight = float(np.prod(q[list(ys)])) if drafted else 1.0
        for k, y in enumerate(ys):
            chance = osp.accept_chance(p, q if drafted else None, ys[:k], y)
            total[y] += weight * chance
            weight *= 1.0 - chance
        left = osp.residual(p, q if drafted else None, ys)
        if weight > 1e-15:
            total += weight * left / left.sum()
    np.testing.assert_allclose(total, p, rtol=1e-12)


def test_the_residual_has_a_closed_form():
    """p_k = max(p - c_k q, 0) / N_k with c_(k+1) = c_k + N_k."""
    rng = np.random.default_rng(9)
    for _ in range(20):
        p, q = rng.dirichlet(np.ones(9)), rng.dirichlet(np.ones(9))
        c, N = 0.0, 1.0
        for k in range(5):
            left = osp.residual(p, q, [0] * k)
            np.testing.assert_allclose(left / left.sum(), np.maximum(p - c * q, 0) / N, rtol=1e-9, atol=1e-12)
            c += N
            N = np.maximum(p - c * q, 0).sum()


def test_verify_by_hand():
    ln = np.log
    logits = np.array([[ln(0.5), ln(0.25), ln(0.25)], [ln(0.1), ln(0.2), ln(0.7)], [0.0, 0.0, 0.0]])
    # root, its children 1 (token 1) and 2 (token 0)
    tokens, parents = [9, 1, 0], [-1, 0, 0]
    assert osp.verify(logits, tokens, parents, [0, 0.2, 0.0], 0.25)[:2] == ([0, 1], 1)      # 0.2 < p(1); 0.25 of (.1 .2 .7)
    path, token, near, edge = osp.verify(logits, tokens, parents, [0, 0.3, 0.6], 0.999)
    assert (path, token) == ([0, 2], 2)  # 0.3 > 0.25; 0.6 < 0.5 / 0.75; the last of a flat row
    np.testing.assert_allclose(near, 0.05)
    np.testing.assert_allclose(edge, 0.999 - 2 / 3)
    assert osp.verify(logits, tokens, parents, [0, 0.3, 0.7], 0.0)[:2] == ([0], 2)  # only token 2 is left
    assert osp.verify(logits, tokens, parents, [0, 0.3, 0.7], 0.0, temperature=0)[:2] == ([0, 2], 0)  # ties: the first
    draft = np.array([[0.25, 0.5, 0.25]] * 3)
    assert osp.verify(logits, tokens, parents, [0, 0.6, 0.0], 0.5, draft=draft)[:2] == ([0, 2], 1)  # 0.25/0.5 < 0.6
    logits[0, 2] = np.inf
    assert osp.verify(logits, tokens, parents, [0, 0.0, 0.0], 0.5)[:2] == ([0], -1)


def test_commit_by_hand():
    rows = np.arange(8)
    got, length = osp.commit(rows, 3, [0, 2, 4])
    np.testing.assert_array_equal(got, [0, 1, 2, 3, 5, 7, 6, 7])
    assert length == 6
