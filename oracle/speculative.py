"""A speculative step with a tree of drafted tokens, in numpy and 64 bits.

Test infrastructure: written from the formulas, with nothing of the package.

* ``ancestors``: which rows of a tree each row sees, itself and those on its way to the root;
* ``attend_tree``: out = softmax(scale q K^T) V of one sequence whose last rows form a tree, with the sums that a bound
  on a kernel's error needs;
* ``verify``: which drafted tokens the target accepts and the token behind them, with the distance of every choice from
  its border;
* ``commit``: the rows of a cache after the accepted ones have moved.
"""
from __future__ import annotations

import numpy as np


def ancestors(parents) -> np.ndarray:
    """[n][n], true where row i sees row j. A parent that does not lie in front of its row counts as none."""
    n = len(parents)
    seen = np.eye(n, dtype=bool)
    for i, p in enumerate(parents):
        if 0 <= p < i:
            seen[i] |= seen[p]
    return seen


def attend_tree(q, k, v, parents, scale):
    """One sequence: q [n][heads][D], k, v [m][kv heads][D], the last n keys being the rows' own.

    Returns out [n][heads][D], lse [n][heads], and for error bounds spread [n][heads][D] = sum_j p_j |v_j|, reach
    [n][heads] = the largest scale * sum_d |q_d k_jd| over the row's keys, and seen [n][m]."""
    n, H, D = q.shape
    m, K = k.shape[:2]
    seen = np.zeros((n, m), dtype=bool)
    seen[:, :max(0, m - n)] = True
    tree = ancestors(parents)
    for j in range(n):
        if m - n + j >= 0:
            seen[:, m - n + j] = tree[:, j]
    out, spread = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, reach = np.full((n, H), -np.inf), np.zeros((n, H))
    for h in range(H):
        kk, vv = k[:, h // (H // K)], v[:, h // (H // K)]
        s = np.where(seen, (q[:, h] @ kk.T) * scale, -np.inf)
        some = seen.any(1)
        if not some.any():
            continue
        top = s[some].max(1)
        p = np.exp(s[some] - top[:, None])
        lse[some, h] = top + np.log(p.sum(1))
        p /= p.sum(1, keepdims=True)
        out[some, h], spread[some, h] = p @ vv, p @ np.abs(vv)
        reach[some, h] = abs(scale) * np.where(seen, np.abs(q[:, h]) @ np.abs(kk).T, 0.0)[some].max(1)
    return out, lse, spread, reach, seen


def softmax(x, temperature):
    """The target's probabilities; at temperature 0 all on the first largest logit. None without a distribution."""
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or (x == np.inf).any() or not np.isfinite(x).any():
        return None
    if temperature == 0:
        p = np.zeros_like(x)
        p[np.argmax(x)] = 1.0
        return p
    w = np.exp((x - x.max()) / temperature)
    return w / w.sum()


def residual(p, draft, rejected):
    """What is left of p after rejections, not normalised: with a draft max(p_k - q, 0) in turn, else p without the tokens."""
    left = np.array(p)
    if draft is None:
        left[list(rejected)] = 0.0
        return left
    for _ in rejected:
        left = np.maximum(left / left.sum() - draft, 0.0) if left.sum() > 0 else left
    return left


def accept_chance(p, draft, rejected, token) -> float:
    """The probability with which a child is accepted when those in `rejected` have been rejected."""
    left = residual(p, draft, rejected)
    whole = left.sum()
    if whole <= 0:
        return 0.0
    q = 1.0 if draft is None else float(draft[token])
    return min(1.0, left[token] / whole / q) if q > 0 else float(left[token] > 0)


def verify(logits, tokens, parents, accept_u, sample_u, temperature=1.0, draft=None):
    """One sequence. Returns the accepted rows from the root on, the new token (-1 without a distribution), and the
    distances of the choices from their borders: the smallest |u - chance| over the children that were asked, and of the
    new token's running sums from sample_u, both as parts of the whole."""
    n, node, path, near = len(tokens), 0, [0], np.inf
    while True:
        p = softmax(logits[node], temperature)
        if p is None:
            return path, -1, near, np.inf
        q = None if draft is None else np.asarray(draft[node], dtype=np.float64)
        rejected, found = [], None
        for i in range(1, n):
            if parents[i] != node or not 0 <= tokens[i] < len(p):
                continue
            if temperature == 0:
                yes = p[tokens[i]] == 1.0
            else:
                chance = accept_chance(p, q, rejected, tokens[i])
                near = min(near, abs(float(accept_u[i]) - chance))
                yes = float(accept_u[i]) < chance
            if yes:
                found = i
                break
            rejected.append(tokens[i])
        if found is None:
            break
        node = found
        path.append(found)
    if temperature == 0:
        return path, int(np.argmax(p)), near, np.inf
    left = residual(p, q, rejected)
    if left.sum() <= 0:
        left = p
    sums = np.cumsum(left) / left.sum()
    u = float(sample_u)
    above = np.flatnonzero((sums > u) & (left > 0))
    token = int(above[0]) if len(above) else int(np.flatnonzero(left > 0)[-1])
    inner = sums[:-1][left[1:] > 0]  # borders between tokens
    return path, token, near, float(np.abs(inner - u).min(initial=np.inf))


def commit(rows, base, path):
    """rows [tokens][...] of one sequence after row base + path[j] has moved to base + j; the new length."""
    out = np.array(rows)
    for j, p in enumerate(path):
        out[base + j] = rows[base + p]
    return out, base + len(path)
