"""The attention operators in numpy, 64 bits.

Test infrastructure: written from the formulas, with nothing of the package.
Rows are [token][head][dim]; 16-bit inputs come as float64 arrays of their exact
values.

* ``norm_rotate``: n = x w / sqrt(mean(x^2) + eps) per head, then the rotation
  (a cos t - b sin t, b cos t + a sin t) of pairs (i, i + R/2) or (2i, 2i + 1);
* ``round16``: one rounding to bf16 or fp16, nearest even;
* ``attend``: out = softmax(scale q K^T) V of one sequence, with the sums that
  a bound on a kernel's error needs.
"""
from __future__ import annotations

import numpy as np

# significant bits, exponent of the smallest step
_FORMATS = {"bf16": (8, -133), "fp16": (11, -24)}


def round16(x: np.ndarray, dtype: str) -> np.ndarray:
    """x rounded to a 16-bit type (nearest even, subnormals kept; no overflow), as float64."""
    bits, lowest = _FORMATS[dtype]
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - bits, lowest))
    return np.rint(x / step) * step


def norm_rotate(x, weight, eps, cos, sin, interleaved):
    """x [T][heads][D]; weight [D] or None; cos, sin [T][R/2]."""
    y = np.array(x, dtype=np.float64)
    if weight is not None:
        y = y * weight / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps)
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        first, second = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        first, second = slice(0, half), slice(half, 2 * half)
    a, b = y[..., first].copy(), y[..., second].copy()
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def attend(q, k, v, scale, causal=True):
    """One sequence: q [n][heads][D], k, v [m][kv heads][D]; row i sees keys 0 .. m - n + i (causal) or all.

    Returns out [n][heads][D], lse [n][heads], and for error bounds spread [n][heads][D] = sum_j p_j |v_j| and
    reach [n][heads] = the largest scale * sum_d |q_d k_jd| over the row's keys."""
    n, H, D = q.shape
    m, K = k.shape[:2]
    out, spread = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, reach = np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        end = max(0, m - n + i + 1) if causal else m
        if end == 0:
            continue
        for h in range(H):
            kk, vv = k[:end, h // (H // K)], v[:end, h // (H // K)]
            s = (kk @ q[i, h]) * scale
            top = s.max()
            p = np.exp(s - top)
            lse[i, h] = top + np.log(p.sum())
            p /= p.sum()
            out[i, h], spread[i, h] = p @ vv, p @ np.abs(vv)
            reach[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, spread, reach
