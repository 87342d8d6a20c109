"""Shared helpers of the GPU tests of a step with drafted trees."""
from __future__ import annotations

import numpy as np
import torch

import attention_cases as ac
from oracle import speculative as osp
from moe_expert_layer_top_gb300 import abi, attention


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def random_tree(rng, n, kind="tree"):
    """Parents of n rows: a chain, a tree in any order that puts rows behind their parents, or several roots."""
    if kind == "chain":
        return list(range(-1, n - 1))
    parents = [-1]
    for i in range(1, n):
        parents.append(-int(rng.integers(1, 9)) if kind == "forest" and rng.random() < 0.2 else int(rng.integers(0, i)))
    return parents[:n]


def check_tree(out, lse, q, k, v, parents, scale, dtype):
    """One sequence's rows against the oracle, element by element, within the bound that
    attention_cases.check_attention derives (probabilities rounded to fp16), for the keys that each row sees."""
    D = q.shape[-1]
    o, z, spread, reach, seen = osp.attend_tree(q, k, v, parents, scale)
    m = len(k)
    delta = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -21
    bound = ac.HALF_STEP[dtype] * np.abs(o) + 1.05 * (ac.HALF_STEP["fp16"] + 2 * delta + 2 * m * 2.0 ** -24)[..., None] * spread
    tiny = np.einsum("nm,mkd->nkd", seen.astype(float), np.abs(v)) if m else np.zeros((len(q),) + v.shape[1:])
    bound += ac.HALF_TINY[dtype] + ac.HALF_TINY["fp16"] * np.repeat(tiny, q.shape[1] // v.shape[1], axis=1)
    got = ac.f64(out)
    assert np.isfinite(got).all()
    err = np.abs(got - o)
    assert (err <= bound).all(), f"out: {np.max(err / np.maximum(bound, 1e-300)):.3f} of its bound"
    if lse is not None:
        empty = np.isneginf(z)
        got = ac.f64(lse)
        assert (np.isneginf(got) == empty).all()
        zz = np.where(empty, 0.0, z)
        lim = delta + m * 2.0 ** -24 + 4 * 2.0 ** -24 * (np.abs(zz) + reach)
        assert (np.abs(np.where(empty, 0.0, got) - zz) <= lim).all()


def run_tree(seqs, H, K, D, page, dtype, max_rows, seed=0, sigma=1.0, kind="tree", scale=None):
    """seqs: (rows, length) of each. Two rows of q and out lie behind the last sequence."""
    rng = np.random.default_rng(seed)
    lengths = [s[1] for s in seqs]
    c = ac.Cache(rng, lengths, K, D, page, sigma=sigma)
    cr = ac.offsets([s[0] for s in seqs])
    trees = [random_tree(rng, n, kind) for n, _ in seqs]
    q = ac.rows16(rng, (cr[-1] + 2, H, D), dtype, 1.5)
    out = torch.full((cr[-1] + 2, H, D), 3.0, device="cuda").to(ac.TORCH[dtype])
    st = status()
    parents = ac.i32(sum(trees, []) + [5, 7])  # those behind the last sequence are not looked at
    got, lse = attention.attend_tree(ac.dev(q, dtype), c.cache, c.table, ac.i32(lengths), ac.i32(cr), parents,
                                     max_rows=max_rows, scale=scale, out=out, return_lse=True, d_status=st)
    assert st.item() == abi.MOE_OK
    assert (out[cr[-1]:] == 3).all()
    for b in range(len(seqs)):
        r = slice(cr[b], cr[b + 1])
        check_tree(got[r], lse[r], q[r], c.k[b], c.v[b], trees[b], D ** -0.5 if scale is None else scale, dtype)
    return c, q, parents, ac.i32(cr), got, lse
