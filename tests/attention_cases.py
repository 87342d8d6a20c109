"""Shared helpers of the attention GPU tests: seeded inputs, the oracle on them, and derived error bounds."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from oracle import attention as oa
from moe_expert_layer_top_gb300 import attention

TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # largest relative error of one rounding
HALF_TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # largest absolute error among the type's subnormal values


def rows16(rng, shape, dtype, sigma=1.0):
    """Random values of a 16-bit type, as float64."""
    return oa.round16(rng.standard_normal(shape) * sigma, dtype)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(TORCH[dtype]) if dtype else t).cuda()


def f64(t):
    return t.double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def check_attention(out, lse, q, k, v, scale, dtype, inner, causal=True):
    """One sequence's rows against the oracle, element by element.

    Error of a probability p_j before it meets V: the score is a binary32 sum of D products of at most `reach` in
    total magnitude (recursive summation: D 2^-24 reach), scaled and moved by the maximum (three roundings of
    values of at most 2 reach), then exp2 (2^-22) - together delta, absolute in the exponent - and p is rounded to
    `inner`. Sums over the keys are binary32: m 2^-24 of the sum of magnitudes. The result is divided by a sum with
    the same delta and rounded to its type. So |error| <= half |o| + (inner + 2 delta + 2 m 2^-24) sum_j p_j |v_j|,
    up to products of these. Where a rounding falls among subnormal values its error is absolute instead: half the
    smallest step of the result's type for o, and for a p_j (taken relative to the row's maximum, so the sum of all
    is at least 1) half the smallest step of `inner`, or 2^-126 where exp2 flushes, times |v_j|."""
    n, H, D = q.shape
    o, z, spread, reach = oa.attend(q, k, v, scale, causal)
    m = len(k)
    delta = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -21
    rel = HALF_STEP[inner]
    bound = HALF_STEP[dtype] * np.abs(o) + 1.05 * (rel + 2 * delta + 2 * m * 2.0 ** -24)[..., None] * spread
    tiny = max(HALF_TINY[inner], 2.0 ** -126)
    seen = np.concatenate([np.zeros((1,) + v.shape[1:]), np.cumsum(np.abs(v), axis=0)])  # sums of |v| over the first keys
    ends = np.clip(m - n + np.arange(n) + 1, 0, m) if causal else np.full(n, m)
    bound += HALF_TINY[dtype] + tiny * np.repeat(seen[ends], H // v.shape[1], axis=1)
    err = np.abs(f64(out) - o)
    assert np.isfinite(f64(out)).all()
    assert (err <= bound).all(), f"out: {np.max(err / np.maximum(bound, 1e-300)):.3f} of its bound"
    empty = np.isneginf(z)
    if lse is not None:
        got = f64(lse)
        assert (np.isneginf(got) == empty).all()
        zz = np.where(empty, 0.0, z)
        lim = delta + m * 2.0 ** -24 + 4 * 2.0 ** -24 * (np.abs(zz) + reach)
        assert (np.abs(np.where(empty, 0.0, got) - zz) <= lim).all()
    return err


class Cache:
    """A paged cache with random rows in shuffled pages, and the values it stands for."""

    def __init__(self, rng, lengths, K, D, page, spare=3, sigma=1.0):
        self.lengths, self.page = lengths, page
        need = [-(-n // page) for n in lengths]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        self.max_pages = max(need + [1])
        table = np.full((len(lengths), self.max_pages), -7, dtype=np.int32)  # past the length: never looked at
        parts = {}
        for name, width in (("k_codes", D // 2), ("k_scales", D // 32), ("v_codes", D // 2), ("v_scales", D // 32)):
            parts[name] = rng.integers(0, 256, (pages, K, page, width)).astype(np.uint8)
            if name.endswith("scales"):
                parts[name][:] = 255  # NaN by the format: reading one would show
        self.k, self.v = [], []
        at = 0
        for b, n in enumerate(lengths):
            mine = order[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine
            for x in ("k", "v"):
                rows = oa.round16(rng.standard_normal((n, K, D)) * sigma, "bf16")
                codes, scales = oracle.mxfp4_quantize(rows)
                for j in range(n):
                    parts[x + "_codes"][mine[j // page], :, j % page] = codes[j]
                    parts[x + "_scales"][mine[j // page], :, j % page] = scales[j]
                getattr(self, x).append(np.asarray(oracle.mxfp4_dequantize(codes, scales), dtype=np.float64))
        self.table = dev(table)
        self.cache = attention.KVCacheMXFP4(*(dev(parts[p]) for p in ("k_codes", "k_scales", "v_codes", "v_scales")))


def offsets(counts):
    return [0] + np.cumsum(counts).tolist()
