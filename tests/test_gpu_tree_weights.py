"""Attention of trees where values of very different size lie in one cache: a value far above the others, of a key that a row
does not see or that has no weight, must not cost the weights of the others bits."""
import numpy as np
import pytest
import torch

from moe_expert_layer_top_gb300 import abi, attention
from oracle import speculative as osp

import attention_cases as ac
import tree_cases as tc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_top_gb300.build as b
    b.build()
    abi.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("rows", [3, 60, 200])  # of a kv head 12, 240 and 800: both kinds of kernel
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("at", [5, 700, "unseen"])
@pytest.mark.parametrize("shift", [6, 12])
def test_a_large_value_without_weight(rows, D, dtype, at, shift):
    """Key 0 has nearly all the weight and a value of 0; what the row gets comes of 1,500 others, each some 2^-16 of the
    largest. One value is 2^shift above the rest, of a key whose score is far below, or of a row that the others do not see.

    A weight is 2^7 (or more) times its part of the row's largest, rounded to fp16: off by at most half a step, 2^-11 of
    itself, or 2^-25 in 2^7, 2^-32 of the largest, which the row's sum is not below. Beside that the bound is that of
    tree_cases.check_tree."""
    H, K, m = 4, 1, 1500
    rng = np.random.default_rng(rows + D)
    c = ac.Cache(rng, [m], K, D, 16)
    table = c.table[0].long()
    place = lambda j: (int(table[j // 16]), slice(None), j % 16)
    c.cache.v_scales[place(0)] = 0
    c.v[0][0] = 0.0
    parents = [-1, 0, 0] + [2] * (rows - 3)  # only row 1 sees row 1
    big = m - rows + 1 if at == "unseen" else at
    c.cache.v_scales[place(big)] += shift
    c.v[0][big] *= 2.0 ** shift
    if at != "unseen":  # the opposite of key 0, twice as large
        c.cache.k_codes[place(big)] = c.cache.k_codes[place(0)] ^ 0x88
        c.cache.k_scales[place(big)] = c.cache.k_scales[place(0)] + 1
        c.k[0][big] = -2.0 * c.k[0][0]
    k0 = c.k[0][0, 0]
    q = (11.0 * D ** 0.5 / (k0 @ k0)) * k0 + 0.2 * rng.standard_normal((rows, H, D))
    x = torch.from_numpy(q).to(ac.TORCH[dtype])
    q = x.double().numpy()
    st = tc.status()
    out, lse = attention.attend_tree(x.cuda(), c.cache, c.table, ac.i32([m]), ac.i32([0, rows]), ac.i32(parents), max_rows=rows,
                                     return_lse=True, d_status=st)
    assert st.item() == abi.MOE_OK
    o, z, spread, reach, seen = osp.attend_tree(q, c.k[0], c.v[0], parents, D ** -0.5)
    others = seen.copy()
    others[:, big] = False
    delta = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -21
    bound = ac.HALF_STEP[dtype] * np.abs(o) + 1.05 * (ac.HALF_STEP["fp16"] + 2 * delta + 2 * m * 2.0 ** -24)[..., None] * spread
    tiny = np.einsum("nm,mkd->nkd", others.astype(float), np.abs(c.v[0]))
    bound += ac.HALF_TINY[dtype] + 2.0 ** -32 * np.repeat(tiny, H // K, axis=1)
    keep = [i for i in range(rows) if not (at == "unseen" and i == 1)]
    err = np.abs(ac.f64(out) - o)[keep]
    assert (err <= bound[keep]).all(), f"{np.max(err / bound[keep]):.2f} of its bound"
    zz = lambda a: np.asarray(a)[keep]
    lim = delta + m * 2.0 ** -24 + 4 * 2.0 ** -24 * (np.abs(z) + reach)
    assert (np.abs(zz(ac.f64(lse)) - zz(z)) <= zz(lim)).all()


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
def test_large_values_along_long_contexts(D, dtype):
    """As above, with runs of more than 16 tiles of 128 keys, which agree on a scale together, several items a block, and
    large values without weight on both sides of where a run may end. Also scale codes of 255 behind the last
    token, and large ones: neither counts."""
    B, K, group, rows, m = 8, 8, 2, 40, 6000
    H = K * group
    rng = np.random.default_rng(D)
    lengths = [m - 37 * b for b in range(B)]
    c = ac.Cache(rng, lengths, K, D, 64)
    parents = [tc.random_tree(rng, rows) for _ in range(B)]
    q = np.zeros((B * rows, H, D))
    heavy = [(300, 3), (700, 12), (2047, 12), (2048, 13), (2303, 9), (4100, 13)]
    for b in range(B):
        table = c.table[b].long()
        place = lambda j: (int(table[j // 64]), slice(None), j % 64)
        c.cache.v_scales[place(0)] = 0
        c.v[b][0] = 0.0
        for j, shift in heavy:
            c.cache.v_scales[place(j)] += shift
            c.v[b][j] *= 2.0 ** shift
            c.cache.k_codes[place(j)] = c.cache.k_codes[place(0)] ^ 0x88
            c.cache.k_scales[place(j)] = c.cache.k_scales[place(0)] + 1
            c.k[b][j] = -2.0 * c.k[b][0]
        for j in range(lengths[b], -(-lengths[b] // 64) * 64):
            c.cache.v_scales[place(j)] = 255 if j % 2 else 250
        for h in range(H):
            k0 = c.k[b][0, h // group]
            q[b * rows:(b + 1) * rows, h] = (11.0 * D ** 0.5 / (k0 @ k0)) * k0
    q += 0.2 * rng.standard_normal(q.shape)
    x = torch.from_numpy(q).to(ac.TORCH[dtype])
    q = x.double().numpy()
    st = tc.status()
    out = attention.attend_tree(x.cuda(), c.cache, c.table, ac.i32(lengths), ac.i32([rows * b for b in range(B + 1)]),
                                ac.i32(sum(parents, [])), max_rows=rows, d_status=st)
    assert st.item() == abi.MOE_OK
    for b in range(B):
        r = slice(b * rows, (b + 1) * rows)
        o, z, spread, reach, seen = osp.attend_tree(q[r], c.k[b], c.v[b], parents[b], D ** -0.5)
        seen[:, [j for j, _ in heavy]] = False
        delta = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -21
        bound = ac.HALF_STEP[dtype] * np.abs(o) + 1.05 * (ac.HALF_STEP["fp16"] + 2 * delta + 2 * m * 2.0 ** -24)[..., None] * spread
        tiny = np.einsum("nm,mkd->nkd", seen.astype(float), np.abs(c.v[b]))
        bound += ac.HALF_TINY[dtype] + 2.0 ** -32 * np.repeat(tiny, group, axis=1)
        err = np.abs(ac.f64(out[r]) - o)
        assert (err <= bound).all(), f"{np.max(err / bound):.2f} of its bound"
