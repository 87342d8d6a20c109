"""The attention calls where inputs, offsets or statuses are out of the ordinary, against the 64-bit oracle or against
the same call without the odd part."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
from moe_expert_layer_top_gb300 import abi, attention

import attention_cases as ac

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_top_gb300.build as b
    b.build()
    abi.load()
    assert torch.cuda.is_available()


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def seeded(seed, *shape):
    return torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))


# ------------------------------------------------------------------ rows whose scores are not finite
# A NaN or +inf among a row's scores makes its out and lse NaN: lse = -inf is kept for rows without a weight.

POISON = [float("nan"), float("inf"), 2.0 ** 100]  # with keys of 2^100: a score past binary32


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("rows,keys", [(150, 150), (3, 5000)])  # in one pass; keys in parts
@pytest.mark.parametrize("poison", POISON[:2])
def test_prompt_lse_of_a_poisoned_query(D, dtype, rows, keys, poison):
    q, k, v = (x.to(ac.TORCH[dtype]) for x in (seeded(1, rows, 2, D), seeded(2, keys, 1, D).abs() + 0.5, seeded(3, keys, 1, D)))
    cu = ac.i32([0, rows]), ac.i32([0, keys])
    want, z = attention.attend_prompt(q, k, v, *cu, return_lse=True)
    q[1, 0, 3] = poison
    out, lse = attention.attend_prompt(q, k, v, *cu, return_lse=True)
    hit = torch.zeros(rows, 2, dtype=torch.bool, device="cuda")
    hit[1, 0] = True
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    assert torch.equal(lse[~hit], z[~hit]) and torch.equal(out[~hit], want[~hit])


@pytest.mark.parametrize("keys,at", [(300, 5), (300, 290), (5000, 4990), (5000, 3)])
@pytest.mark.parametrize("poison", POISON)
def test_prompt_lse_of_a_poisoned_key(keys, at, poison):
    """Rows that see the key, and rows that do not; in the first key tile and the last, in the first part and the last.
    The poisoned row's other scores are far above, so that the key's part has no weight beside the others'."""
    rows, D = 20, 128
    q, k, v = seeded(4, rows, 2, D).bfloat16(), seeded(5, keys, 1, D).bfloat16(), seeded(6, keys, 1, D).bfloat16()
    q[:, :, 0], k[:, :, 0] = 4.0, 0.0
    k[keys // 2, :, 0] = 900.0
    if poison == 2.0 ** 100:
        q[:, :, 0] = poison
        k[:, :, 0] = -poison  # the others overflow to -inf: no weight
    cu = ac.i32([0, rows]), ac.i32([0, keys])
    k[at, :, 0] = poison
    out, lse = attention.attend_prompt(q, k, v, *cu, return_lse=True)
    seen = torch.arange(rows, device="cuda") + keys - rows >= at
    assert seen.any()
    assert torch.isnan(lse[seen]).all() and torch.isnan(out[seen]).all()
    assert not torch.isnan(lse[~seen]).any() and not torch.isnan(out[~seen]).any()


@pytest.mark.parametrize("rows,keys", [(4, 100), (4, 5000)])
def test_prompt_scores_that_are_all_minus_infinity(rows, keys):
    """No key has a weight: out 0 and lse -inf, as without keys."""
    q, k, v = seeded(7, rows, 2, 64).bfloat16(), seeded(8, keys, 1, 64).bfloat16(), seeded(9, keys, 1, 64).bfloat16()
    k[:, :, 0] = -float("inf")
    q[:, :, 0] = torch.tensor([1.0, 2.0, 3.0, 4.0], device="cuda")[:, None]
    out, lse = attention.attend_prompt(q, k, v, ac.i32([0, rows]), ac.i32([0, keys]), return_lse=True)
    assert torch.isneginf(lse).all() and not out.any()


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("rows,length", [(1, 20), (4, 33), (6, 9000)])  # one block's, and joined from several
@pytest.mark.parametrize("poison", POISON[:2])
def test_paged_lse_of_a_poisoned_query(D, dtype, rows, length, poison):
    c = ac.Cache(np.random.default_rng(length), [length, 40], 1, D, 16)
    q = seeded(10, rows + 2, 4, D).to(ac.TORCH[dtype])
    cu, lens = ac.i32([0, rows, rows + 2]), ac.i32([length, 40])
    call = lambda: attention.attend_paged(q, c.cache, c.table, lens, cu, max_rows=rows, return_lse=True)
    want, z = call()
    q[rows - 1, 1] = poison  # the whole head: every score is NaN, or both signs of infinity are added
    out, lse = call()
    hit = torch.zeros(rows + 2, 4, dtype=torch.bool, device="cuda")
    hit[rows - 1, 1] = True
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    assert torch.equal(lse[~hit], z[~hit]) and torch.equal(out[~hit], want[~hit])
