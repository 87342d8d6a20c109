"""Verification of drafted tokens where a step could go wrong in a few calls of a million: random numbers on the borders
of the decisions, and residuals that lie in a few places of the vocabulary.

On the border of a decision either answer is right, but all threads of the cluster have to give the same: what they write
then fits one walk."""
import numpy as np
import pytest
import torch

from moe_expert_layer_top_gb300 import abi, speculative
from oracle import speculative as osp

import attention_cases as ac
from tree_cases import status

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CHOICE = 2.0 ** -34


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_top_gb300.build as b
    b.build()
    abi.load()
    assert torch.cuda.is_available()


def chains(rng, B, n, V, dtype, drafted):
    """B chains of n rows; the children are likely tokens. Logits on the device, in 64 bits, the draft, the tokens."""
    logits = torch.from_numpy(2.0 * rng.standard_normal((B * n, V))).to(TYPES[dtype])
    for r in range(B * n):  # a few tokens hold much of the row
        logits[r, torch.from_numpy(rng.choice(V, 5, replace=False))] += 9.0
    exact = logits.double().numpy()
    draft = None
    if drafted:
        d = exact + 0.5 * rng.standard_normal(exact.shape)
        d = np.exp(d - d.max(1, keepdims=True))
        draft = (d / d.sum(1, keepdims=True)).astype(np.float32)
    tokens = np.zeros(B * n, np.int32)
    for r in range(B * n):
        if r % n:
            tokens[r] = np.argsort(-exact[r - 1])[rng.integers(0, 4)]
    return logits, exact, draft, tokens


# sequences: clusters of 16, 8, 4 and 1 blocks
@pytest.mark.parametrize("B", [3, 24, 96, 400])
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_one_walk_whatever_the_border_decides(dtype, drafted, B):
    rng = np.random.default_rng(B + drafted)
    n, V = (6, 33001) if B < 300 else (4, 5000)
    logits, exact, draft, tokens = chains(rng, B, n, V, dtype, drafted)
    device = [logits.cuda(), ac.dev(tokens), ac.i32([n * b for b in range(B + 1)])]
    chance = np.zeros(B * n)
    for r in range(B * n):
        if r % n:
            chance[r] = osp.accept_chance(osp.softmax(exact[r - 1], 1.0), None if draft is None else draft[r - 1].astype(np.float64),
                                          [], tokens[r])
    sample = rng.random(B).astype(np.float32)
    kw = {"draft_probs": ac.dev(draft)} if drafted else {}
    ways = np.zeros(n, int)
    wants = {}  # the new token of (sequence, accepted), and how near it is to a border
    for trial in range(12):
        u = chance.astype(np.float32)
        for _ in range(trial // 2):  # 0 to 5 steps above and below
            u = np.nextafter(u, np.float32(0 if trial % 2 else 1))
        sure = rng.random(B * n) < 0.5  # half of them are surely accepted, so that the walk gets further
        u = np.where(sure & (chance > 1e-3), np.float32(0.0), u).astype(np.float32)
        st = status()
        args = (*device, ac.dev(u), ac.dev(sample))
        out = speculative.verify_drafts(*args, **kw, max_rows=n, d_status=st)
        again = speculative.verify_drafts(*args, **kw, max_rows=n)
        assert st.item() == abi.MOE_OK and all(torch.equal(out[k], again[k]) for k in out)
        said, accepted, path = (out[k].cpu().numpy() for k in ("tokens", "accepted", "path"))
        for b in range(B):
            a = int(accepted[b])
            ways[a] += 1
            r0 = n * b
            for i in range(1, n):  # what is far from its border is decided
                if abs(float(u[r0 + i]) - chance[r0 + i]) > 2.0 ** -20 and i <= a + 1:
                    assert (u[r0 + i] < chance[r0 + i]) == (i <= a)
            assert path[b].tolist() == list(range(a + 1)) + [-1] * (n - 1 - a)
            assert said[b, :a].tolist() == tokens[r0 + 1:r0 + 1 + a].tolist() and (said[b, a + 1:] == -1).all()
            if (b, a) not in wants:
                row = r0 + a
                rejected = [tokens[row + 1]] if a < n - 1 else []
                p = osp.softmax(exact[row], 1.0)
                left = osp.residual(p, None if draft is None else draft[row].astype(np.float64), rejected)
                whole = left.sum()
                sums = np.cumsum(left) / whole
                edge = np.abs(sums - float(sample[b])).min() * whole  # as a part of p's whole
                wants[b, a] = int(np.flatnonzero((sums > sample[b]) & (left > 0))[0]), edge
            token, edge = wants[b, a]
            assert edge < CHOICE or said[b, a] == token
    assert B < 24 or (ways > 0).all()


@pytest.mark.parametrize("B, V", [(190, 4096), (97, 8200), (40, 16400), (14, 32800)])
def test_short_rows_of_more_clusters_than_fit(B, V):
    """Blocks whose part of a row is done at once, and clusters that begin behind others: the first values that blocks give
    one another must not come before their receiver has begun. Calls one behind another, all with the same result."""
    rng = np.random.default_rng(V)
    logits, exact, _, tokens = chains(rng, B, 2, V, "bf16", False)
    u, sample = rng.random(2 * B).astype(np.float32), rng.random(B).astype(np.float32)
    args = (logits.cuda(), ac.dev(tokens), ac.i32([2 * b for b in range(B + 1)]), ac.dev(u), ac.dev(sample))
    outs = [speculative.verify_drafts(*args, max_rows=2) for _ in range(60)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], outs[0][k]) for o in outs for k in o)
    said, accepted = outs[0]["tokens"].cpu().numpy(), outs[0]["accepted"].cpu().numpy()
    for b in range(B):
        r = slice(2 * b, 2 * b + 2)
        path, token, near, edge = osp.verify(exact[r], tokens[r], [-1, 0], u[r], sample[b])
        assert near < 2.0 ** -20 or accepted[b] == len(path) - 1
        assert near < 2.0 ** -20 or edge < CHOICE or said[b, accepted[b]] == token


# sequences: clusters of 16 and of 4 blocks
@pytest.mark.parametrize("B", [3, 96])
@pytest.mark.parametrize("moved", [0.05, 2.0 ** -10])
@pytest.mark.parametrize("end", ["front", "back"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_residual_in_one_end_of_the_vocabulary(dtype, end, moved, B):
    """The draft is the target's own distribution but for a part of it that lies in the other end: what is left of nearly
    all tokens is next to nothing, and an error in c or a rounding of their weights, added up, would move every border.

    The sums have an error of about 2^-34 of p's whole: random numbers closer than 2^-32 of it to a border do not count."""
    V, rng = 33001, np.random.default_rng(B)
    logits = torch.from_numpy(2.0 * rng.standard_normal((2 * B, V))).to(TYPES[dtype])
    exact = logits.double().numpy()
    draft = np.zeros((2 * B, V), np.float32)
    sample, want = np.zeros(B, np.float32), np.zeros(B, np.int32)
    tokens = np.zeros(2 * B, np.int32)
    few = V // 16
    for b in range(B):
        p = osp.softmax(exact[2 * b], 1.0)
        less, more = (slice(0, few), slice(V - few, V)) if end == "front" else (slice(V - few, V), slice(0, few))
        q = p.copy()
        part = min(moved, 0.9 * p[less].sum())
        q[less] *= 1 - part / p[less].sum()
        q[more] *= 1 + part / p[more].sum()
        draft[2 * b] = q.astype(np.float32)
        tokens[2 * b + 1] = more.start + int(np.argmax(p[more]))  # rejected by a number of 1
        left = np.maximum(p - draft[2 * b].astype(np.float64), 0.0)
        N = left.sum()
        sums = np.cumsum(left) / N
        sample[b] = np.float32(sums[np.argmin(np.abs(sums - rng.uniform(0.05, 0.95)))])
        while np.abs(sums - float(sample[b])).min() * N < 2.0 ** -32:
            sample[b] = np.nextafter(sample[b], np.float32(1))
        want[b] = np.flatnonzero((sums > float(sample[b])) & (left > 0))[0]
    st = status()
    out = speculative.verify_drafts(logits.cuda(), ac.dev(tokens), ac.i32([2 * b for b in range(B + 1)]),
                                    torch.ones(2 * B, device="cuda"), ac.dev(sample), draft_probs=ac.dev(draft), max_rows=2,
                                    d_status=st)
    assert st.item() == abi.MOE_OK and not out["accepted"].any()
    assert np.array_equal(out["tokens"][:, 0].cpu().numpy(), want)


@pytest.mark.parametrize("B", [3, 96])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["rounded", "softmax", "exact"])
def test_draft_equal_to_the_target(kind, dtype, B):
    """What is left behind a rejection is the draft's rounding, or nothing: 2^-26 of the whole where each probability is
    rounded, about 2^-22 where they come of a softmax in binary32, 0 where they are p to the last bit. Every sequence gets a
    token, the formula's where the random number is not next to a border."""
    V, rng = 33001, np.random.default_rng(B)
    if kind == "exact":  # powers of two, so that p is exact in binary32
        x = np.full((2 * B, V), -np.inf)
        for r in range(2 * B):
            x[r, rng.choice(V, 5, replace=False)] = np.log(np.array([8, 4, 2, 1, 1.0]))
        logits = torch.from_numpy(np.where(np.isneginf(x), -np.inf, np.round(x / np.log(2)))).to(TYPES[dtype])
        t = float(np.float32(1 / np.log(2)))
    else:
        logits, t = torch.from_numpy(2.0 * rng.standard_normal((2 * B, V))).to(TYPES[dtype]), 1.0
    exact = logits.double().numpy()
    if kind == "softmax":
        draft = torch.softmax(logits.float(), -1).numpy()
    else:
        draft = np.stack([osp.softmax(e, t) for e in exact]).astype(np.float32)
    sample = rng.random(B).astype(np.float32)
    tokens = np.zeros(2 * B, np.int32)
    tokens[1::2] = exact[::2].argmax(1)
    lo, u, temp = logits.cuda(), torch.ones(2 * B, device="cuda"), torch.full((B,), t, device="cuda")
    out = [torch.full((B, 2), -77, dtype=torch.int32, device="cuda") for _ in range(2)]
    accepted, st = torch.full((B,), -77, dtype=torch.int32, device="cuda"), status()
    held = (lo, ac.dev(draft), ac.dev(tokens), ac.i32([2 * b for b in range(B + 1)]), temp, u, ac.dev(sample))
    io = abi.MoeVerifyDraftsIO(held[0].data_ptr(), V, held[1].data_ptr(), V, held[2].data_ptr(), None, held[3].data_ptr(),
                               held[4].data_ptr(), held[5].data_ptr(), held[6].data_ptr(), out[0].data_ptr(), out[1].data_ptr(),
                               accepted.data_ptr(), B, 2 * B, 2, V, {"bf16": abi.MOE_DTYPE_BF16, "fp32": abi.MOE_DTYPE_F32}[dtype], 0)
    assert abi.moe_verify_drafts(io, st, torch.cuda.current_stream()) == abi.MOE_OK
    torch.cuda.synchronize()
    assert st.item() == abi.MOE_OK
    said = out[0].cpu().numpy()
    assert ((said[:, 0] >= 0) & (said[:, 0] < V)).all() and not (said == -77).any() and not (out[1] == -77).any()
    away = 0
    for b in range(B):
        p = osp.softmax(exact[2 * b], t)
        assert p[said[b, 0]] > 0
        path, token, near, edge = osp.verify(exact[2 * b:2 * b + 2], tokens[2 * b:2 * b + 2], [-1, 0], [1.0, 1.0], sample[b], t,
                                             draft[2 * b:2 * b + 2])
        if accepted[b]:  # the child's own rounding is above its p: accepted as surely as the number is 1
            assert near < 2.0 ** -20
            continue
        N = np.maximum(p - draft[2 * b].astype(np.float64), 0).sum()
        nothing = N < 2.0 ** -31
        if nothing:  # by the formula a residue of the 64-bit softmax; for the call nothing: p's own choice
            sums = np.cumsum(p)
            token, edge = int(np.flatnonzero(sums > sample[b])[0]), np.abs(sums - float(sample[b])).min()
        elif N < 2.0 ** -29:
            continue
        if edge * (1.0 if nothing else N) > 2.0 ** -32:
            away += 1
            assert said[b, 0] == token
    assert away > 0 or kind == "rounded"


def nodes(parents_of, B):
    """cu_rows and parents of B equal trees."""
    n = len(parents_of)
    return ac.i32([n * b for b in range(B + 1)]), ac.i32(list(parents_of) * B)


@pytest.mark.parametrize("heavy", [[0.999], [1 - 2.0 ** -16], [0.4, 0.5, 0.09], [0.6, 0.3999, 0.0000999]])
@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_chances_behind_rejected_likely_children(dtype, heavy):
    """Children that hold nearly all of the row are rejected; the others' chances are p over the little that is left. Their
    random numbers lie 2^-18 of the chance beside it, four times the error that the decisions may have."""
    B, V, rng = 32, 9001, np.random.default_rng(len(heavy))
    h, n = len(heavy), len(heavy) + 4
    logits = rng.standard_normal((B * n, V))
    tokens, u, want = np.zeros(B * n, np.int32), np.ones(B * n, np.float32), np.zeros(B, int)
    exact = np.zeros((B, V))
    for b in range(B):
        own = rng.choice(V, h + 3, replace=False)
        w = np.exp(logits[n * b])
        w[own[:h]] = 0
        w[own[h:]] *= 50  # so that their chances are some percent
        w *= (1 - sum(heavy)) / w.sum()
        w[own[:h]] = heavy
        logits[n * b] = np.log(w)
        tokens[n * b + 1:n * b + 4 + h] = own
        if b % 3 == 0:
            tokens[n * b + h] = own[0] if h > 1 else own[h - 1]  # one of the heavy twice, another one left
    held = torch.from_numpy(logits).to(TYPES[dtype])
    for b in range(B):
        p = osp.softmax(held[n * b].double().numpy(), 1.0)
        gone = list(tokens[n * b + 1:n * b + 1 + h])
        good = int(rng.integers(0, 4))  # which of the others is accepted; 3: none
        for j in range(3):
            child = n * b + 1 + h + j
            chance = osp.accept_chance(p, None, gone, tokens[child])
            u[child] = np.float32(chance * (1 - 2.0 ** -18 if j == good else 1 + 2.0 ** -18))
            gone.append(tokens[child])
        want[b] = good
    cu, parents = nodes([-1] + [0] * (n - 1), B)
    out = speculative.verify_drafts(held.cuda(), ac.dev(tokens), cu, ac.dev(u), torch.full((B,), 0.5, device="cuda"),
                                    parents=parents, max_rows=n)
    for b in range(B):
        assert out["path"][b, :2].tolist() == ([0, -1] if want[b] == 3 else [0, 1 + h + want[b]]), b


@pytest.mark.parametrize("noise", [0.01, 0.001])
@pytest.mark.parametrize("B", [3, 40])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_chances_behind_a_draft_close_to_the_target(dtype, B, noise):
    """N is 2^-8 and 2^-11 of p, and a child's chance what is left of its p over what is left in all."""
    V, rng = 33001, np.random.default_rng(B)
    n = 4
    logits = torch.from_numpy(2.0 * rng.standard_normal((B * n, V))).to(TYPES[dtype])
    exact = logits.double().numpy()
    draft = np.zeros((B * n, V), np.float32)
    tokens, u, want = np.zeros(B * n, np.int32), np.ones(B * n, np.float32), np.zeros(B, int)
    for b in range(B):
        p = osp.softmax(exact[n * b], 1.0)
        q = p * np.exp(noise * rng.standard_normal(V))
        draft[n * b] = (q / q.sum()).astype(np.float32)
        q = draft[n * b].astype(np.float64)
        gone = [int(np.argmax(np.where(q > p, p, 0)))]  # surely rejected by a number of 1
        tokens[n * b + 1] = gone[0]
        good = int(rng.integers(0, 3))
        for j in range(2):
            left = osp.residual(p, q, gone)
            ratio = left / left.sum() / q
            some = np.flatnonzero((ratio > 0.2) & (ratio < 0.8))
            y = int(some[rng.integers(0, len(some))])
            child = n * b + 2 + j
            tokens[child] = y
            u[child] = np.float32(ratio[y] * (1 - 2.0 ** -18 if j == good else 1 + 2.0 ** -18))
            gone.append(y)
        want[b] = good
    cu, parents = nodes([-1, 0, 0, 0], B)
    out = speculative.verify_drafts(logits.cuda(), ac.dev(tokens), cu, ac.dev(u), torch.full((B,), 0.5, device="cuda"),
                                    parents=parents, draft_probs=ac.dev(draft), max_rows=n)
    for b in range(B):
        assert out["path"][b, :2].tolist() == ([0, -1] if want[b] == 2 else [0, 2 + want[b]]), b


def test_rejected_tokens_that_were_all_there_was():
    """Three tokens allowed, all of them rejected, then children without a chance: the new token is one of the three."""
    V, n = 5000, 200
    logits = torch.full((n, V), -float("inf"), device="cuda")
    logits[:, [10, 20, 4999]] = torch.tensor([1.0, 2.0, 3.0], device="cuda")
    tokens = ac.i32([0, 10, 20, 4999] + list(range(100, 100 + n - 4)))
    u = torch.zeros(n, device="cuda")
    u[:4] = 1.0
    out = speculative.verify_drafts(logits, tokens, ac.i32([0, n]), u, torch.tensor([0.2], device="cuda"),
                                    parents=ac.i32([-1] + [0] * (n - 1)), max_rows=n)
    assert out["accepted"].item() == 0 and out["tokens"][0, :2].tolist() == [20, -1]


@pytest.mark.parametrize("t", [2.0 ** 100, 1e37, 3e38])
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("V", [129, 5000])
def test_large_temperatures_make_all_allowed_tokens_alike(V, drafted, t):
    """Also beside logits of -inf, and in a row whose last unit is cut."""
    rng = np.random.default_rng(V)
    B = 40
    logits = torch.from_numpy(rng.standard_normal((2 * B, V))).float()
    out_of = torch.from_numpy(rng.random((2 * B, V)) < 0.3)
    out_of[:, 0] = False
    logits[out_of] = -float("inf")
    exact = logits.double().numpy()
    draft = np.zeros((2 * B, V), np.float32)
    draft[:, 0] = 0.75
    draft[:, 1:] = 0.25 / (V - 1)
    u, sample, tokens = rng.random(2 * B).astype(np.float32), rng.random(B).astype(np.float32), np.zeros(2 * B, np.int32)
    u[1::4] = 1.0  # every second child is surely rejected
    out = speculative.verify_drafts(logits.cuda(), ac.dev(tokens), ac.i32([2 * b for b in range(B + 1)]), ac.dev(u),
                                    ac.dev(sample), draft_probs=ac.dev(draft) if drafted else None,
                                    temperature=torch.full((B,), t, device="cuda"), max_rows=2)
    checked = 0
    for b in range(B):
        r = slice(2 * b, 2 * b + 2)
        path, token, near, edge = osp.verify(exact[r], tokens[r], [-1, 0], u[r], sample[b], float(np.float32(t)),
                                             draft[r] if drafted else None)
        if near > 2.0 ** -20 and edge > 2.0 ** -24:  # equal weights: the borders are multiples of one
            checked += 1
            assert out["tokens"][b].tolist() == ([0, token] if len(path) == 2 else [token, -1])
    assert checked > B // 2
