"""Verification of drafted tokens and the commit of the accepted ones on the GPU, against the 64-bit oracle.

Tokens and rows are whole numbers: they have to be the oracle's wherever the given random numbers are not next to a
border. What "next to" means is what the header states: 2^-20 of the whole for the decisions (their two sides each have
an error of some binary32 roundings), 2^-34 for the new token.
"""
import numpy as np
import pytest
import torch

from moe_expert_layer_top_gb300 import abi, attention, speculative
from oracle import speculative as osp

import attention_cases as ac
import tree_cases as tc
from tree_cases import status

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DECISION, CHOICE = 2.0 ** -20, 2.0 ** -34


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_top_gb300.build as b
    b.build()
    abi.load()
    assert torch.cuda.is_available()


# ------------------------------------------------------------------ verification

def verify_case(seed, counts, V, dtype, kind, drafted, sharp=2.0, temperature=None, spare=0):
    """Inputs on the device and, in 64 bits, their exact values. The children of a row are drawn from the draft's
    probabilities, or are the likeliest tokens (one of them twice)."""
    rng = np.random.default_rng(seed)
    T, B = sum(counts), len(counts)
    logits = torch.from_numpy(sharp * rng.standard_normal((T + spare, V))).to(TYPES[dtype])
    exact = logits.double().numpy()
    trees = [tc.random_tree(rng, n, kind) for n in counts]
    cu = ac.offsets(counts)
    draft = None
    if drafted:
        d = exact + 0.7 * rng.standard_normal(exact.shape)
        d = np.exp(d - d.max(1, keepdims=True))
        draft = (d / d.sum(1, keepdims=True)).astype(np.float32)
    tokens = np.zeros(T + spare, dtype=np.int32)
    for b, parents in enumerate(trees):
        for i, p in enumerate(parents):
            if p < 0 or p >= i:
                continue
            row = cu[b] + p
            if drafted:
                tokens[cu[b] + i] = rng.choice(V, p=draft[row].astype(np.float64) / draft[row].astype(np.float64).sum())
            else:
                order = np.argsort(-exact[row], kind="stable")
                tokens[cu[b] + i] = order[rng.integers(0, min(V, 4))]
    state = {"counts": counts, "trees": trees, "cu": cu, "exact": exact, "draft": draft, "tokens": tokens,
             "accept_u": rng.random(T + spare).astype(np.float32), "sample_u": rng.random(B).astype(np.float32),
             "temperature": temperature}
    state["args"] = (logits.cuda(), ac.dev(tokens), ac.i32(cu), ac.dev(state["accept_u"]), ac.dev(state["sample_u"]))
    state["kw"] = {"parents": ac.i32(sum(trees, []) + [-1] * spare), "max_rows": max(counts + [1])}
    if drafted:
        state["kw"]["draft_probs"] = ac.dev(draft)
    if temperature is not None:
        state["kw"]["temperature"] = torch.tensor(temperature, dtype=torch.float32, device="cuda")
    return state


def check_verify(s, out):
    """Every sequence against the oracle; the number of those that were next to a border."""
    tokens, accepted, path = (out[x].cpu().numpy() for x in ("tokens", "accepted", "path"))
    close = 0
    for b, n in enumerate(s["counts"]):
        if n == 0:
            assert accepted[b] == 0 and (tokens[b] == -1).all() and (path[b] == -1).all()
            continue
        r = slice(s["cu"][b], s["cu"][b + 1])
        t = 1.0 if s["temperature"] is None else float(np.float32(s["temperature"][b]))
        want, new, near, edge = osp.verify(s["exact"][r], s["tokens"][r], s["trees"][b], s["accept_u"][r], s["sample_u"][b], t,
                                           None if s["draft"] is None else s["draft"][r])
        if near < DECISION or edge < CHOICE:
            close += 1
            continue
        k = len(want)
        assert accepted[b] == k - 1
        np.testing.assert_array_equal(path[b], want + [-1] * (path.shape[1] - k))
        said = [int(s["tokens"][r][i]) for i in want[1:]] + [new]
        np.testing.assert_array_equal(tokens[b], said + [-1] * (tokens.shape[1] - k))
    return close


@pytest.mark.parametrize("drafted", [False, True], ids=["alone", "behind_a_rejection"])
@pytest.mark.parametrize("V", [300, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_new_token_next_to_borders(dtype, V, drafted):
    """The random numbers lie next to borders between tokens, as close as their 24 bits allow, mostly 2^-26 to 2^-30 of the
    whole. What the sums are off by is about 2^-34: those closer than 2^-31 are moved on by a step."""
    B, rng = 96, np.random.default_rng(V + len(dtype))
    n = 2 if drafted else 1
    logits = torch.from_numpy(3.0 * rng.standard_normal((B * n, V))).to(TYPES[dtype])
    if drafted:
        logits[0::2, 0] = -40.0  # the child's token: sure to be rejected
    exact = logits.double().numpy()[::n]
    draft = rng.random((B * n, V)).astype(np.float32) ** 4
    draft[:, 0] = draft.sum(1)
    draft /= draft.sum(1, keepdims=True)
    temperature = rng.uniform(0.7, 1.3, B).astype(np.float32)
    u, want = np.zeros(B, dtype=np.float32), np.zeros(B, dtype=np.int32)
    for b in range(B):
        p = osp.softmax(exact[b], float(temperature[b]))
        left = np.maximum(p - draft[2 * b].astype(np.float64), 0) if drafted else p
        sums = np.cumsum(left) / left.sum()
        u[b] = np.float32(sums[np.argmin(np.abs(sums - rng.uniform(0.1, 0.9)))])
        while np.abs(sums - float(u[b])).min() < 2.0 ** -31:
            u[b] = np.nextafter(u[b], np.float32(1))
        want[b] = np.flatnonzero((sums > float(u[b])) & (left > 0))[0]
    st, dev = status(), lambda a: torch.from_numpy(a).cuda()
    got = speculative.verify_drafts(logits.cuda(), torch.zeros(B * n, dtype=torch.int32, device="cuda"),
                                    ac.i32([n * b for b in range(B + 1)]), torch.full((B * n,), 0.9, device="cuda"), dev(u),
                                    draft_probs=dev(draft) if drafted else None, temperature=dev(temperature), max_rows=n,
                                    d_status=st)
    assert st.item() == abi.MOE_OK and not got["accepted"].any()
    assert np.array_equal(got["tokens"][:, 0].cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 1000, 4099, 33333])
@pytest.mark.parametrize("kind", ["chain", "tree", "forest"])
def test_verify_matches_the_oracle(kind, V, drafted, dtype):
    s = verify_case(V, [6, 1, 9, 3, 0, 30, 4, 17], V, dtype, kind, drafted)
    st = status()
    out = speculative.verify_drafts(*s["args"], **s["kw"], d_status=st)
    assert st.item() == abi.MOE_OK
    assert check_verify(s, out) == 0


@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("counts", [[6], [64], [6] * 40, [256], [2] * 700])
def test_verify_sizes(counts, drafted):
    s = verify_case(len(counts) + counts[0], counts, 5003, "bf16", "tree", drafted, sharp=3.0)
    assert check_verify(s, speculative.verify_drafts(*s["args"], **s["kw"])) == 0


@pytest.mark.parametrize("drafted", [False, True])
def test_verify_a_large_vocabulary(drafted):
    """Every token can be told from its neighbours: 2^18 tokens of about equal probability."""
    s = verify_case(1, [3, 2, 4, 3, 2, 3], 262147, "fp32", "chain", drafted, sharp=0.3)
    assert check_verify(s, speculative.verify_drafts(*s["args"], **s["kw"])) == 0


def test_verify_the_choice_between_many_tokens():
    """512 sequences whose new token is one of 2^16, next to a few likely ones."""
    B, V = 512, 65536
    rng = np.random.default_rng(5)
    row = 2 * rng.standard_normal((2, V))
    row[:, rng.integers(0, V, 12)] += 9.0
    logits = torch.from_numpy(row).bfloat16()
    s = {"counts": [1] * B, "trees": [[-1]] * B, "cu": list(range(B + 1)), "draft": None, "temperature": [0.9] * B,
         "tokens": np.zeros(B, dtype=np.int32), "accept_u": np.zeros(B, dtype=np.float32),
         "sample_u": ((np.arange(B) + rng.random(B)) / B).astype(np.float32), "exact": logits.double().numpy()[np.arange(B) % 2]}
    out = speculative.verify_drafts(logits.cuda()[torch.arange(B) % 2], ac.dev(s["tokens"]), ac.i32(s["cu"]),
                                    ac.dev(s["accept_u"]), ac.dev(s["sample_u"]), max_rows=1,
                                    temperature=torch.full((B,), 0.9, device="cuda"))
    assert check_verify(s, out) <= 1


@pytest.mark.parametrize("drafted", [False, True])
def test_verify_temperatures(drafted):
    s = verify_case(11, [9] * 8, 3001, "bf16", "tree", drafted, temperature=[0.0, 1e-3, 0.3, 1.0, 2.5, 100.0, 0.0, 1e30])
    assert check_verify(s, speculative.verify_drafts(*s["args"], **s["kw"])) == 0


def test_verify_tiny_temperatures_take_the_largest():
    s = verify_case(12, [9] * 3, 501, "fp32", "tree", False, temperature=[1e-38, 2.0 ** -100, 1e-45])
    got = speculative.verify_drafts(*s["args"], **s["kw"])
    s["temperature"] = [0.0] * 3
    assert check_verify(s, got) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("drafted", [False, True])
def test_verify_strided_rows(dtype, drafted):
    """Rows of a wider matrix, every alignment of their beginnings."""
    s = verify_case(13, [6, 20], 1003, dtype, "tree", drafted)
    wide = torch.full((27, 1017), float("nan"), device="cuda", dtype=TYPES[dtype])
    for shift in (0, 1, 3, 8):
        x = wide[:26, shift:shift + 1003]
        x.copy_(s["args"][0])
        kw = dict(s["kw"])
        if drafted:
            kw["draft_probs"] = torch.full((26, 1019), 9.0, device="cuda")[:, shift:shift + 1003].copy_(s["kw"]["draft_probs"])
        assert check_verify(s, speculative.verify_drafts(x, *s["args"][1:], **kw)) == 0
        wide.fill_(float("nan"))


def test_verify_default_parents_are_chains():
    s = verify_case(14, [6, 1, 4], 997, "bf16", "chain", False)
    kw = dict(s["kw"])
    want = speculative.verify_drafts(*s["args"], **kw)
    del kw["parents"]
    got = speculative.verify_drafts(*s["args"], **kw)
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert check_verify(s, got) == 0


def test_verify_masked_vocabularies():
    """-inf among the logits: never chosen; a rejected token is not the new one; the only one left is taken with any number."""
    s = verify_case(15, [5] * 16, 600, "bf16", "tree", False)
    keep = np.zeros((80, 600), dtype=bool)
    rng = np.random.default_rng(2)
    for r in range(80):
        keep[r, rng.choice(600, rng.integers(1, 6), replace=False)] = True
    s["exact"][~keep] = -np.inf
    s["args"][0].masked_fill_(torch.from_numpy(~keep).cuda(), -float("inf"))
    for b in range(16):  # children: allowed tokens and others
        for i in range(1, 5):
            row = 5 * b + s["trees"][b][i]
            s["tokens"][5 * b + i] = rng.choice(np.flatnonzero(keep[row])) if rng.random() < 0.8 else rng.integers(0, 600)
    s["args"][1].copy_(ac.dev(s["tokens"]))
    assert check_verify(s, speculative.verify_drafts(*s["args"], **s["kw"])) == 0


@pytest.mark.parametrize("drafted", [False, True])
def test_verify_nothing_left_falls_back_to_the_target(drafted):
    """One token has all of p, and the draft too: a number of 1 rejects it, nothing is left, and it is the new token."""
    V = 300
    logits = torch.full((2, V), -float("inf"), device="cuda")
    logits[:, 77] = 3.0
    draft = torch.zeros(2, V, device="cuda")
    draft[:, 77] = 1.0
    out = speculative.verify_drafts(logits, ac.i32([0, 77]), ac.i32([0, 2]), torch.ones(2, device="cuda"),
                                    torch.zeros(1, device="cuda"), max_rows=2, draft_probs=draft if drafted else None)
    assert out["accepted"].item() == 0 and out["tokens"].tolist() == [[77, -1]] and out["path"].tolist() == [[0, -1]]


@pytest.mark.parametrize("poison", ["nan", "inf", "all"])
@pytest.mark.parametrize("greedy", [False, True])
def test_verify_rows_without_a_distribution(poison, greedy):
    s = verify_case(16, [4, 4, 4], 700, "fp32", "chain", False, sharp=0.0, temperature=[0.0 if greedy else 1.0] * 3)
    x = s["args"][0]
    s["tokens"][:] = 0
    s["args"][1].zero_()
    s["args"][3].zero_()  # u = 0 accepts whatever has a chance
    s["accept_u"][:] = 0.0
    if poison == "all":
        x[5] = -float("inf")
    else:
        x[5, 333] = float(poison)
    s["exact"] = x.double().cpu().numpy()
    out = speculative.verify_drafts(*s["args"], **s["kw"])
    assert out["accepted"].tolist() == [3, 1, 3]
    assert out["tokens"][1].tolist() == [0, -1, -1, -1] and out["path"][1].tolist() == [0, 1, -1, -1]
    assert check_verify(s, out) == 0


def test_verify_random_numbers_at_the_ends():
    V = 129
    logits = torch.zeros(1, V, device="cuda")
    logits[0, :3] = -float("inf")
    logits[0, -5:] = -float("inf")
    for u, want in ((0.0, 3), (1.0, V - 6), (7.0, V - 6), (-1.0, 3), (float("nan"), None)):
        out = speculative.verify_drafts(logits, ac.i32([0]), ac.i32([0, 1]), torch.zeros(1, device="cuda"),
                                        torch.tensor([u], device="cuda"), max_rows=1)
        token = out["tokens"].item()
        assert 3 <= token < V - 5 and (want is None or token == want)


def test_verify_reports_what_is_out_of_range():
    s = verify_case(17, [5, 6, 5], 200, "bf16", "chain", False)
    kw = s["kw"]
    good = speculative.verify_drafts(*s["args"], **kw)

    def others(out):  # the sequences beside the bad one have their results
        return all(torch.equal(out[k][[0, 2]], good[k][[0, 2]]) for k in good)

    def call(at, value, **more):
        args, st = list(s["args"]), status()
        if at is not None:
            args[at] = value
        out = speculative.verify_drafts(*args, **{**kw, **more}, d_status=st)
        assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
        return out

    token = s["args"][1].clone()
    token[6], token[0] = 200, -7  # a root's token is not looked at
    out = call(1, token)
    assert others(out) and out["accepted"][1] == 0
    token[6] = -1
    assert others(call(1, token))
    parents = kw["parents"].clone()
    parents[7] = 4
    assert others(call(None, None, parents=parents))
    t = torch.ones(3, device="cuda")
    for bad in (-1.0, float("nan"), float("inf")):
        t[1] = bad
        out = call(None, None, temperature=t)
        assert others(out) and torch.equal(out["tokens"], good["tokens"])  # counts as 1
    for cu in ([0, 5, 3, 8], [0, 5, 99, 16], [-1, 5, 11, 16]):
        out = call(2, ac.i32(cu))
        assert out["tokens"].shape == (3, 6)
    out = call(None, None, max_rows=5)
    assert others({k: torch.nn.functional.pad(v, (0, 1), value=-1) if v.dim() == 2 else v for k, v in out.items()})
    assert out["accepted"][1] == 0 and (out["tokens"][1] == -1).all() and (out["path"][1] == -1).all()


def test_verify_repeats_on_streams_and_in_graphs():
    states = [verify_case(20 + i, [6, 20, 1, 9], 50021, "bf16", "tree", bool(i)) for i in range(2)]
    want = [speculative.verify_drafts(*s["args"], **s["kw"]) for s in states]
    graphs, outs = [], []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(speculative.verify_drafts(*s["args"], **s["kw"]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for change in range(4):
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(o[k], w[k]) for k in w)
        for s in states:
            s["args"][3].uniform_()
            s["args"][4].uniform_()
        want = [speculative.verify_drafts(*s["args"], **s["kw"]) for s in states]
        for s in states:
            s["accept_u"], s["sample_u"] = s["args"][3].cpu().numpy(), s["args"][4].cpu().numpy()
        assert sum(check_verify(s, w) for s, w in zip(states, want)) == 0
    for s, w, stream in zip(states, want, streams):
        stream.wait_stream(torch.cuda.current_stream())
        got = speculative.verify_drafts(*s["args"], **s["kw"], stream=stream.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], w[k]) for k in w)


def test_verify_wrapper_refusals():
    s = verify_case(18, [3, 4], 100, "bf16", "chain", True)
    kw = s["kw"]
    for at, value in ((0, s["args"][0].cpu()), (0, s["args"][0].double()), (0, s["args"][0][0]), (0, s["args"][0].T),
                      (0, s["args"][0].clone().requires_grad_()), (1, s["args"][1].long()), (1, s["args"][1][:3]),
                      (2, s["args"][2][:1]), (3, s["args"][3][:2]), (3, s["args"][3].double()), (4, s["args"][4][:1])):
        args = list(s["args"])
        args[at] = value
        with pytest.raises(ValueError):
            speculative.verify_drafts(*args, **kw)
    for name, value in (("parents", kw["parents"].long()), ("draft_probs", kw["draft_probs"].bfloat16()),
                        ("draft_probs", kw["draft_probs"][:, :50]), ("draft_probs", kw["draft_probs"].T),
                        ("temperature", torch.ones(3, device="cuda")), ("max_rows", 0), ("max_rows", 257)):
        with pytest.raises(ValueError):
            speculative.verify_drafts(*s["args"], **{**kw, name: value})
    out = speculative.verify_drafts(s["args"][0][:0], s["args"][1][:0], ac.i32([0]), s["args"][3][:0], s["args"][4][:0],
                                    max_rows=4)
    assert out["tokens"].shape == (0, 4) and out["accepted"].shape == (0,)
    out = speculative.verify_drafts(s["args"][0][:0], s["args"][1][:0], ac.i32([0, 0]), s["args"][3][:0], s["args"][4][:1],
                                    max_rows=2)
    assert out["accepted"].tolist() == [0] and out["tokens"].tolist() == [[-1, -1]]


# ------------------------------------------------------------------ commit

PARTS = ("k_codes", "k_scales", "v_codes", "v_scales")


def commit_case(seed, seqs, paths, K, D, page, layers):
    """seqs: (rows, length) of each. Caches of random bytes; the pages of the sequences lie anywhere in them."""
    rng = np.random.default_rng(seed)
    need = [-(-m // page) for _, m in seqs]
    pages = sum(need) + 3
    order, at = rng.permutation(pages), 0
    table = np.full((len(seqs), max(need + [1])), -9, dtype=np.int32)
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    gen = torch.Generator("cuda").manual_seed(seed)
    caches = [attention.KVCacheMXFP4(*(torch.randint(0, 256, (pages, K, page, w), generator=gen, device="cuda").to(torch.uint8)
                                       for w in (D // 2, D // 32, D // 2, D // 32))) for _ in range(layers)]
    width = max(len(p) for p in paths)
    path = ac.i32([p + [-1] * (width - len(p)) for p in paths])
    args = (dev32(table), ac.i32([m for _, m in seqs]), ac.i32(ac.offsets([n for n, _ in seqs])), path,
            ac.i32([len(p) - 1 for p in paths]))
    return caches, args, table


def dev32(x):
    return ac.dev(np.asarray(x, dtype=np.int32))


def expected_commit(caches, seqs, paths, table, page):
    """The caches' bytes and the lengths after the commit."""
    lengths, want = [], []
    for c in caches:
        parts = {x: getattr(c, x).cpu().numpy() for x in PARTS}
        after = {x: p.copy() for x, p in parts.items()}
        for b, ((n, m), way) in enumerate(zip(seqs, paths)):
            for x in PARTS:
                rows = np.stack([parts[x][table[b, j // page], :, j % page] for j in range(m)]) if m else np.zeros((0, 1))
                if n:
                    rows, length = osp.commit(rows, m - n, way)
                    for j in range(m):
                        after[x][table[b, j // page], :, j % page] = rows[j]
        want.append(after)
    for (n, m), way in zip(seqs, paths):
        lengths.append(m - n + len(way) if n else m)
    return want, lengths


def same(caches, want):
    return all(np.array_equal(getattr(c, x).cpu().numpy(), w[x]) for c, w in zip(caches, want) for x in PARTS)


COMMITS = [
    # (rows, length) of each sequence, their paths, kv heads, D, page, layers
    ([(6, 40)], [[0, 2, 3, 5]], 2, 128, 16, 1),
    ([(1, 1)], [[0]], 1, 64, 16, 1),
    ([(8, 8), (3, 50), (0, 20), (5, 37), (1, 9)], [[0, 1, 2, 3], [0], [0], [0, 4], [0]], 3, 64, 16, 3),
    ([(16, 70)], [[0] + list(range(2, 16))], 8, 128, 64, 2),           # every row's place is read by the one before
    ([(256, 300), (200, 200)], [[0] + list(range(2, 256)), [0] + list(range(1, 200, 2))], 2, 64, 32, 5),
    ([(12, 500)] * 20, [[0, 3, 7, 11]] * 20, 8, 128, 64, 1),
    ([(9, 33), (9, 34)], [[0, 1, 5, 8], [0, 8]], 1, 128, 1024, 67),    # more layers than one launch takes
    ([(256, 600)], [[0] + list(range(2, 256))], 16, 128, 16, 2),       # more bytes than a block holds at once
]


@pytest.mark.parametrize("seqs,paths,K,D,page,layers", COMMITS, ids=[f"{len(c[0])}x{c[0][0][0]}_D{c[3]}_L{c[5]}" for c in COMMITS])
def test_commit_matches_the_oracle(seqs, paths, K, D, page, layers):
    caches, args, table = commit_case(len(seqs), seqs, paths, K, D, page, layers)
    want, lengths = expected_commit(caches, seqs, paths, table, page)
    version = [c.v_codes._version for c in caches]
    st = status()
    got = speculative.commit_drafts(caches if layers > 1 else caches[0], *args, d_status=st)
    assert st.item() == abi.MOE_OK
    assert got.tolist() == lengths and same(caches, want)
    assert all(c.v_codes._version > v for c, v in zip(caches, version))


def test_commit_random_paths():
    rng = np.random.default_rng(4)
    seqs = [(int(n), int(n + x)) for n, x in zip(rng.integers(1, 65, 50), rng.integers(0, 200, 50))]
    paths = [[0] + sorted(rng.choice(np.arange(1, n), rng.integers(0, n), replace=False).tolist()) if n > 1 else [0]
             for n, _ in seqs]
    caches, args, table = commit_case(9, seqs, paths, 4, 128, 32, 9)
    want, lengths = expected_commit(caches, seqs, paths, table, 32)
    assert speculative.commit_drafts(caches, *args).tolist() == lengths
    assert same(caches, want)


@pytest.mark.parametrize("change", ["start", "order", "same", "past", "negative", "accepted", "minus", "length", "short", "offset"])
def test_commit_leaves_what_is_out_of_range(change):
    seqs, paths = [(8, 40), (8, 60), (5, 20)], [[0, 3, 5], [0, 2, 4, 6], [0, 2]]
    caches, args, table = commit_case(3, seqs, paths, 2, 64, 16, 2)
    want, lengths = expected_commit(caches, seqs, [paths[0], [0], paths[2]], table, 16)
    lengths[1] = 60
    table_t, lens, cu, path, accepted = (t.clone() for t in args)
    if change == "start":
        path[1, 0] = 1
    if change == "order":
        path[1, 2] = 1
    if change == "same":
        path[1, 2] = 2
    if change == "past":
        path[1, 3] = 8
    if change == "negative":
        path[1, 1] = -3
    if change == "accepted":
        accepted[1] = 8
    if change == "minus":
        accepted[1] = -1
    if change == "length":
        lens[1] = 10 ** 6
        lengths[1] = 10 ** 6
    if change == "short":
        lens[1] = lengths[1] = 7
    st = status()
    if change == "offset":
        cu = ac.i32([0, 8, 7, 12])
        got = speculative.commit_drafts(caches, table_t, lens, cu, path, accepted, d_status=st)
        assert got.tolist()[:2] == lengths[:2]
    else:
        got = speculative.commit_drafts(caches, table_t, lens, cu, path, accepted, d_status=st)
        assert got.tolist() == lengths and same(caches, want)
    assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS


def test_commit_skips_pages_out_of_range():
    seqs, paths = [(20, 40), (4, 20)], [[0, 18, 19], [0, 2]]
    caches, args, table = commit_case(5, seqs, paths, 2, 128, 16, 2)
    want, lengths = expected_commit(caches, seqs, [[0], paths[1]], table, 16)
    lengths[0] = 23
    bad = args[0].clone()
    bad[0, 2] = 10 ** 6  # the page of the last rows
    st = status()
    got = speculative.commit_drafts(caches, bad, *args[1:], d_status=st)
    assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
    assert got.tolist() == lengths and same(caches, want)


def test_commit_offsets_past_32_bits():
    K, D, page, pages = 8, 128, 64, 90_000
    c = attention.KVCacheMXFP4.empty(pages, page, K, D)
    rows = torch.arange(page, device="cuda", dtype=torch.uint8)
    for x in PARTS:
        getattr(c, x)[pages - 2:] = rows[:, None]
    got = speculative.commit_drafts(c, ac.i32([[pages - 1, pages - 2]]), ac.i32([72]), ac.i32([0, 12]), ac.i32([[0, 5, 11]]),
                                    ac.i32([2]))
    assert got.tolist() == [63]
    for x in PARTS:
        t = getattr(c, x)
        assert (t[pages - 1, :, 61] == 1).all() and (t[pages - 1, :, 62] == 7).all()  # tokens 65 and 71
        assert (t[pages - 1, :, :61] == rows[:61, None]).all() and (t[pages - 2] == rows[:, None]).all()


def test_commit_in_graphs_and_on_streams():
    seqs, paths = [(8, 40), (8, 60)], [[0, 3, 5], [0, 2, 4, 6]]
    for seed, stream in ((6, None), (7, torch.cuda.Stream())):
        caches, args, table = commit_case(seed, seqs, paths, 2, 64, 16, 2)
        want, lengths = expected_commit(caches, seqs, paths, table, 16)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            got = speculative.commit_drafts(caches, *args, stream=stream)
        else:
            keep = [[getattr(c, x).clone() for x in PARTS] for c in caches]
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                got = speculative.commit_drafts(caches, *args)
            for _ in range(2):
                for c, k in zip(caches, keep):
                    for x, t in zip(PARTS, k):
                        getattr(c, x).copy_(t)
                g.replay()
        torch.cuda.synchronize()
        assert got.tolist() == lengths and same(caches, want)


def test_commit_wrapper_refusals():
    caches, args, _ = commit_case(8, [(4, 20)], [[0, 2]], 2, 64, 16, 2)
    other = attention.KVCacheMXFP4.empty(4, 32, 2, 64)
    with pytest.raises(abi.MoeError):
        speculative.commit_drafts([caches[0], other], *args)
    for bad in ([], [caches[0], caches[0]], [object()]):
        with pytest.raises((ValueError, AttributeError)):
            speculative.commit_drafts(bad, *args)
    with pytest.raises(TypeError):
        speculative.commit_drafts(None, *args)
    for at, value in ((0, args[0][0]), (0, args[0].long()), (1, args[1].long()), (1, args[1].cpu()), (2, args[2][:1]),
                      (3, args[3].cpu()), (3, args[3][0]), (4, args[4].long())):
        a = list(args)
        a[at] = value
        with pytest.raises(ValueError):
            speculative.commit_drafts(caches, *a)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("D,K,H,page", [(64, 2, 8, 16), (128, 1, 4, 64)])
def test_steps_with_trees_leave_the_cache_of_plain_steps(D, K, H, page):
    """Three steps of two sequences: append a tree, attend, verify, commit. The cache then is, byte for byte, what appending
    the accepted tokens one after another leaves, and the next step's attention reads it so."""
    V, layers, B, width = 400, 2, 2, 9
    gen = torch.Generator("cuda").manual_seed(D)
    rng = np.random.default_rng(D)
    rnd = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    wq, wk, wv = (rnd(V, n * D).bfloat16() for n in (H, K, K))  # a token's rows, the same wherever it stands
    rope = attention.rope_table(256, D)
    table = ac.i32(np.random.default_rng(1).permutation(2 * (96 // page + 1)).reshape(2, -1).tolist())
    trees, plain = ([attention.KVCacheMXFP4.empty(table.numel(), page, K, D) for _ in range(layers)] for _ in range(2))

    def append(cache, layer, tokens, seqs, positions, at):
        slots = table[seqs, at // page].long() * page + at % page
        rows = [w[tokens].view(-1, n, D) * (1 + layer) for w, n in ((wq, H), (wk, K), (wv, K))]
        return attention.qkv_append(*rows, positions=positions.int(), rope=rope, cache=cache, slots=slots)["q"]

    said = [[5], [17]]
    lengths = ac.i32([0, 0])
    st = status()
    for step in range(3):
        parents = [tc.random_tree(rng, n) for n in (width, width - 2)]
        depth = [osp.ancestors(p).sum(1) - 1 for p in parents]
        counts = [len(p) for p in parents]
        cu = ac.i32(ac.offsets(counts))
        par = ac.i32(sum(parents, []))
        draft = torch.softmax(0.3 * rnd(sum(counts), V), -1)  # near the target's, so that some are accepted
        drawn = torch.multinomial(draft, width, replacement=True, generator=gen)
        tokens = [[s[-1]] for s in said]
        for b in range(B):
            for i in range(1, counts[b]):
                tokens[b].append(int(drawn[int(cu[b]) + parents[b][i], i]))
        flat = ac.i32(sum(tokens, []))
        seqs = torch.arange(B, device="cuda").repeat_interleave(torch.tensor(counts, device="cuda"))
        place = torch.cat([torch.arange(n, device="cuda") for n in counts])
        deep = torch.tensor(np.concatenate(depth), device="cuda")
        full = lengths + ac.i32(counts)
        x = 0
        for layer in range(layers):
            q = append(trees[layer], layer, flat.long(), seqs, lengths[seqs] + deep, lengths[seqs].long() + place)
            x = x + attention.attend_tree(q, trees[layer], table, full, cu, par, max_rows=width, d_status=st).float()
        logits = x.flatten(1) @ rnd(H * D, V) * 0.005
        out = speculative.verify_drafts(logits, flat, cu, torch.rand(sum(counts), generator=gen, device="cuda"),
                                        torch.rand(B, generator=gen, device="cuda"), parents=par, draft_probs=draft,
                                        max_rows=width, d_status=st)
        new = speculative.commit_drafts(trees, table, full, cu, out["path"], out["accepted"], d_status=st)
        assert st.item() == abi.MOE_OK
        for b in range(B):
            k = int(out["accepted"][b])
            assert int(new[b]) == int(lengths[b]) + 1 + k
            settled = [said[b][-1]] + out["tokens"][b, :k].tolist()
            at = torch.arange(int(lengths[b]), int(new[b]), device="cuda")
            for layer in range(layers):
                append(plain[layer], layer, torch.tensor(settled, device="cuda"), torch.full_like(at, b), at, at)
            said[b] += out["tokens"][b, :k + 1].tolist()
        lengths = new
        for a, c in zip(trees, plain):
            for b in range(B):
                at = torch.arange(int(lengths[b]), device="cuda")
                for part in PARTS:
                    assert torch.equal(getattr(a, part)[table[b, at // page].long(), :, at % page],
                                       getattr(c, part)[table[b, at // page].long(), :, at % page])
    assert max(lengths.tolist()) > 3  # something was accepted
