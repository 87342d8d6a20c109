"""Cases and plain forms of the operators of a speculative step with trees of drafted tokens.

Three operators, in the order in which a serving program calls them once the drafted rows are in the cache:

* tree: attention of a tree of drafted tokens over the paged MXFP4 cache (``attention.attend_tree``);
* verify: the drafted tokens against the target's probabilities, from given random numbers
  (``speculative.verify_drafts``);
* commit: the accepted tokens' keys and values moved together in the caches of all layers
  (``speculative.commit_drafts``).

``run`` computes a case in elementary torch operations, or, with ``own`` set, through the library's entry points.
``exact`` computes it in 64 bits, written separately.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 32


# ---------------------------------------------------------------- cases

def listed():
    heads = {"heads": 32, "kv_heads": 8, "dim": 128}
    return [
        # a small tree of one sequence: the latency of a layer
        {"name": "tree_bs1_16", "op": "tree", "dtype": "bf16", **heads, "seqs": 1, "rows_min": 16, "rows_max": 16,
         "len_min": 4096, "len_max": 4096, "page": 64, "lens_seed": 1},
        # a wide tree of one sequence with a long context
        {"name": "tree_bs1_64_long", "op": "tree", "dtype": "bf16", **heads, "seqs": 1, "rows_min": 64, "rows_max": 64,
         "len_min": 131071, "len_max": 131071, "page": 64, "lens_seed": 2},
        # trees as small as the six rows of a verify step, 64 sequences of 1K to 5K tokens
        {"name": "tree_bs64_6", "op": "tree", "dtype": "bf16", **heads, "seqs": 64, "rows_min": 6, "rows_max": 6,
         "len_min": 1024, "len_max": 5120, "page": 64, "lens_seed": 3},
        # half-width heads, eight query heads to a kv head, small pages, trees and contexts of very different sizes
        {"name": "tree_ragged_d64", "op": "tree", "dtype": "fp16", "heads": 64, "kv_heads": 8, "dim": 64, "seqs": 24,
         "rows_min": 1, "rows_max": 61, "len_min": 70, "len_max": 9000, "page": 16, "lens_seed": 4},
        # wide trees of a batch with long contexts: the tensor cores' work
        {"name": "tree_bs16_64", "op": "tree", "dtype": "bf16", **heads, "seqs": 16, "rows_min": 64, "rows_max": 64,
         "len_min": 8000, "len_max": 32000, "page": 64, "lens_seed": 5},
        # the chain of one sequence's verify step, drafted without chance
        {"name": "verify_chain_bs1", "op": "verify", "dtype": "bf16", "vocab": 131072, "seqs": 1, "rows_min": 6,
         "rows_max": 6, "chain": True, "draft": False, "greedy": 0.0, "lens_seed": 6},
        # 64 sequences' verify steps with the draft's probabilities
        {"name": "verify_chain_bs64_drafted", "op": "verify", "dtype": "fp32", "vocab": 131072, "seqs": 64, "rows_min": 6,
         "rows_max": 6, "chain": True, "draft": True, "greedy": 0.0, "lens_seed": 7},
        # wide trees, each node with the likeliest tokens as its children, some sequences greedy
        {"name": "verify_tree_bs16", "op": "verify", "dtype": "bf16", "vocab": 131072, "seqs": 16, "rows_min": 64,
         "rows_max": 64, "chain": False, "draft": False, "greedy": 0.25, "lens_seed": 8},
        # small trees drawn from the draft's probabilities, several children to a node, an odd vocabulary
        {"name": "verify_tree_ragged_drafted", "op": "verify", "dtype": "fp16", "vocab": 50021, "seqs": 24, "rows_min": 1,
         "rows_max": 16, "chain": False, "draft": True, "greedy": 0.1, "lens_seed": 9},
        # one sequence, one layer
        {"name": "commit_bs1", "op": "commit", "kv_heads": 8, "dim": 128, "layers": 1, "seqs": 1, "rows_min": 16,
         "rows_max": 16, "len_min": 4096, "len_max": 4096, "page": 64, "lens_seed": 10},
        # a batch, the caches of all layers of a model at once
        {"name": "commit_bs64_32_layers", "op": "commit", "kv_heads": 8, "dim": 128, "layers": 32, "seqs": 64,
         "rows_min": 64, "rows_max": 64, "len_min": 80, "len_max": 400, "page": 64, "lens_seed": 11},
        # ragged trees, half-width heads, small pages
        {"name": "commit_ragged_d64", "op": "commit", "kv_heads": 8, "dim": 64, "layers": 12, "seqs": 24, "rows_min": 1,
         "rows_max": 61, "len_min": 70, "len_max": 900, "page": 16, "lens_seed": 12},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "verify", "commit"])
    lens_seed = rng.randrange(1 << 20)
    rows = _log_uniform(rng, 1, 128)
    rows_min = rng.choice([rows, max(1, rows // 3), 1])
    if op == "verify":
        vocab = _log_uniform(rng, 1000, 131072)
        seqs = max(1, min(_log_uniform(rng, 1, 64), 60_000_000 // (vocab * rows)))
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "vocab": vocab, "seqs": seqs,
                "rows_min": rows_min, "rows_max": rows, "chain": rng.random() < 0.4, "draft": rng.random() < 0.5,
                "greedy": rng.choice([0.0, 0.0, 0.3]), "lens_seed": lens_seed}
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "commit":
        longest = rows + _log_uniform(rng, 1, 500)
        seqs = _log_uniform(rng, 1, 64)
        layers = max(1, min(_log_uniform(rng, 1, 32), 64 * 32 * 400 // (seqs * longest)))
        return {"op": op, "kv_heads": kv_heads, "dim": dim, "layers": layers, "seqs": seqs, "rows_min": rows_min,
                "rows_max": rows, "len_min": rows + (longest - rows) // rng.choice([1, 4]), "len_max": longest,
                "page": page, "lens_seed": lens_seed}
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    longest = rows + _log_uniform(rng, 1, 100000)
    # scores of all rows, heads and keys, no more of them than the largest listed case has, and 400,000 cached tokens
    seqs = max(1, min(_log_uniform(rng, 1, 64), 130_000_000 * 4 // (heads * rows * longest), 400_000 // longest))
    if heads * rows * longest > 520_000_000:
        longest = rows + 520_000_000 // (heads * rows)
    return {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "seqs": seqs, "rows_min": rows_min, "rows_max": rows,
            "len_min": rows + (longest - rows) // rng.choice([1, 3, 40]), "len_max": longest, "page": page,
            "lens_seed": lens_seed}


def _lens(case):
    """Rows of every sequence's tree, and its tokens in the cache with these among them."""
    rng = random.Random(case["lens_seed"])
    rows, keys = [], []
    for _ in range(case["seqs"]):
        rows.append(rng.randint(case["rows_min"], case["rows_max"]))
        keys.append(_log_uniform(rng, case["len_min"], case["len_max"]) if "len_min" in case else 0)
    return rows, keys


def _parents(case, rows, rng):
    """The parent of every row, by its place in its sequence; the first row is the root."""
    if case.get("chain"):
        return [[i - 1 for i in range(n)] for n in rows]
    trees = []
    for n in rows:
        branch = rng.choice([2, 3, 4, 8])
        # breadth first, uneven: rows lie behind their parents, and a node's children next to one another
        parents = [-1]
        while len(parents) < n:
            low = parents[-1] if len(parents) > 1 else 0
            parents.append(min(len(parents) - 1, max(low, (len(parents) - 1) // branch) + (rng.random() < 0.15)))
        trees.append(parents)
    return trees


def _depth(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _tree_rng(case):
    return random.Random(case["lens_seed"] + 1000003)


def work(case):
    rows, keys = _lens(case)
    T = sum(rows)
    if case["op"] == "verify":
        # the least: the logits behind every sequence's first row, and with a draft also those behind the child that
        # was accepted, or the draft's probabilities that a rejection takes off; and the small arrays
        size = 4 if case["dtype"] == "fp32" else 2
        values = case["vocab"] * sum(2 if case["draft"] and n > 1 else 1 for n in rows)
        return {"bytes": values * size + T * 12 + len(rows) * 24, "flops": 3 * values}
    token = 2 * (case["dim"] // 2 + case["dim"] // GROUP)  # bytes of one token and kv head in a cache
    if case["op"] == "commit":
        paths = _paths(case, rows, _tree_rng(case))
        moves = sum(sum(j != i for j, i in enumerate(p)) for p in paths)
        return {"bytes": 2 * moves * case["layers"] * case["kv_heads"] * token + 16 * len(rows) + 4 * T, "flops": 0}
    H, D = case["heads"], case["dim"]
    depths = [_depth(p) for p in _parents(case, rows, _tree_rng(case))]
    pairs = sum(n * (m - n) + sum(d) + n for n, m, d in zip(rows, keys, depths))
    return {"bytes": sum(keys) * case["kv_heads"] * token + 4 * T * H * D + 4 * T * H, "flops": 4 * D * H * pairs}


def _paths(case, rows, rng):
    """The rows of an accepted path for every sequence. A row that moves comes from behind all the places that are
    moved to, so that a pass over the same caches again finds what the first one found."""
    paths = []
    for n in rows:
        accepted = min(rng.choice([0, 1, 2, 2, 3, 3, 4, 5, 6]), n - 1)
        same = rng.randint(0, accepted)  # the first rows of the path are in place already
        free = list(range(accepted + 1, n))
        moved = sorted(rng.sample(free, min(accepted - same, len(free))))
        paths.append(list(range(same + 1)) + moved)
    return paths


# ---------------------------------------------------------------- inputs

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return _ints(out)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, keys = _lens(case)
    T, B = sum(rows), len(rows)
    rng = _tree_rng(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def draw_ints(high, *shape):
        return torch.randint(0, high, shape, generator=gen, device="cuda")

    state = {"case": case, "cu_rows": _offsets(rows), "max_rows": max(rows), "max_keys": max(keys)}
    if case["op"] != "commit":
        state["parents"] = _ints(sum(_parents(case, rows, rng), []))
    if case["op"] == "verify":
        return _prepare_verify(state, case, rows, gen)
    K, D, page = case["kv_heads"], case["dim"], case["page"]
    need = [-(-n // page) for n in keys]
    order = torch.randperm(sum(need), generator=gen, device="cuda").int()  # pages lie anywhere in the cache
    table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    state |= {"page_table": table, "lengths": _ints(keys)}
    L = case.get("layers", 1)  # codes and scales as the quantiser leaves them for values of about unit size
    shape = (L, sum(need), K, page)
    for part in ("k", "v"):
        state[part + "_codes"] = draw_ints(256, *shape, D // 2).to(torch.uint8)
        state[part + "_scales"] = (125 + (0.7 * normal(*shape, D // GROUP)).round()).clamp_(120, 128).to(torch.uint8)
    if own:  # a program keeps the handles of its caches
        state["caches"] = _handles(state)
    if case["op"] == "commit":
        paths = _paths(case, rows, rng)
        width = max(rows)
        state |= {"path": _ints([p + [-1] * (width - len(p)) for p in paths]), "accepted": _ints([len(p) - 1 for p in paths])}
        return state
    state |= {"q": (1.5 * normal(T, case["heads"], D)).to(DTYPES[case["dtype"]]), "scale": D ** -0.5}
    return state


def _prepare_verify(state, case, rows, gen):
    """Logits with a few likely tokens a row; drafted tokens that the target likes often enough."""
    T, B, V = sum(rows), len(rows), case["vocab"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    logits = 2 * normal(T, V)
    likely = torch.randint(0, V, (T, 12), generator=gen, device="cuda")
    logits.scatter_(1, likely, 8 + 5 * uniform(T, 12))
    start = state["cu_rows"][:-1].long().repeat_interleave(_ints(rows, torch.int64))
    first = torch.arange(T, device="cuda") == start
    parents = state["parents"].long()
    above = torch.where(first, start, start + parents)  # the row whose children a row belongs to
    # which child of its parent a row is: its place behind the first of them (children lie next to one another)
    order = 2 * above + ~first
    nth = torch.arange(T, device="cuda") - torch.searchsorted(order, order)
    guess = logits + 0.7 * normal(T, V)
    if case["draft"]:
        probs = torch.softmax(guess, -1)
        drawn = torch.multinomial(probs, max(rows), replacement=True, generator=gen)
        state["draft_probs"] = probs
    else:
        drawn = torch.topk(guess, min(V, max(rows)), dim=-1).indices
    state["tokens"] = drawn[above, nth.clamp(0, drawn.shape[1] - 1)].int()
    state["logits"] = logits.to(DTYPES[case["dtype"]])
    state["accept_u"], state["sample_u"] = uniform(T), uniform(B)
    temperature = 0.6 + 0.6 * uniform(B)
    state["temperature"] = torch.where(uniform(B) < case["greedy"], 0.0, temperature)
    return state


# ---------------------------------------------------------------- the library's calls

def _handles(s):
    from moe_expert_layer_top_gb300 import attention

    layers = zip(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    return [attention.KVCacheMXFP4(*layer) for layer in layers]


def _run_own(s):
    from moe_expert_layer_top_gb300 import attention, speculative

    case = s["case"]
    if case["op"] == "verify":
        out = speculative.verify_drafts(s["logits"], s["tokens"], s["cu_rows"], s["accept_u"], s["sample_u"],
                                        parents=s["parents"], draft_probs=s.get("draft_probs"),
                                        temperature=s["temperature"], max_rows=s["max_rows"])
        return out["tokens"], out["accepted"], out["path"]
    if case["op"] == "commit":
        lengths = speculative.commit_drafts(s["caches"], s["page_table"], s["lengths"], s["cu_rows"], s["path"],
                                            s["accepted"])
        return lengths, s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"]
    return attention.attend_tree(s["q"], s["caches"][0], s["page_table"], s["lengths"], s["cu_rows"], s["parents"],
                                 max_rows=s["max_rows"], scale=s["scale"], return_lse=True)


# ---------------------------------------------------------------- the plain forms

def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree, "verify": _verify, "commit": _commit}[state["case"]["op"]](state)


def _padded(cu, width):
    """Rows of every sequence, [sequence][width], and which of them are real."""
    r = torch.arange(width, device="cuda")
    count = cu[1:] - cu[:-1]
    return cu[:-1, None] + torch.minimum(r, count[:, None] - 1), r < count[:, None]


def _cache_values(codes, scales, table, length):
    """The cached rows 0..length-1 of every sequence, as fp32 [sequence][kv head][row][dim]."""
    page = codes.shape[2]
    at = torch.arange(length, device="cuda")
    pages, offset = table[:, at // page].long(), at % page
    c = codes[pages, :, offset].permute(0, 2, 1, 3)
    sc = scales[pages, :, offset].permute(0, 2, 1, 3)
    values = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    x = torch.stack([values[(c & 15).int()], values[(c >> 4).int()]], dim=-1).flatten(-2)
    scale = (sc.int() << 23).view(torch.float32)  # 2^(code - 127)
    return (x.unflatten(-1, (-1, GROUP)) * scale[..., None]).flatten(-2)


def _tree(s):
    q, cu, lengths = s["q"], s["cu_rows"].long(), s["lengths"].long()
    (T, H, D), K, R = q.shape, s["k_codes"].shape[2], s["max_rows"]
    B, G = len(lengths), H // K
    rows, real = _padded(cu, R)
    parent = torch.where(real, s["parents"][rows].long(), -1)
    r = torch.arange(R, device="cuda")
    above = (parent[..., None] == r) | (r[:, None] == r)  # a row's parent and itself, then all ancestors by squaring
    for _ in range(max(1, (R - 1).bit_length())):
        above = torch.matmul(above.float(), above.float()) > 0
    before = lengths - (cu[1:] - cu[:-1])  # keys in front of the tree
    key = torch.arange(s["max_keys"], device="cuda") - before[:, None]
    inside = ((key >= 0) & (key < R))[:, None]
    seen = torch.where(inside, above.gather(2, key.clamp(0, R - 1)[:, None].expand(B, R, -1)), (key < 0)[:, None])
    seen &= (key < (cu[1:] - cu[:-1])[:, None])[:, None]
    qh = (q[rows.flatten()].float() * s["scale"]).view(B, R, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, R * G, D)
    scores = torch.matmul(qh, _cache_values(s["k_codes"][0], s["k_scales"][0], s["page_table"], s["max_keys"]).transpose(-1, -2))
    scores.view(B, K, R, G, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    values = _cache_values(s["v_codes"][0], s["v_scales"][0], s["page_table"], s["max_keys"])
    out = torch.matmul(p, values) / torch.where(total == 0, 1.0, total)
    lse = (total.log() + top).squeeze(-1)
    out = out.view(B, K, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, H, D)[real].to(q.dtype)
    return out, lse.view(B, K, R, G).permute(0, 2, 1, 3).reshape(B, R, H)[real]


def _verify(s):
    """In 64 bits: a token is chosen where a long sum passes a border."""
    cu, R, B = s["cu_rows"].long(), s["max_rows"], len(s["sample_u"])
    rows, real = _padded(cu, R)
    V = s["logits"].shape[1]
    greedy, seq = s["temperature"] == 0, torch.arange(B, device="cuda")
    t = torch.where(greedy, 1.0, s["temperature"]).double()
    draft = s.get("draft_probs")

    def target(node):  # the target's probabilities behind a row of every sequence
        x = s["logits"][rows[seq, node]].double()
        w = torch.exp((x - x.amax(-1, keepdim=True)) / t[:, None])
        best = torch.zeros_like(w).scatter_(1, x.argmax(-1, keepdim=True), 1.0)
        return torch.where(greedy[:, None], best, w / w.sum(-1, keepdim=True))

    def one(x, token):
        return x.gather(1, token[:, None]).squeeze(1)

    node = torch.zeros(B, dtype=torch.int64, device="cuda")
    accepted = torch.zeros(B, dtype=torch.int64, device="cuda")
    path = torch.full((B, R), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    p = target(node)
    left, mass, taken = p.clone(), torch.ones(B, dtype=torch.float64, device="cuda"), torch.zeros(B, dtype=torch.float64, device="cuda")
    for i in range(1, R):
        row = rows[:, i]
        asked = real[:, i] & (s["parents"][row].long() == node)
        token = s["tokens"][row].long()
        u = s["accept_u"][row].double()
        q = draft[rows[seq, node]].double() if draft is not None else None
        drafted = one(q, token) if draft is not None else torch.ones_like(u)
        yes = asked & (u * mass * drafted < one(left, token))
        no = asked & ~yes
        # rejected: what the target has beyond the draft so far, or without the token, is left
        taken = torch.where(no, taken + mass, taken)
        rest = (p - taken[:, None] * q).clamp_min(0.0) if draft is not None else left.scatter(1, token[:, None], 0.0)
        left = torch.where(no[:, None], rest, left)
        node = torch.where(yes, i, node)
        accepted = accepted + yes
        path[seq, accepted] = torch.where(yes, i, path[seq, accepted])
        p = torch.where(yes[:, None], target(node), p)
        left = torch.where(yes[:, None], p, left)
        taken = torch.where(yes, 0.0, taken)
        mass = torch.where(no, left.sum(-1), torch.where(yes, 1.0, mass))
    left = torch.where(mass[:, None] > 0, left, p)
    sums = left.cumsum(-1)
    last = V - 1 - (left.flip(-1) > 0).int().argmax(-1)  # the last token with a weight
    new = torch.searchsorted(sums, (s["sample_u"].double() * sums[:, -1])[:, None], right=True).squeeze(1)
    new = torch.minimum(new, last)
    place = torch.arange(R, device="cuda")
    tokens = s["tokens"][rows[seq[:, None], path.roll(-1, 1).clamp_min(0)]].long()
    tokens = torch.where(place < accepted[:, None], tokens, torch.where(place == accepted[:, None], new[:, None], -1))
    return tokens.int(), accepted.int(), path.int()


def _commit(s):
    cu, lengths, accepted, path = s["cu_rows"].long(), s["lengths"].long(), s["accepted"].long(), s["path"].long()
    page = s["k_codes"].shape[3]
    before = lengths - (cu[1:] - cu[:-1])
    place = torch.arange(path.shape[1], device="cuda")
    b, j = torch.nonzero((place <= accepted[:, None]) & (path != place), as_tuple=True)
    source, target = before[b] + path[b, j], before[b] + j

    def page_of(at):
        return s["page_table"][b, at // page].long()

    parts = [s[x] for x in ("k_codes", "k_scales", "v_codes", "v_scales")]

    def move(x):
        x[:, page_of(target), :, target % page] = x[:, page_of(source), :, source % page]
        return x

    return (before + 1 + accepted).int(), *map(move, parts)


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "verify": _exact_verify, "commit": _exact_commit}[case["op"]](s)


def _exact_rows(codes, scales, pages, length):
    """One sequence's cached rows in 64 bits, [row][kv head][dim], from the bits of E2M1: sign, two exponent bits, one fraction bit."""
    c = codes[pages.long()].transpose(1, 2).flatten(0, 1)[:length].long()
    sc = scales[pages.long()].transpose(1, 2).flatten(0, 1)[:length].long()
    n = torch.stack([c % 16, c // 16], dim=-1).flatten(-2)
    e, f = n // 2 % 4, (n % 2).double()
    x = torch.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e.double() - 1)) * (1 - 2.0 * (n // 8))
    return x * (2.0 ** (sc - 127).double()).repeat_interleave(GROUP, -1)


def _exact_tree(s):
    cu, keys, parents = s["cu_rows"].tolist(), s["lengths"].tolist(), s["parents"].tolist()
    out, lse = [], []
    for b, m in enumerate(keys):
        first, n = cu[b], cu[b + 1] - cu[b]
        q = s["q"][first:first + n].double()
        k, v = (_exact_rows(s[x + "_codes"][0], s[x + "_scales"][0], s["page_table"][b], m) for x in ("k", "v"))
        seen = torch.zeros(n, m, dtype=torch.bool)
        seen[:, :m - n] = True
        for i in range(n):
            at = i
            while at >= 0:
                seen[i, m - n + at] = True
                at = parents[first + at]
        seen = seen.cuda()
        G = q.shape[1] // k.shape[1]
        o, z = torch.empty_like(q), torch.empty(n, q.shape[1], dtype=torch.float64, device="cuda")
        for h in range(q.shape[1]):
            x = ((q[:, h] @ k[:, h // G].T) * s["scale"]).masked_fill(~seen, -math.inf)
            z[:, h] = torch.logsumexp(x, -1)
            o[:, h] = torch.exp(x - z[:, h:h + 1]) @ v[:, h // G]
        out.append(o)
        lse.append(z)
    return torch.cat(out), torch.cat(lse)


def _exact_verify(s):
    """One sequence after another, with the residual as a list of the factors taken off."""
    cu, parents, drawn = s["cu_rows"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    u_accept, u_sample = s["accept_u"].tolist(), s["sample_u"].tolist()
    temperature, draft = s["temperature"].tolist(), s.get("draft_probs")
    tokens, accepted, paths = [], [], []

    def probabilities(row, t):
        x = s["logits"][row].double()
        if t == 0:
            p = torch.zeros_like(x)
            p[torch.nonzero(x == x.max())[0, 0]] = 1.0
            return p
        return torch.softmax(x / t, -1)

    for b in range(len(cu) - 1):
        first, n, node, path, said = cu[b], cu[b + 1] - cu[b], 0, [0], []
        while True:
            p = probabilities(first + node, temperature[b])
            rest, total, found = p, 1.0, None
            for i in range(1, n):
                if parents[first + i] != node:
                    continue
                y = drawn[first + i]
                q = 1.0 if draft is None else float(draft[first + node, y])
                if u_accept[first + i] * q * total < float(rest[y]):
                    found = i
                    break
                if draft is None:
                    rest = rest.clone()
                    rest[y] = 0.0
                else:  # max(rest / total - draft, 0), without the division
                    rest = (rest - total * draft[first + node].double()).clamp_min(0.0)
                total = float(rest.sum())
            if found is None:
                break
            node = found
            path.append(found)
            said.append(drawn[first + found])
        if total <= 0:
            rest = p
        sums = torch.cumsum(rest, 0)
        above = torch.nonzero(sums > u_sample[b] * float(sums[-1]))
        said.append(int(above[0, 0]) if len(above) else int(torch.nonzero(rest > 0)[-1, 0]))
        R = s["max_rows"]
        tokens.append(said + [-1] * (R - len(said)))
        accepted.append(len(path) - 1)
        paths.append(path + [-1] * (R - len(path)))
    return _ints(tokens), _ints(accepted), _ints(paths)


def _exact_commit(s):
    cu, keys, path, accepted = s["cu_rows"].tolist(), s["lengths"].tolist(), s["path"].tolist(), s["accepted"].tolist()
    table, page = s["page_table"].tolist(), s["k_codes"].shape[3]
    parts = [s[x].clone() for x in ("k_codes", "k_scales", "v_codes", "v_scales")]
    lengths = []
    for b, m in enumerate(keys):
        base = m - (cu[b + 1] - cu[b])
        for j in range(accepted[b] + 1):
            source, target = base + path[b][j], base + j
            for new, name in zip(parts, ("k_codes", "k_scales", "v_codes", "v_scales")):
                new[:, table[b][target // page], :, target % page] = s[name][:, table[b][source // page], :, source % page]
        lengths.append(base + 1 + accepted[b])
    return _ints(lengths), *parts
