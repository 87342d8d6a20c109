"""Cases and plain forms of the attention operators next to the MoE step.

Three operators, as a serving program uses them in a decoder layer:

* append: RMSNorm of each query and key head, rotary positions, and the MXFP4 quantisation of keys and values into the
  paged cache (``attention.qkv_append``);
* prompt: causal attention over packed prompts with grouped heads (``attention.attend_prompt``);
* paged: attention of one token, or of the few rows of a verify step, over the paged MXFP4 cache
  (``attention.attend_paged``).

``run`` computes a case in elementary torch operations, or, with ``own`` set, through the library's entry points.
``exact`` computes it in 64 bits, written separately.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
GROUP = 32
EPS = 1e-6
MAX_POSITION = 65536


# ---------------------------------------------------------------- cases

def listed():
    heads = {"heads": 32, "kv_heads": 8, "dim": 128}
    return [
        # the six rows of one sequence's verify step
        {"name": "append_verify_bs1", "op": "append", "dtype": "bf16", **heads, "rows": 6, "rotary": 128,
         "interleaved": False, "norm": True, "page": 64},
        # 64 sequences' verify rows, half-width heads, interleaved partial rotation
        {"name": "append_verify_bs64_d64", "op": "append", "dtype": "fp16", "heads": 64, "kv_heads": 8, "dim": 64,
         "rows": 384, "rotary": 32, "interleaved": True, "norm": True, "page": 16},
        # a prompt chunk as long as the library's largest step
        {"name": "append_prompt_4096", "op": "append", "dtype": "bf16", **heads, "rows": 4096, "rotary": 128,
         "interleaved": False, "norm": True, "page": 64},
        # one short prompt of odd length
        {"name": "prompt_257", "op": "prompt", "dtype": "bf16", **heads, "seqs": 1, "len_min": 257, "len_max": 257,
         "prefix": 0, "lens_seed": 1},
        # a batch of prompts of very different lengths, packed
        {"name": "prompt_packed_16", "op": "prompt", "dtype": "bf16", **heads, "seqs": 16, "len_min": 1,
         "len_max": 2000, "prefix": 0, "lens_seed": 2},
        # chunks of longer prompts: each chunk's rows also see the keys before it
        {"name": "prompt_chunks_d64", "op": "prompt", "dtype": "fp16", "heads": 64, "kv_heads": 8, "dim": 64,
         "seqs": 3, "len_min": 500, "len_max": 1500, "prefix": 4000, "lens_seed": 3},
        # one long prompt
        {"name": "prompt_16384", "op": "prompt", "dtype": "bf16", **heads, "seqs": 1, "len_min": 16384,
         "len_max": 16384, "prefix": 0, "lens_seed": 4},
        # one new token of one sequence
        {"name": "paged_token_bs1", "op": "paged", "dtype": "bf16", **heads, "seqs": 1, "rows_min": 1, "rows_max": 1,
         "len_min": 4096, "len_max": 4096, "page": 64, "lens_seed": 5},
        # the six-row verify step of one sequence with a long context
        {"name": "paged_verify_bs1_long", "op": "paged", "dtype": "bf16", **heads, "seqs": 1, "rows_min": 6,
         "rows_max": 6, "len_min": 131071, "len_max": 131071, "page": 64, "lens_seed": 6},
        # six-row verify steps of 64 sequences, 1K to 5K tokens each
        {"name": "paged_verify_bs64", "op": "paged", "dtype": "bf16", **heads, "seqs": 64, "rows_min": 6,
         "rows_max": 6, "len_min": 1024, "len_max": 5120, "page": 64, "lens_seed": 7},
        # half-width heads, eight query heads to a kv head, small pages, one to four rows a sequence
        {"name": "paged_ragged_d64", "op": "paged", "dtype": "fp16", "heads": 64, "kv_heads": 8, "dim": 64,
         "seqs": 24, "rows_min": 1, "rows_max": 4, "len_min": 7, "len_max": 9000, "page": 16, "lens_seed": 8},
        # single tokens of a large batch
        {"name": "paged_token_bs128", "op": "paged", "dtype": "bf16", **heads, "seqs": 128, "rows_min": 1,
         "rows_max": 1, "len_min": 4000, "len_max": 16000, "page": 64, "lens_seed": 9},
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    dim = rng.choice([64, 128, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    base = {"dtype": rng.choice(["bf16", "fp16"]), "heads": heads, "kv_heads": kv_heads, "dim": dim}
    op = rng.choice(["append", "prompt", "paged"])
    if op == "append":
        return {"op": op, **base, "rows": _log_uniform(rng, 1, 4096), "rotary": rng.choice([dim // 2, dim]),
                "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.8, "page": rng.choice([16, 32, 64, 128])}
    lens_seed = rng.randrange(1 << 20)
    if op == "prompt":
        longest = _log_uniform(rng, 1, 8000)
        seqs = max(1, min(_log_uniform(rng, 1, 24), 12000 // longest))
        return {"op": op, **base, "seqs": seqs, "len_min": max(1, longest // rng.choice([1, 4, 50])),
                "len_max": longest, "prefix": rng.choice([0, 0, _log_uniform(rng, 1, 3000)]), "lens_seed": lens_seed}
    longest = _log_uniform(rng, 1, 100000)
    seqs = max(1, min(_log_uniform(rng, 1, 128), 400000 // longest))
    rows = rng.choice([1, 1, 2, 6, 8])
    return {"op": op, **base, "seqs": seqs, "rows_min": rng.choice([1, rows]), "rows_max": rows,
            "len_min": max(1, longest // rng.choice([1, 3, 40])), "len_max": longest,
            "page": rng.choice([16, 32, 64, 128]), "lens_seed": lens_seed}


def _lens(case):
    """Query rows and keys of every sequence of an attention case."""
    rng = random.Random(case["lens_seed"])
    rows, keys = [], []
    for _ in range(case["seqs"]):
        n = _log_uniform(rng, case["len_min"], case["len_max"])
        if case["op"] == "prompt":
            rows.append(n)
            keys.append(n + (rng.randint(0, case["prefix"]) if case["prefix"] else 0))
        else:
            rows.append(rng.randint(case["rows_min"], case["rows_max"]))
            keys.append(n)
    return rows, keys


def _pairs(rows, keys):
    """(row, key) pairs that the causal mask leaves: row i of n sees keys j <= i + keys - n."""
    total = 0
    for n, m in zip(rows, keys):
        first = m - n + 1  # keys of row 0
        skipped = max(0, -first + 1) if first < 1 else 0
        live = max(0, n - skipped)
        low = max(first, 1)
        total += live * low + live * (live - 1) // 2
    return total


def work(case):
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    cached = 2 * (D // 2 + D // GROUP)  # bytes of one token and kv head in the cache
    if case["op"] == "append":
        T = case["rows"]
        moved = T * (H + 2 * K) * D * 2 + T * H * D * 2 + T * K * (cached + 2 * D * 2) + T * case["rotary"] * 4 + T * 12
        return {"bytes": moved, "flops": T * (H + K) * D * 10}
    rows, keys = _lens(case)
    T = sum(rows)
    flops = 4 * D * H * _pairs(rows, keys)
    if case["op"] == "prompt":
        return {"bytes": 4 * T * H * D + 4 * sum(keys) * K * D + 4 * T * H, "flops": flops}
    return {"bytes": sum(keys) * K * cached + 4 * T * H * D + 4 * T * H, "flops": flops}


# ---------------------------------------------------------------- inputs

def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _rope_table(rotary):
    """fp32 [position][cos of rotary/2 angles, then sin], from 64-bit angles."""
    freq = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64, device="cuda") / rotary)
    angle = torch.arange(MAX_POSITION, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H, K, D = case["heads"], case["kv_heads"], case["dim"]
    dtype = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def draw_ints(high, *shape):
        return torch.randint(0, high, shape, generator=gen, device="cuda")

    state = {"case": case, "scale": D ** -0.5}
    if case["op"] == "append":
        T, page = case["rows"], case["page"]
        pages = 2 * T // page + 2
        qkv = (normal(T, H + 2 * K, D) * (1 + 0.5 * normal(H + 2 * K, 1)).abs()).to(dtype)  # one projection's output
        state |= {"q": qkv[:, :H], "k": qkv[:, H:H + K], "v": qkv[:, H + K:], "rope": _rope_table(case["rotary"]),
                  "positions": draw_ints(MAX_POSITION, T).int(),
                  "slots": torch.randperm(pages * page, generator=gen, device="cuda")[:T],
                  "q_norm": (1 + 0.25 * normal(D)).to(dtype) if case["norm"] else None,
                  "k_norm": (1 + 0.25 * normal(D)).to(dtype) if case["norm"] else None}
        state |= _empty_cache(pages, K, page, D)
        return state
    rows, keys = _lens(case)
    T = sum(rows)
    state |= {"cu_rows": _offsets(rows), "max_rows": max(rows), "max_keys": max(keys)}
    if case["op"] == "prompt":
        state |= {"q": (1.5 * normal(T, H, D)).to(dtype), "k": normal(sum(keys), K, D).to(dtype),
                  "v": (normal(sum(keys), K, D) + 0.25 * normal(K, D)).to(dtype), "cu_keys": _offsets(keys)}
        return state
    page = case["page"]
    need = [-(-n // page) for n in keys]
    state["q"] = (1.5 * normal(T, H, D)).to(dtype)
    order = torch.randperm(sum(need), generator=gen, device="cuda").int()  # pages lie anywhere in the cache
    table = torch.zeros(len(keys), max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    state |= {"page_table": table, "lengths": torch.tensor(keys, dtype=torch.int32, device="cuda")}
    state |= _empty_cache(sum(need), K, page, D)
    for part in ("k", "v"):  # codes and scales as the quantiser leaves them for values of about unit size
        state[part + "_codes"].copy_(draw_ints(256, *state[part + "_codes"].shape))
        scales = 125 + (0.7 * normal(*state[part + "_scales"].shape)).round()
        state[part + "_scales"].copy_(scales.clamp(120, 128))
    return state


def _empty_cache(pages, kv_heads, page, dim):
    def zeros(width):
        return torch.zeros(pages, kv_heads, page, width, dtype=torch.uint8, device="cuda")

    return {"k_codes": zeros(dim // 2), "k_scales": zeros(dim // GROUP), "v_codes": zeros(dim // 2),
            "v_scales": zeros(dim // GROUP)}


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    from moe_expert_layer_top_gb300 import attention

    case = s["case"]
    if case["op"] == "prompt":
        return attention.attend_prompt(s["q"], s["k"], s["v"], s["cu_rows"], s["cu_keys"], scale=s["scale"],
                                       return_lse=True)
    cache = attention.KVCacheMXFP4(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"])
    if case["op"] == "append":
        out = attention.qkv_append(s["q"], s["k"], s["v"], positions=s["positions"], rope=s["rope"],
                                   interleaved=case["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                                   cache=cache, slots=s["slots"], cached_values=True)
        return out["q"], out["k_cached"], out["v_cached"]
    return attention.attend_paged(s["q"], cache, s["page_table"], s["lengths"], s["cu_rows"],
                                  max_rows=s["max_rows"], scale=s["scale"], return_lse=True)


# ---------------------------------------------------------------- the plain forms

def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "prompt": _prompt, "paged": _paged}[state["case"]["op"]](state)


def _power_of_two(exponent):
    """2^exponent in 64 bits, exactly."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _round_to(x, dtype):
    """x (64 bits) rounded once to a 16-bit type, nearest even."""
    bits, lowest = (8, -133) if dtype == torch.bfloat16 else (11, -24)
    step = _power_of_two((torch.frexp(x).exponent - bits).clamp_min(lowest))
    return (torch.round(x / step) * step).to(dtype)


def _norm_rotate(x, gamma, s, wide):
    """RMSNorm of each head, then the rotation of the first `rotary` dimensions."""
    case = s["case"]
    x = x.to(wide)
    if gamma is not None:
        x = x * gamma.to(wide) / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)
    half = case["rotary"] // 2
    table = s["rope"][s["positions"].long()].to(wide)[:, None]
    cos, sin = table[..., :half], table[..., half:]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if case["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1)


def _mxfp4_values(x):
    """The values that MXFP4 (group-32 scales 2^(floor(log2 amax) - 2), E2M1 elements) keeps of x."""
    g = x.double().unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1, keepdim=True)
    code = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 2 + 127, 0).clamp(0, 254)
    scale = _power_of_two(code - 127)
    a = (g / scale).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp_max(6.0)
    return (torch.copysign(a, g) * scale).flatten(-2).to(x.dtype)


def _append(s):
    dtype = s["q"].dtype
    q = _norm_rotate(s["q"], s["q_norm"], s, torch.float32).to(dtype)
    k = _round_to(_norm_rotate(s["k"], s["k_norm"], s, torch.float64), dtype)  # 64 bits: its 4-bit codes lie next to borders
    return q, _mxfp4_values(k), _mxfp4_values(s["v"])


def _softmax_sum(scores, values):
    """(softmax(scores) values, log sum exp) over the last axis of scores; rows of -inf give 0 and -inf."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values) / torch.where(total == 0, 1.0, total)
    return out, (total.log() + top).squeeze(-1)


def _prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    (Tq, H, D), (Tk, K) = q.shape, k.shape[:2]
    G = H // K
    cu_q, cu_k = s["cu_rows"].long(), s["cu_keys"].long()
    row, key = torch.arange(Tq, device="cuda"), torch.arange(Tk, device="cuda")
    row_seq = torch.searchsorted(cu_q, row, right=True) - 1
    key_seq = torch.searchsorted(cu_k, key, right=True) - 1
    last = (row - cu_q[row_seq + 1]) + cu_k[row_seq + 1]  # the last key that a row sees
    seen = (row_seq[:, None] == key_seq) & (key <= last[:, None])
    qh = (q.float() * s["scale"]).view(Tq, K, G, D).permute(1, 2, 0, 3).reshape(K, G * Tq, D)
    scores = torch.matmul(qh, k.float().permute(1, 2, 0))
    scores.view(K, G, Tq, Tk).masked_fill_(~seen, -math.inf)
    out, lse = _softmax_sum(scores, v.float().permute(1, 0, 2))
    out = out.view(K, G, Tq, D).permute(2, 0, 1, 3).reshape(Tq, H, D).to(q.dtype)
    return out, lse.view(H, Tq).t().contiguous()


def _cache_values(codes, scales, table, length):
    """The cached rows 0..length-1 of every sequence, as fp32 [sequence][kv head][row][dim]."""
    page = codes.shape[2]
    at = torch.arange(length, device="cuda")
    pages, offset = table[:, at // page].long(), at % page
    c = codes[pages, :, offset].permute(0, 2, 1, 3)
    sc = scales[pages, :, offset].permute(0, 2, 1, 3)
    values = torch.tensor(E2M1 + tuple(-x for x in E2M1), device="cuda")
    x = torch.stack([values[(c & 15).int()], values[(c >> 4).int()]], dim=-1).flatten(-2)
    return (x.unflatten(-1, (-1, GROUP)) * _power_of_two(sc.int() - 127).float()[..., None]).flatten(-2)


def _paged(s):
    q, cu, lengths = s["q"], s["cu_rows"].long(), s["lengths"].long()
    (T, H, D), K, R = q.shape, s["k_codes"].shape[1], s["max_rows"]
    B, G = len(lengths), H // K
    count = cu[1:] - cu[:-1]
    r = torch.arange(R, device="cuda")
    real = r < count[:, None]
    padded = (cu[:-1, None] + torch.minimum(r, count[:, None] - 1)).flatten()
    qh = (q[padded].float() * s["scale"]).view(B, R, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, R * G, D)
    keys = _cache_values(s["k_codes"], s["k_scales"], s["page_table"], s["max_keys"])
    scores = torch.matmul(qh, keys.transpose(-1, -2))
    limit = (lengths - count)[:, None] + r + 1  # keys that a row sees
    hidden = torch.arange(s["max_keys"], device="cuda") >= limit[..., None]
    scores.view(B, K, R, G, -1).masked_fill_(hidden[:, None, :, None], -math.inf)
    values = _cache_values(s["v_codes"], s["v_scales"], s["page_table"], s["max_keys"])
    out, lse = _softmax_sum(scores, values)
    out = out.view(B, K, R, G, D).permute(0, 2, 1, 3, 4).reshape(B, R, H, D)[real].to(q.dtype)
    return out, lse.view(B, K, R, G).permute(0, 2, 1, 3).reshape(B, R, H)[real]


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    rows, keys = _lens(case)
    out, lse = [], []
    row0 = key0 = 0
    for b, (n, m) in enumerate(zip(rows, keys)):
        q = s["q"][row0:row0 + n].double()
        if case["op"] == "prompt":
            k, v = s["k"][key0:key0 + m].double(), s["v"][key0:key0 + m].double()
        else:
            k, v = (_exact_rows(s[x + "_codes"], s[x + "_scales"], s["page_table"][b], m) for x in ("k", "v"))
        for first in range(0, n, 1024):
            o, z = _exact_rows_attend(q[first:first + 1024], k, v, s["scale"], m - n + first)
            out.append(o)
            lse.append(z)
        row0, key0 = row0 + n, key0 + m
    return torch.cat(out), torch.cat(lse)


def _exact_rows_attend(q, k, v, scale, before):
    """Rows of one sequence; row i sees keys 0 .. before + i."""
    n, H, D = q.shape
    m = max(0, min(len(k), before + n))
    if m == 0:
        return torch.zeros_like(q), torch.full((n, H), -math.inf, dtype=torch.float64, device="cuda")
    G = H // k.shape[1]
    unseen = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(before + 1)
    out, lse = torch.empty_like(q), torch.empty(n, H, dtype=torch.float64, device="cuda")
    for h in range(H):
        x = (q[:, h] @ k[:m, h // G].T) * scale
        x = x.masked_fill(unseen, -math.inf)
        z = torch.logsumexp(x, -1)
        w = torch.exp(x - torch.where(z.isinf(), 0.0, z)[:, None])
        out[:, h], lse[:, h] = w @ v[:m, h // G], z
    return out, lse


def _exact_rows(codes, scales, pages, length):
    """One sequence's cached rows in 64 bits, [row][kv head][dim], from the bits of E2M1: sign, two exponent bits, one fraction bit."""
    c = codes[pages.long()].transpose(1, 2).flatten(0, 1)[:length].long()
    sc = scales[pages.long()].transpose(1, 2).flatten(0, 1)[:length]
    n = torch.stack([c % 16, c // 16], dim=-1).flatten(-2)
    e, f = n // 2 % 4, (n % 2).double()
    x = torch.where(e == 0, f / 2, (1 + f / 2) * 2.0 ** (e.double() - 1)) * (1 - 2.0 * (n // 8))
    return x * _exact_powers(sc.long() - 127).repeat_interleave(GROUP, -1)


def _exact_powers(exponent):
    return torch.tensor([2.0 ** e for e in range(-160, 161)], dtype=torch.float64, device="cuda")[exponent + 160]


def _exact_append(s):
    case, dtype = s["case"], s["q"].dtype
    half = case["rotary"] // 2
    turn = torch.complex(*(s["rope"][s["positions"].long()].double().split(half, -1)))[:, None]
    first = torch.arange(half, device="cuda")
    if case["interleaved"]:
        first, second = 2 * first, 2 * first + 1
    else:
        second = first + half

    def rotated(x, gamma):
        y = x.double().clone()
        if gamma is not None:
            y = y * torch.rsqrt((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + EPS) * gamma.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    def rounded(x):  # to the type's significant bits by adding and taking off a large multiple, and to its lowest step
        bits, lowest = (8, 2.0 ** -133) if dtype == torch.bfloat16 else (11, 2.0 ** -24)
        big = x * (2.0 ** (53 - bits) + 1)
        high = big - (big - x)
        coarse = 1.5 * 2.0 ** 52 * lowest
        return torch.where(x.abs() < lowest * 2.0 ** (bits - 1), (x + coarse) - coarse, high)

    def kept(x):
        g = x.double().unflatten(-1, (-1, GROUP))
        top = g.abs().amax(-1, keepdim=True)
        powers = _exact_powers(torch.arange(-160, 161, device="cuda"))
        scale = _exact_powers((torch.searchsorted(powers, top, right=True) - 161 - 2).clamp(-127, 127))
        grid = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
        low = torch.searchsorted((grid[1:] + grid[:-1]) / 2, g.abs() / scale)  # a tie goes to the lower value ...
        up = torch.searchsorted((grid[1:] + grid[:-1]) / 2, g.abs() / scale, right=True)
        return (grid[torch.where(low % 2 == 0, low, up)] * g.sign() * scale).flatten(-2)  # ... or to the even code

    return rotated(s["q"], s["q_norm"]), kept(rounded(rotated(s["k"], s["k_norm"]))), kept(s["v"])
