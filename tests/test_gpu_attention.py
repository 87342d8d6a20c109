"""The attention calls on the GPU against the 64-bit oracle.

Bounds are derived in ``attention_cases.check_attention`` and beside each test. The 4-bit cache is compared bit for
bit: the keys' codes are those of the exact formula.
"""
import numpy as np
import pytest
import torch

import oracle
from oracle import attention as oa
from moe_expert_layer_top_gb300 import abi, attention
from moe_expert_layer_top_gb300.layer import quantize_mxfp4

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


# ------------------------------------------------------------------ append

APPEND = [
    # T, heads, kv heads, D, R, interleaved, norms, page, dtype
    (6, 32, 8, 128, 128, False, True, 64, "bf16"),
    (1, 1, 1, 128, 64, True, True, 16, "bf16"),
    (7, 5, 1, 64, 64, False, True, 32, "fp16"),
    (33, 8, 8, 64, 32, True, True, 16, "bf16"),
    (19, 12, 4, 128, 48, False, True, 48, "fp16"),    # half of R is not a power of two
    (5, 6, 2, 128, 112, True, False, 16, "bf16"),     # no norm
    (40, 3, 3, 64, 0, False, True, 16, "fp16"),       # no rotation
    (700, 32, 8, 128, 128, False, True, 64, "bf16"),  # one block a token
    (1500, 16, 2, 64, 16, False, True, 128, "fp16"),
]


def append_case(T, H, K, D, R, dtype, norm, page, seed=0):
    rng = np.random.default_rng(seed)
    qkv = ac.rows16(rng, (T, H + 2 * K, D), dtype, 1.7)
    qn = oa.round16(1 + 0.25 * rng.standard_normal(D), dtype) if norm else None
    kn = oa.round16(1 + 0.25 * rng.standard_normal(D), dtype) if norm else None
    pos = rng.integers(0, 50000, T)
    rope = attention.rope_table(50000, R, device="cpu") if R else None
    pages = 2 * T // page + 2
    slots = rng.permutation(pages * page)[:T]
    return qkv, qn, kn, pos, rope, pages, slots


@pytest.mark.parametrize("T,H,K,D,R,inter,norm,page,dtype", APPEND, ids=[f"T{c[0]}_D{c[3]}_R{c[4]}_{c[8]}" for c in APPEND])
def test_append_matches_the_oracle(T, H, K, D, R, inter, norm, page, dtype):
    qkv, qn, kn, pos, rope, pages, slots = append_case(T, H, K, D, R, dtype, norm, page)
    eps = 1e-6
    x = ac.dev(qkv, dtype)
    slots[::5] = -1  # some tokens stay out of the cache
    c = attention.KVCacheMXFP4.empty(pages, page, K, D)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.fill_(0xA5)
    st = status()
    out = attention.qkv_append(x[:, :H], x[:, H:H + K], x[:, H + K:], positions=ac.dev(pos.astype(np.int32)) if R else None,
                               rope=rope.cuda() if R else None, interleaved=inter,
                               q_norm=ac.dev(qn, dtype) if norm else None, k_norm=ac.dev(kn, dtype) if norm else None,
                               eps=eps, cache=c, slots=ac.dev(slots.astype(np.int64)), rotated_keys=True,
                               cached_values=True, d_status=st)
    assert st.item() == abi.MOE_OK
    table = rope.double().numpy()[pos] if R else np.zeros((T, 0))
    cos, sin = table[:, :R // 2], table[:, R // 2:]
    eps32 = float(np.float32(eps))
    q = oa.norm_rotate(qkv[:, :H], qn, eps32, cos, sin, inter)
    # binary32: 8 + log2(D/8) additions of squares, half of that relative in the root, rsqrt (2 ulp), three products,
    # two products and a sum of the rotation: 16 roundings of terms no larger than |a| + |b|
    size = np.abs(q)
    if R:
        size = size + np.sqrt((q[..., :R] ** 2).max(-1, keepdims=True)) * np.sqrt(2)
    bound = ac.HALF_STEP[dtype] * np.abs(q) + 16 * 2.0 ** -24 * size + ac.HALF_TINY[dtype]
    assert (np.abs(ac.f64(out["q"]) - q) <= bound).all()
    k = oa.round16(oa.norm_rotate(qkv[:, H:H + K], kn, eps32, cos, sin, inter), dtype)
    np.testing.assert_array_equal(ac.f64(out["k"]), k)
    want = {}
    for name, vals in (("k", k), ("v", qkv[:, H + K:])):
        codes, scales = oracle.mxfp4_quantize(vals.reshape(T * K, D))
        kept = oracle.mxfp4_dequantize(codes, scales).reshape(T, K, D)
        np.testing.assert_array_equal(ac.f64(out[name + "_cached"]), oa.round16(kept, dtype))
        for part, rows, width in (("codes", codes, D // 2), ("scales", scales, D // 32)):
            full = np.full((pages, K, page, width), 0xA5, dtype=np.uint8)
            for t in range(T):
                if slots[t] >= 0:
                    full[slots[t] // page, :, slots[t] % page] = rows.reshape(T, K, width)[t]
            want[f"{name}_{part}"] = full
    for name, full in want.items():
        np.testing.assert_array_equal(getattr(c, name).cpu().numpy(), full, err_msg=name)


def test_append_codes_are_those_of_the_quantiser():
    T, K, D = 64, 4, 128
    x = torch.randn(T, 3 * K, D, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    c = attention.KVCacheMXFP4.empty(4, 16, K, D)
    out = attention.qkv_append(x[:, :K], x[:, K:2 * K], x[:, 2 * K:], cache=c, slots=torch.arange(T, device="cuda"),
                               rotated_keys=True)
    assert torch.equal(out["q"], x[:, :K]) and torch.equal(out["k"], x[:, K:2 * K])  # no norm, no rotation
    for vals, codes, scales in ((x[:, K:2 * K], c.k_codes, c.k_scales), (x[:, 2 * K:], c.v_codes, c.v_scales)):
        q, s = quantize_mxfp4(vals.contiguous())
        assert torch.equal(codes.transpose(1, 2).reshape(T, K, D // 2), q)
        assert torch.equal(scales.transpose(1, 2).reshape(T, K, D // 32), s)


def test_append_special_values():
    """Zeros, the smallest and largest magnitudes, infinities and NaN: the quantiser's codes, and nothing else moves."""
    K, D = 1, 64
    rows = torch.zeros(7, 1, D)
    rows[1, 0, :4] = torch.tensor([2.0 ** -133, -2.0 ** -130, 2.0 ** -126, 0.0])
    rows[2, 0, 0], rows[2, 0, 40] = 3.3e38, -3.3e38
    rows[3, 0, 5] = float("inf")
    rows[4, 0, 6] = float("nan")
    rows[5] = -0.0
    rows[6] = torch.linspace(-6, 6, D)
    x = rows.bfloat16().cuda()
    c = attention.KVCacheMXFP4.empty(1, 16, K, D)
    attention.qkv_append(x, x, x, cache=c, slots=torch.arange(7, device="cuda"))
    q, s = quantize_mxfp4(x)
    for codes, scales in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)):
        assert torch.equal(codes[0, 0, :7], q[:, 0]) and torch.equal(scales[0, 0, :7], s[:, 0])


def test_append_in_place_and_without_a_cache():
    T, H, K, D = 9, 4, 2, 64
    qkv, qn, kn, pos, rope, _, _ = append_case(T, H, K, D, 64, "bf16", True, 16, seed=4)
    q, k, v = (ac.dev(p, "bf16") for p in (qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]))
    kw = dict(positions=ac.dev(pos.astype(np.int32)), rope=rope.cuda(), q_norm=ac.dev(qn, "bf16"))
    want = attention.qkv_append(q, k, v, **kw)["q"]
    got = attention.qkv_append(q, k, v, q_out=q, **kw)["q"]
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)
    assert attention.qkv_append(q[:0], k[:0], v[:0])["q"].shape == (0, H, D)


def test_append_reports_positions_and_slots_out_of_range():
    T, K, D = 5, 2, 64
    x = torch.randn(T, 3 * K, D, device="cuda").bfloat16()
    rope = attention.rope_table(10, 64)
    c = attention.KVCacheMXFP4.empty(2, 16, K, D)
    for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales):
        t.zero_()
    q_out = torch.full((T, K, D), 7.0, device="cuda").bfloat16()
    st = status()
    attention.qkv_append(x[:, :K], x[:, K:2 * K], x[:, 2 * K:], positions=ac.i32([0, 10, 9, -1, 3]), rope=rope, cache=c,
                         slots=torch.tensor([3, 4, 32, 5, 31], device="cuda"), q_out=q_out, d_status=st)
    assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
    assert (q_out[[1, 3]] == 7).all() and not (q_out[[0, 2, 4]] == 7).all(-1).any()
    live = (c.k_codes != 0).any(-1).any(1).flatten().nonzero().flatten().tolist()
    assert live == [3, 31]


# ------------------------------------------------------------------ prompts

PROMPT = [
    # (rows, keys) of each sequence, heads, kv heads, D, dtype, causal
    ([(1, 1)], 1, 1, 128, "bf16", True),
    ([(5, 5), (0, 0), (1, 1), (70, 70)], 4, 2, 64, "bf16", True),
    ([(33, 33), (127, 127), (128, 128), (129, 129)], 2, 1, 128, "fp16", True),
    ([(3, 200), (40, 41), (17, 300)], 8, 2, 128, "bf16", True),       # chunks behind a prefix
    ([(20, 7), (4, 0), (9, 9)], 3, 3, 64, "fp16", True),              # rows without keys
    ([(20, 7), (4, 0), (65, 140)], 5, 1, 128, "bf16", False),         # no mask
    ([(257, 257)], 8, 1, 64, "bf16", True),
    ([(300, 555)], 2, 2, 128, "fp16", True),
    ([(0, 5), (2, 2)], 16, 1, 128, "bf16", True),
]


def run_prompt(seqs, H, K, D, dtype, causal, seed=0, sigma=1.0, scale=None, check=True):
    rng = np.random.default_rng(seed)
    n, m = sum(s[0] for s in seqs), sum(s[1] for s in seqs)
    q, k, v = ac.rows16(rng, (n, H, D), dtype, 1.5 * sigma), ac.rows16(rng, (m, K, D), dtype, sigma), ac.rows16(rng, (m, K, D), dtype)
    scale = D ** -0.5 if scale is None else scale
    cr, ck = ac.offsets([s[0] for s in seqs]), ac.offsets([s[1] for s in seqs])
    st = status()
    out, lse = attention.attend_prompt(ac.dev(q, dtype), ac.dev(k, dtype), ac.dev(v, dtype), ac.i32(cr), ac.i32(ck),
                                       causal=causal, scale=scale, return_lse=True, d_status=st)
    assert st.item() == abi.MOE_OK
    if check:
        for b in range(len(seqs)):
            r, s = slice(cr[b], cr[b + 1]), slice(ck[b], ck[b + 1])
            ac.check_attention(out[r], lse[r], q[r], k[s], v[s], scale, dtype, dtype, causal)
    return out, lse


@pytest.mark.parametrize("case", PROMPT, ids=[f"{c[0][0][0]}x{c[0][0][1]}_D{c[3]}_{c[4]}_{'c' if c[5] else 'f'}" for c in PROMPT])
def test_prompt_matches_the_oracle(case):
    run_prompt(*case, seed=len(case[0]))


@pytest.mark.parametrize("sigma,scale", [(30.0, None), (1.0, 0.0), (1.0, -0.2), (1e-4, None), (1.0, 3.0)])
def test_prompt_scales(sigma, scale):
    """Peaked rows, flat rows, a zero and a negative scale."""
    run_prompt([(150, 150), (10, 60)], 2, 1, 128, "bf16", True, seed=9, sigma=sigma, scale=scale)


def test_prompt_strides_and_rows_behind_the_last_sequence():
    H, K, D, T = 4, 2, 128, 50
    rng = np.random.default_rng(12)
    qkv = ac.rows16(rng, (T, H + 2 * K, D), "bf16")
    x = ac.dev(qkv, "bf16")
    out = torch.full((T, H + 1, D), 5.0, device="cuda").bfloat16()
    cu = ac.i32([0, 20, 41])
    got, lse = attention.attend_prompt(x[:, :H], x[:, H:H + K], x[:, H + K:], cu, cu, out=out[:, :H], return_lse=True)
    assert (out[41:] == 5).all() and (out[:, H] == 5).all()
    for a, b in ((0, 20), (20, 41)):
        ac.check_attention(got[a:b], lse[a:b], qkv[a:b, :H], qkv[a:b, H:H + K], qkv[a:b, H + K:], D ** -0.5, "bf16", "bf16")


def test_prompt_nan_of_one_sequence_stays_there():
    H, K, D = 2, 1, 64
    x = torch.randn(150, H + 2 * K, D, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).bfloat16()
    cu = ac.i32([0, 60, 75, 150])
    want = attention.attend_prompt(x[:, :H], x[:, H:H + K], x[:, H + K:], cu, cu)
    y = x.clone()
    y[60:75, H:] = float("nan")
    y[62, H + K:] = float("inf")
    got = attention.attend_prompt(y[:, :H], y[:, H:H + K], y[:, H + K:], cu, cu)
    assert torch.equal(got[:60], want[:60]) and torch.equal(got[75:], want[75:])


def test_prompt_nan_in_later_keys_stays_out_of_earlier_rows():
    """Masked keys have no weight: not even a NaN among them reaches a row."""
    H, K, D, n = 2, 1, 128, 40
    x = torch.randn(n, H + 2 * K, D, device="cuda", generator=torch.Generator("cuda").manual_seed(6)).bfloat16()
    cu = ac.i32([0, n])
    want = attention.attend_prompt(x[:, :H], x[:, H:H + K], x[:, H + K:], cu, cu)
    y = x.clone()
    y[30:, H:H + K] = float("nan")  # keys
    got = attention.attend_prompt(y[:, :H], y[:, H:H + K], y[:, H + K:], cu, cu)
    assert torch.equal(got[:30], want[:30])


def test_prompt_reports_bad_offsets():
    x = torch.randn(40, 3, 64, device="cuda").bfloat16()
    q, k, v = x[:, :1], x[:, 1:2], x[:, 2:]
    good = attention.attend_prompt(q, k, v, ac.i32([0, 10, 40]), ac.i32([0, 10, 40]))
    for rows, keys in (([0, 10, 41], [0, 10, 40]), ([0, 10, 40], [0, 10, 50]), ([0, 10, 5], [0, 10, 40]),
                       ([0, 10, 40], [0, 10, -1]), ([0, 10, 2 ** 31 - 1], [0, 10, 40])):
        st = status()
        out = torch.zeros_like(good)
        attention.attend_prompt(q, k, v, ac.i32(rows), ac.i32(keys), out=out, d_status=st)
        assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
        assert torch.equal(out[:10], good[:10])


def test_prompt_offsets_past_32_bits():
    """The last rows of a tensor of more than 2^31 elements."""
    H, K, D, T = 32, 8, 128, 700_000
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    kv = torch.empty(T, 2 * K, D, dtype=torch.bfloat16, device="cuda")
    a, b = T - 130, T - 3
    gen = torch.Generator("cuda").manual_seed(8)
    q[a:b] = torch.randn(b - a, H, D, device="cuda", generator=gen)
    kv[a:b] = torch.randn(b - a, 2 * K, D, device="cuda", generator=gen)
    cu = ac.i32([a, b])
    out = torch.zeros_like(q)
    attention.attend_prompt(q, kv[:, :K], kv[:, K:], cu, cu, out=out)
    one = ac.i32([0, b - a])
    want = attention.attend_prompt(q[a:b].clone(), kv[a:b, :K].clone(), kv[a:b, K:].clone(), one, one)
    assert torch.equal(out[a:b], want) and not out[b:].any() and not out[a - 200:a].any()


@pytest.mark.parametrize("D,H,K,dtype", [(64, 2, 1, "bf16"), (128, 2, 1, "fp16"), (64, 1, 1, "fp16"), (128, 4, 1, "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_rising_scores(D, H, K, dtype, causal):
    """Scores that rise by 12 in the exponent from 100 keys to the next in one row and fall or stay in others: the
    references move in several key tiles, in both row tiles and in a lone one."""
    rng = np.random.default_rng(D + H)
    n = 700
    q = ac.rows16(rng, (n, H, D), dtype, 0.05)
    k = ac.rows16(rng, (n, K, D), dtype, 0.05)
    v = ac.rows16(rng, (n, K, D), dtype)
    step = (np.arange(n) // 100)[:, None]
    k[:, :, 0] = step * 8.0
    q[:, :, 0] = np.array([1.0, -1.0, 0.0, 2.0])[np.arange(n) % 4][:, None]
    for rows in (n, 90):  # several row tiles; a lone one at the end of the keys
        cr, ck = ac.i32([0, rows]), ac.i32([0, n])
        x = q[n - rows:]
        out, lse = attention.attend_prompt(ac.dev(x, dtype), ac.dev(k, dtype), ac.dev(v, dtype), cr, ck, causal=causal,
                                           scale=1.0, return_lse=True)
        ac.check_attention(out, lse, x, k, v, 1.0, dtype, dtype, causal)


@pytest.mark.parametrize("H,K,D", [(96, 2, 64), (200, 1, 64), (130, 1, 128), (56, 8, 128), (1024, 1024, 64), (1024, 1, 64)])
def test_prompt_groups(H, K, D):
    """Groups that do not divide a row tile, and larger than one."""
    run_prompt([(5, 9), (11, 140)] if H < 1000 else [(3, 150)], H, K, D, "bf16", True, seed=H)


@pytest.mark.parametrize("B,longest", [(33, 60), (70, 200), (1100, 12)])
def test_prompt_many_sequences(B, longest):
    rng = np.random.default_rng(B)
    rows = rng.integers(0, longest, B)
    run_prompt([(int(n), int(n + x)) for n, x in zip(rows, rng.integers(0, 9, B))], 2, 1, 64, "fp16", True, seed=B)


# ------------------------------------------------------------------ paged cache

PAGED = [
    # (rows, length) of each sequence, heads, kv heads, D, page, dtype, max_rows
    ([(1, 1)], 1, 1, 128, 16, "bf16", 1),
    ([(1, 16), (1, 17), (1, 15), (1, 64), (1, 65)], 4, 1, 128, 16, "bf16", 1),
    ([(6, 100)], 8, 2, 128, 64, "bf16", 6),
    ([(6, 6), (6, 300), (6, 129)], 12, 3, 64, 32, "fp16", 6),
    ([(4, 2), (3, 0), (0, 50), (2, 2), (0, 0)], 4, 2, 128, 16, "bf16", 4),   # rows without keys, sequences without rows
    ([(1, 700), (2, 63), (8, 200), (3, 1000)], 8, 1, 64, 48, "bf16", 8),
    ([(1, 900)] * 3, 5, 5, 128, 128, "fp16", 1),
    ([(40, 500), (1, 31)], 8, 2, 128, 64, "bf16", 1),                         # more rows than announced
    ([(3, 77)], 64, 1, 64, 16, "fp16", 3),                                    # 192 rows on one kv head
    ([(2, 1500)], 32, 8, 128, 1024, "bf16", 1000),
]


def run_paged(seqs, H, K, D, page, dtype, max_rows, seed=0, sigma=1.0, vsigma=None):
    rng = np.random.default_rng(seed)
    lengths = [s[1] for s in seqs]
    c = ac.Cache(rng, lengths, K, D, page, sigma=sigma)
    cr = ac.offsets([s[0] for s in seqs])
    q = ac.rows16(rng, (cr[-1] + 2, H, D), dtype, 1.5)
    out = torch.full((cr[-1] + 2, H, D), 3.0, device="cuda").to(ac.TORCH[dtype])
    st = status()
    got, lse = attention.attend_paged(ac.dev(q, dtype), c.cache, c.table, ac.i32(lengths), ac.i32(cr), max_rows=max_rows,
                                      out=out, return_lse=True, d_status=st)
    assert st.item() == abi.MOE_OK
    assert (out[cr[-1]:] == 3).all()
    for b in range(len(seqs)):
        r = slice(cr[b], cr[b + 1])
        ac.check_attention(got[r], lse[r], q[r], c.k[b], c.v[b], D ** -0.5, dtype, "fp16")
    return c, q, got, lse


@pytest.mark.parametrize("case", PAGED, ids=[f"{c[0][0][0]}x{c[0][0][1]}_H{c[1]}_D{c[3]}_p{c[4]}_{c[5]}" for c in PAGED])
def test_paged_matches_the_oracle(case):
    run_paged(*case, seed=len(case[0]) + case[1])


@pytest.mark.parametrize("sigma", [2.0 ** -9, 2.0 ** 6, 20.0])
def test_paged_scales(sigma):
    run_paged([(3, 130), (1, 40)], 4, 2, 128, 16, "bf16", 3, seed=20, sigma=sigma)


def test_paged_long_sequence():
    run_paged([(2, 20011)], 4, 1, 128, 64, "bf16", 2, seed=21)


def test_paged_value_outliers():
    """Values 2^12 times the rest in a few tokens, and tiny ones: scales far apart within a tile."""
    rng = np.random.default_rng(22)
    n, H, K, D = 300, 4, 1, 128
    c = ac.Cache(rng, [n], K, D, 16)
    s = c.cache.v_scales
    table = c.table[0].long()
    for j, shift in ((7, 12), (100, 9), (101, -12), (250, 12)):
        s[table[j // 16], :, j % 16] += shift
        c.v[0][j] *= 2.0 ** shift
    q = ac.rows16(rng, (2, H, D), "bf16", 1.5)
    out, lse = attention.attend_paged(ac.dev(q, "bf16"), c.cache, c.table, ac.i32([n]), ac.i32([0, 2]), return_lse=True)
    ac.check_attention(out, lse, q, c.k[0], c.v[0], D ** -0.5, "bf16", "fp16")


def test_paged_strides():
    rng = np.random.default_rng(23)
    H, K, D = 8, 2, 64
    c = ac.Cache(rng, [90, 33], K, D, 32)
    q = ac.rows16(rng, (5, H + 3, D), "fp16", 1.5)
    out = torch.full((5, H + 2, D), 3.0, device="cuda").half()
    x = ac.dev(q, "fp16")
    got, lse = attention.attend_paged(x[:, 1:H + 1], c.cache, c.table, ac.i32([90, 33]), ac.i32([0, 2, 5]), out=out[:, :H],
                                      return_lse=True, max_rows=3)
    assert (out[:, H:] == 3).all()
    for b, r in ((0, slice(0, 2)), (1, slice(2, 5))):
        ac.check_attention(got[r], lse[r], q[r, 1:H + 1], c.k[b], c.v[b], D ** -0.5, "fp16", "fp16")


def test_paged_repeats_bit_for_bit():
    c, q, got, lse = run_paged([(6, 777), (2, 1200), (1, 30)], 8, 2, 128, 64, "bf16", 6, seed=24)
    x = ac.dev(q, "bf16")
    for _ in range(3):
        again, z = attention.attend_paged(x[:9], c.cache, c.table, ac.i32([777, 1200, 30]), ac.i32([0, 6, 8, 9]), max_rows=6,
                                          return_lse=True)
        assert torch.equal(again, got[:9]) and torch.equal(z, lse[:9])


def test_paged_reports_bad_pages_lengths_and_offsets():
    rng = np.random.default_rng(25)
    H, K, D = 4, 1, 128
    lengths = [70, 40]
    c = ac.Cache(rng, lengths, K, D, 16)
    q = torch.randn(4, H, D, device="cuda").bfloat16()
    cu = ac.i32([0, 2, 4])
    good = attention.attend_paged(q, c.cache, c.table, ac.i32(lengths), cu)
    bad_page, negative = c.table.clone(), c.table.clone()
    bad_page[1, 2], negative[1, 0] = 10 ** 6, -1
    for table, lens, rows in ((bad_page, lengths, [0, 2, 4]), (negative, lengths, [0, 2, 4]),
                              (c.table, [70, 10 ** 8], [0, 2, 4]), (c.table, [70, -5], [0, 2, 4]),
                              (c.table, lengths, [0, 2, 9]), (c.table, lengths, [0, 2, 1])):
        st = status()
        out = attention.attend_paged(q, c.cache, table, ac.i32(lens), ac.i32(rows), d_status=st)
        assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
        assert torch.equal(out[:2], good[:2])


def test_paged_offsets_past_32_bits():
    """Pages beyond 2^31 bytes of codes."""
    H, K, D, page, pages = 4, 8, 128, 64, 90_000
    c = attention.KVCacheMXFP4.empty(pages, page, K, D)
    small = attention.KVCacheMXFP4.empty(2, page, K, D)
    gen = torch.Generator("cuda").manual_seed(26)
    for a, b in ((small.k_codes, c.k_codes), (small.v_codes, c.v_codes)):
        a.copy_(torch.randint(0, 256, a.shape, device="cuda", generator=gen))
        b[-2:] = a
    for a, b in ((small.k_scales, c.k_scales), (small.v_scales, c.v_scales)):
        a.copy_(torch.randint(122, 128, a.shape, device="cuda", generator=gen))
        b[-2:] = a
    q = torch.randn(1, 2 * K, D, device="cuda", generator=gen).bfloat16()
    far = attention.attend_paged(q, c, ac.i32([[pages - 2, pages - 1]]), ac.i32([100]), ac.i32([0, 1]))
    near = attention.attend_paged(q, small, ac.i32([[0, 1]]), ac.i32([100]), ac.i32([0, 1]))
    assert torch.equal(far, near)
    # and an append there
    x = torch.randn(1, 3 * K, D, device="cuda", generator=gen).bfloat16()
    attention.qkv_append(x[:, :K], x[:, K:2 * K], x[:, 2 * K:], cache=c,
                         slots=torch.tensor([pages * page - 1], device="cuda"))
    codes, scales = quantize_mxfp4(x[:, 2 * K:].contiguous())
    assert torch.equal(c.v_codes[-1, :, -1], codes[0]) and torch.equal(c.v_scales[-1, :, -1], scales[0])


@pytest.mark.parametrize("case", [
    ([(4, 500), (2, 33)], 8, 2, 64, 16, "bf16", 4),       # 16 rows
    ([(4, 700), (3, 95)], 8, 2, 128, 64, "fp16", 4),
    ([(6, 300), (5, 1000), (6, 31)], 16, 2, 128, 32, "bf16", 6),  # 48 rows: two blocks of 24
    ([(8, 260), (8, 77)], 8, 2, 128, 16, "fp16", 8),      # 32 rows
    ([(8, 260), (7, 777)], 16, 4, 64, 64, "bf16", 8),
    ([(1, 333), (1, 2)], 8, 1, 64, 32, "fp16", 1),        # 8 rows
    ([(3, 500)], 130, 1, 64, 16, "bf16", 3),              # 390 rows of a head
], ids=lambda c: f"H{c[1]}_D{c[3]}_r{c[6]}_{c[5]}")
def test_paged_row_block_sizes(case):
    run_paged(*case, seed=case[1])


@pytest.mark.parametrize("B,longest,D,H,K,rows", [(33, 200, 64, 4, 2, 3), (70, 300, 128, 4, 1, 2), (1100, 40, 64, 2, 1, 2)])
def test_paged_many_sequences(B, longest, D, H, K, rows):
    """More sequences than a warp has lanes, and than a warp has lanes times lanes; some without rows or keys."""
    rng = np.random.default_rng(B)
    seqs = [(int(n), int(m)) for n, m in zip(rng.integers(0, rows + 1, B), rng.integers(0, longest, B))]
    run_paged(seqs, H, K, D, 16, "bf16", rows, seed=B)


@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_paged_other_scales(scale):
    rng = np.random.default_rng(27)
    n, H, K, D = 200, 6, 2, 64
    c = ac.Cache(rng, [n], K, D, 32)
    q = ac.rows16(rng, (2, H, D), "fp16", 1.5)
    out, lse = attention.attend_paged(ac.dev(q, "fp16"), c.cache, c.table, ac.i32([n]), ac.i32([0, 2]), scale=scale,
                                      max_rows=2, return_lse=True)
    ac.check_attention(out, lse, q, c.k[0], c.v[0], scale, "fp16", "fp16")


def test_paged_rising_scores():
    """Scores that rise by 2^4 in the exponent from stage to stage, and values whose scales do: every move of the
    references."""
    rng = np.random.default_rng(28)
    n, H, K, D = 1000, 8, 1, 128
    c = ac.Cache(rng, [n], K, D, 16, sigma=0.125)
    table = c.table[0].long()
    one = np.full((1, D // 2), 0x22, dtype=np.uint8)  # every code 1.0
    for j in range(n):  # keys: a constant row of 2^e with e rising, so that q . k rises
        page, at = table[j // 16], j % 16
        c.cache.k_codes[page, :, at] = torch.from_numpy(one).cuda()
        e = min(j // 64, 10)
        c.cache.k_scales[page, :, at] = 127 - 6 + e
        c.cache.v_scales[page, :, at] += j // 100
        c.k[0][j] = 2.0 ** (e - 6)
        c.v[0][j] *= 2.0 ** (j // 100)
    q = np.zeros((3, H, D))
    for r in range(3):
        for h in range(H):
            q[r, h, : 8 * (h + 1)] = (1, -1, 0.25)[r]
    out, lse = attention.attend_paged(ac.dev(q, "bf16"), c.cache, c.table, ac.i32([n]), ac.i32([0, 3]), max_rows=3,
                                      return_lse=True)
    ac.check_attention(out, lse, q, c.k[0], c.v[0], D ** -0.5, "bf16", "fp16")


def test_paged_sequences_that_share_pages():
    """One prefix in the tables of three sequences, and the same page twice in one table."""
    rng = np.random.default_rng(29)
    H, K, D, page = 8, 2, 64, 16
    c = ac.Cache(rng, [100], K, D, page)
    t = c.table[0].tolist()
    table = [t, t[:3] + [t[0], t[0]] + t[5:], t]
    lens = [100, 80, 37]
    q = ac.rows16(rng, (6, H, D), "bf16", 1.5)
    out, lse = attention.attend_paged(ac.dev(q, "bf16"), c.cache, ac.i32(table), ac.i32(lens), ac.i32([0, 2, 4, 6]),
                                      max_rows=2, return_lse=True)
    for b in range(3):
        at = np.array([t.index(table[b][j // page]) * page + j % page for j in range(lens[b])])
        r = slice(2 * b, 2 * b + 2)
        ac.check_attention(out[r], lse[r], q[r], c.k[0][at], c.v[0][at], D ** -0.5, "bf16", "fp16")


# ------------------------------------------------------------------ streams, graphs, a run of all

def test_other_streams_and_concurrent_calls():
    """Two streams at once, each with its own workspace, against the same calls one by one."""
    rng = np.random.default_rng(30)
    cases = []
    for lengths in ([3000, 100, 40], [50, 2500]):
        c = ac.Cache(rng, lengths, 2, 128, 64)
        q = torch.randn(len(lengths) * 2, 8, 128, device="cuda").bfloat16()
        cases.append((q, c.cache, c.table, ac.i32(lengths), ac.i32([2 * i for i in range(len(lengths) + 1)])))
    want = [attention.attend_paged(*x, max_rows=2) for x in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [attention.attend_paged(*x, max_rows=2, stream=s) for x, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


def test_graph_replay_follows_lengths_and_two_graphs_do_not_share():
    rng = np.random.default_rng(31)
    H, K, D, page = 8, 2, 128, 16
    c = ac.Cache(rng, [1000, 333], K, D, page)
    q = torch.randn(4, H, D, device="cuda").bfloat16()
    lens, cu = ac.i32([1000, 333]), ac.i32([0, 2, 4])
    calls = [(q, 2), (q * 0.5, 2)]
    for x, r in calls:
        attention.attend_paged(x, c.cache, c.table, lens, cu, max_rows=r)  # warm up before the capture
    graphs, outs = [], []
    for x, r in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attention.attend_paged(x, c.cache, c.table, lens, cu, max_rows=r))
        graphs.append(g)
    for a, b in ((1000, 333), (17, 300), (0, 1), (999, 2)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        want = [attention.attend_paged(x, c.cache, c.table, lens, cu, max_rows=r) for x, r in calls]
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for s, g in zip((s1, s2), graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_prompt_in_a_graph():
    x = torch.randn(300, 6, 128, device="cuda").bfloat16()
    cu = ac.i32([0, 100, 300])
    want = attention.attend_prompt(x[:, :4], x[:, 4:5], x[:, 5:], cu, cu)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = attention.attend_prompt(x[:, :4], x[:, 4:5], x[:, 5:], cu, cu)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)


def test_prompt_calls_at_once():
    cases = []
    for n, gen in ((400, 1), (90, 2)):
        x = torch.randn(n, 6, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(gen)).half()
        cases.append((x[:, :4], x[:, 4:5], x[:, 5:], ac.i32([0, n // 3, n]), ac.i32([0, n // 3, n])))
    want = [attention.attend_prompt(*c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = [torch.zeros_like(w) for w in want]
        torch.cuda.synchronize()
        for c, s, o in zip(cases, streams, outs):
            attention.attend_prompt(*c, out=o, stream=s)
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_append_in_a_graph_and_on_another_stream():
    """A captured append follows the positions and slots of its replay; one on another stream writes the same."""
    T, H, K, D, page = 12, 4, 2, 128, 16
    x = torch.randn(T, H + 2 * K, D, device="cuda", generator=torch.Generator("cuda").manual_seed(50)).bfloat16()
    rope = attention.rope_table(100, D)
    pos, slots = ac.i32(list(range(T))), torch.arange(T, device="cuda")
    parts = ("k_codes", "k_scales", "v_codes", "v_scales")
    caches = [attention.KVCacheMXFP4.empty(4, page, K, D) for _ in range(3)]

    def call(c, **kw):
        return attention.qkv_append(x[:, :H], x[:, H:H + K], x[:, H + K:], positions=pos, rope=rope, cache=c, slots=slots,
                                    **kw)["q"]

    call(caches[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = call(caches[0])
    pos.copy_(torch.arange(T, dtype=torch.int32) * 7)
    slots.copy_(torch.arange(T).flip(0) * 5)
    for c in caches:
        for part in parts:
            getattr(c, part).zero_()
    want = call(caches[1])
    torch.cuda.synchronize()
    g.replay()
    stream = torch.cuda.Stream()
    other = torch.zeros_like(want)
    torch.cuda.synchronize()
    call(caches[2], q_out=other, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(other, want)
    for part in parts:
        w = getattr(caches[1], part)
        assert w.any() and torch.equal(getattr(caches[0], part), w) and torch.equal(getattr(caches[2], part), w)


def test_streams_as_handles():
    """A raw handle, the legacy default stream's 0 among them; outputs belong to the call's stream."""
    x = torch.randn(40, 6, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(51)).bfloat16()
    cu = ac.i32([0, 40])
    c = ac.Cache(np.random.default_rng(52), [40], 1, 64, 16)
    args = x[:, :4], x[:, 4:5], x[:, 5:]
    want = (attention.qkv_append(*args)["q"], attention.attend_prompt(*args, cu, cu),
            attention.attend_paged(args[0], c.cache, c.table, ac.i32([40]), cu))
    lens = ac.i32([40])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s.cuda_stream, 0, s):
        got = (attention.qkv_append(*args, stream=handle)["q"], attention.attend_prompt(*args, cu, cu, stream=handle),
               attention.attend_paged(args[0], c.cache, c.table, lens, cu, stream=handle))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w)


@pytest.mark.parametrize("B,longest,H,K,D,dtype", [(250, 300, 4, 2, 128, "bf16"), (700, 40, 8, 4, 64, "fp16")])
def test_prompt_many_mixed_sequences(B, longest, H, K, D, dtype):
    """Far more row tiles than the GPU holds at once, of every kind in turn: without rows, without keys, with one row tile
    or two, with key tiles that end inside, at the end and behind a prefix."""
    rng = np.random.default_rng(B)
    rows = rng.integers(0, longest, B)
    extra = rng.choice([-longest, -5, 0, 3, 128, 300], B)
    run_prompt([(int(n), max(0, int(n + x))) for n, x in zip(rows, extra)], H, K, D, dtype, True, seed=B)


def test_prompt_mostly_empty_sequences():
    """4,096 sequences of which few have rows: searches far into the list, and many blocks past the last tile."""
    rng = np.random.default_rng(60)
    seqs = [(0, int(x)) for x in rng.integers(0, 3, 4096)]
    for b in rng.choice(4096, 30, replace=False):
        seqs[b] = (int(rng.integers(1, 90)), int(rng.integers(0, 200)))
    seqs[4095] = (33, 40)
    run_prompt(seqs, 4, 2, 64, "bf16", True, seed=61)


@pytest.mark.parametrize("seqs,H,K,D,dtype,causal", [
    ([(1, 2100)], 1, 1, 128, "bf16", True),
    ([(7, 5000)], 8, 2, 64, "fp16", True),
    ([(70, 3333)], 4, 1, 128, "fp16", True),                         # two row tiles
    ([(130, 2300)], 2, 2, 128, "bf16", False),
    ([(3, 4096), (0, 50), (5, 0), (9, 60), (2, 1500)], 4, 2, 64, "bf16", True),  # parts of one, two and more
    ([(2200, 2200)], 1, 1, 64, "bf16", True),                        # rows that see no key of the later parts
    ([(20, 2500)], 130, 1, 64, "bf16", True),
])
def test_prompt_few_rows_many_keys(seqs, H, K, D, dtype, causal):
    """The keys split over the GPU, and the same without a workspace."""
    run_prompt(seqs, H, K, D, dtype, causal, seed=H + D)
    gen = torch.Generator("cuda").manual_seed(70)
    n, m = sum(s[0] for s in seqs), sum(s[1] for s in seqs)
    make = lambda r, h: torch.randn(r, h, D, device="cuda", generator=gen).to(ac.TORCH[dtype])
    q, k, v = make(n, H), make(m, K), make(m, K)
    cu = [ac.i32(ac.offsets([s[i] for s in seqs])) for i in range(2)]
    st = status()
    split, z = attention.attend_prompt(q, k, v, *cu, causal=causal, return_lse=True, d_status=st)
    for _ in range(3):
        again = attention.attend_prompt(q, k, v, *cu, causal=causal, d_status=st)
        assert torch.equal(again, split)
    out, lse = torch.full_like(q, 3.0), torch.zeros(n, H, device="cuda")
    io = abi.MoeAttendPromptIO(q.data_ptr(), k.data_ptr(), v.data_ptr(), H * D, K * D, K * D, out.data_ptr(), H * D,
                               lse.data_ptr(), cu[0].data_ptr(), cu[1].data_ptr(), len(seqs), n, m, H, K, D,
                               abi.MOE_DTYPE_BF16 if dtype == "bf16" else abi.MOE_DTYPE_F16, int(causal), D ** -0.5)
    bytes = abi.moe_attend_prompt_workspace(io)
    assert bytes > 0
    assert abi.moe_attend_prompt(io, st, torch.cuda.current_stream()) == abi.MOE_OK and st.item() == abi.MOE_OK
    # both are within their bounds of one result: two roundings of o, and the probabilities' roundings of values of
    # about 1 (at most half a step of each value's weight, twice)
    half = ac.HALF_STEP[dtype]
    v_top = v.float().abs().max().item()
    assert ((out.float() - split.float()).abs() <= 2 * half * (out.float().abs() + 1.1 * v_top)).all()
    assert ((lse - z).abs()[torch.isfinite(z)] <= 1e-4).all() and torch.equal(torch.isinf(lse), torch.isinf(z))
    small = torch.empty(bytes - 4, dtype=torch.uint8, device="cuda")
    io.workspace, io.workspace_bytes = small.data_ptr(), bytes - 4
    assert abi.moe_attend_prompt(io, st, torch.cuda.current_stream()) == abi.MOE_ERR_INVALID_ARG


def test_split_prompts_in_graphs_and_on_streams():
    """Two captured calls with split keys replayed at once, following the offsets of their replay."""
    gen = torch.Generator("cuda").manual_seed(71)
    calls = []
    for n, m in ((5, 3000), (40, 2500)):
        x = torch.randn(m, 4, 64, device="cuda", generator=gen).bfloat16()
        calls.append((x[:n, :2], x[:, 2:3], x[:, 3:], ac.i32([0, n]), ac.i32([0, m])))
    graphs, outs = [], []
    for c in calls:
        attention.attend_prompt(*c)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(attention.attend_prompt(*c))
        graphs.append(g)
    for ends in ((3000, 2500), (1700, 900), (3, 2500)):
        for c, m in zip(calls, ends):
            c[4].copy_(torch.tensor([0, m], dtype=torch.int32))
        want = [attention.attend_prompt(*c) for c in calls]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_wrapper_refusals():
    """What the wrappers and entry points refuse, before anything runs on the GPU."""
    z = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
    q, k = z(4, 8, 64), z(4, 2, 64)
    cu, pos, slots = ac.i32([0, 4]), ac.i32([0, 1, 2, 3]), torch.arange(4, device="cuda")
    rope, cache, table, lens = attention.rope_table(8, 64), attention.KVCacheMXFP4.empty(2, 16, 2, 64), ac.i32([[0, 1]]), ac.i32([4])
    wrong = ValueError
    for error, match, call in (
        (wrong, "type of q", lambda: attention.qkv_append(q, k.half(), k)),
        (wrong, "contiguous", lambda: attention.qkv_append(q, k.transpose(1, 2).contiguous().transpose(1, 2), k)),
        (wrong, "k and v", lambda: attention.qkv_append(q, k[:3], k[:3])),
        (wrong, "together", lambda: attention.qkv_append(q, k, k, rope=rope)),
        (wrong, "together", lambda: attention.qkv_append(q, k, k, cache=cache)),
        (wrong, "positions", lambda: attention.qkv_append(q, k, k, rope=rope, positions=pos.long())),
        (wrong, "positions", lambda: attention.qkv_append(q, k, k, rope=rope, positions=pos[:3])),
        (wrong, "rope", lambda: attention.qkv_append(q, k, k, rope=rope.double(), positions=pos)),
        (wrong, "slots", lambda: attention.qkv_append(q, k, k, cache=cache, slots=slots.int())),
        (wrong, "slots", lambda: attention.qkv_append(q, k, k, cache=cache, slots=slots.cpu())),
        (wrong, "q_norm", lambda: attention.qkv_append(q, k, k, q_norm=z(32))),
        (wrong, "q_out", lambda: attention.qkv_append(q, k, k, q_out=z(4, 9, 64)[:, :8])),
        (wrong, "cache", lambda: attention.qkv_append(q, z(4, 4, 64), z(4, 4, 64), cache=cache, slots=slots)),
        (wrong, "d_status", lambda: attention.qkv_append(q, k, k, d_status=slots)),
        (wrong, "bf16 or fp16", lambda: attention.qkv_append(q.float(), k, k)),
        (TypeError, "tensor", lambda: attention.qkv_append(q, k, [1])),
        (abi.MoeError, None, lambda: attention.qkv_append(q, k, k, eps=float("nan"))),
        (abi.MoeError, None, lambda: attention.qkv_append(z(4, 8, 96), z(4, 2, 96), z(4, 2, 96))),
        (abi.MoeError, None, lambda: attention.qkv_append(q, z(4, 3, 64), z(4, 3, 64))),
        (wrong, "lengths", lambda: attention.attend_paged(q, cache, table, lens.long(), cu)),
        (wrong, "cu_rows", lambda: attention.attend_paged(q, cache, table, lens, ac.i32([0, 2, 4]))),
        (wrong, "page_table", lambda: attention.attend_paged(q, cache, table[0], lens, cu)),
        (wrong, "page_table", lambda: attention.attend_paged(q, cache, ac.i32([[0, 1], [0, 1]]), lens, cu)),
        (wrong, "cache", lambda: attention.attend_paged(z(4, 8, 128), cache, table, lens, cu)),
        (AttributeError, None, lambda: attention.attend_paged(q, k, table, lens, cu)),
        (wrong, "32 bits", lambda: attention.attend_paged(q, cache, table, lens, cu, max_rows=2 ** 40)),
        (abi.MoeError, None, lambda: attention.attend_paged(q, cache, table, lens, cu, max_rows=0)),
        (abi.MoeError, None, lambda: attention.attend_paged(q, cache, table, lens, cu, scale=1e300)),
        (TypeError, None, lambda: attention.attend_paged(q, cache, table, lens, cu, scale="1")),
        (wrong, "out", lambda: attention.attend_prompt(q, k, k, cu, cu, out=z(4, 8, 128))),
        (wrong, "cu_keys", lambda: attention.attend_prompt(q, k, k, cu, pos)),
        (wrong, "cu_rows", lambda: attention.attend_prompt(q, k, k, cu[:0], cu[:0])),
        (wrong, "k and v", lambda: attention.attend_prompt(q, k, k[:3], cu, cu)),
        (abi.MoeError, None, lambda: attention.attend_prompt(z(4, 516)[:, :512].view(4, 8, 64), k, k, cu, cu)),  # row stride
        (wrong, "k_scales", lambda: attention.KVCacheMXFP4(cache.k_codes, cache.k_codes, cache.v_codes, cache.v_scales)),
        (wrong, "dimensions", lambda: attention.KVCacheMXFP4(cache.k_codes[0], cache.k_scales, cache.v_codes, cache.v_scales)),
    ):
        with pytest.raises(error, match=match):
            call()


def test_calls_from_threads():
    """Three threads, each with its stream and its call, many times over."""
    import threading
    x = torch.randn(40, 6, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(53)).bfloat16()
    args, cu, lens = (x[:, :4], x[:, 4:5], x[:, 5:]), ac.i32([0, 40]), ac.i32([90])
    c = ac.Cache(np.random.default_rng(54), [90], 1, 64, 16)
    calls = [lambda: attention.qkv_append(*args)["q"], lambda: attention.attend_prompt(*args, cu, cu),
             lambda: attention.attend_paged(args[0], c.cache, c.table, lens, cu)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    got = [None] * 3

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()) as _:
            got[i] = [calls[i]() for _ in range(100)]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g, w in zip(got, want):
        assert len(g) == 100 and all(torch.equal(y, w) for y in g)


def test_layer_prompt_then_verify_steps():
    """A layer as a server runs it: a prompt through append and prompt attention, then steps of six rows through
    append, paged attention and the MoE step; the paged rows equal prompt attention over the cached values."""
    from moe_expert_layer_top_gb300 import synthetic
    from moe_expert_layer_top_gb300.layer import MoEStep
    gen = torch.Generator("cuda").manual_seed(40)
    H, K, D, page = 8, 2, 64, 16
    hidden = H * D
    lens = [45, 18]
    pages = [list(range(0, 5)), list(range(5, 10))]
    c = attention.KVCacheMXFP4.empty(10, page, K, D)
    table = ac.i32(pages)
    rope = attention.rope_table(200, D)
    kn = torch.ones(D, device="cuda").bfloat16()
    w = synthetic.make_weights(5, 8, hidden, 256)
    step = MoEStep(hidden, 256, 8, 2, w, 12)
    keys, values = [[], []], [[], []]

    def rows(counts, starts):
        n = sum(counts)
        x = torch.randn(n, H + 2 * K, D, device="cuda", generator=gen).bfloat16()
        pos = torch.cat([torch.arange(s, s + k) for s, k in zip(starts, counts)])
        slot = torch.tensor([pages[b][p // page] * page + p % page for b in range(2) for p in
                             range(starts[b], starts[b] + counts[b])], device="cuda")
        st = status()
        o = attention.qkv_append(x[:, :H], x[:, H:H + K], x[:, H + K:], positions=pos.int().cuda(), rope=rope,
                                 q_norm=kn, k_norm=kn, cache=c, slots=slot, cached_values=True, d_status=st)
        assert st.item() == abi.MOE_OK
        at = ac.offsets(counts)
        for b in range(2):
            keys[b].append(o["k_cached"][at[b]:at[b + 1]])
            values[b].append(o["v_cached"][at[b]:at[b + 1]])
        return o, at

    o, at = rows(lens, [0, 0])
    y = attention.attend_prompt(o["q"], o["k_cached"], o["v_cached"], ac.i32(at), ac.i32(at))
    assert torch.isfinite(y).all()
    for _ in range(3):
        o, at = rows([6, 6], lens)
        lens = [n + 6 for n in lens]
        y, lse = attention.attend_paged(o["q"], c, table, ac.i32(lens), ac.i32(at), max_rows=6, return_lse=True)
        for b in range(2):
            ac.check_attention(y[at[b]:at[b + 1]], lse[at[b]:at[b + 1]], ac.f64(o["q"][at[b]:at[b + 1]]),
                               ac.f64(torch.cat(keys[b])), ac.f64(torch.cat(values[b])), D ** -0.5, "bf16", "fp16")
        # the same rows by prompt attention over the cached values: both within their bounds of the same result
        far = attention.attend_prompt(o["q"], torch.cat(keys[0] + keys[1]), torch.cat(values[0] + values[1]), ac.i32(at),
                                      ac.i32(ac.offsets(lens)))
        assert (far.float() - y.float()).abs().max() <= 4 * 2.0 ** -8 * max(1.0, y.float().abs().max().item())
        x = y.reshape(12, hidden)
        out = step.forward_fused(x, w_router=torch.randn(8, hidden, device="cuda", generator=gen).bfloat16(),
                                 resid=x.view(12, 1, hidden).clone(), norm_weight=torch.ones(hidden, device="cuda").bfloat16())
        assert torch.isfinite(out["y"]).all()
    step.close()
