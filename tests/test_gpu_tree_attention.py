"""Attention of trees of drafted tokens on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from moe_expert_layer_top_gb300 import abi, attention

import attention_cases as ac
import tree_cases as tc
from tree_cases import run_tree, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_top_gb300.build as b
    b.build()
    abi.load()
    assert torch.cuda.is_available()


TREES = [
    # (rows, length) of each sequence, heads, kv heads, D, page, dtype, max_rows
    ([(1, 1)], 1, 1, 128, 16, "bf16", 1),
    ([(1, 16), (1, 17), (1, 15), (1, 64), (1, 65)], 4, 1, 128, 16, "bf16", 1),
    ([(6, 100)], 8, 2, 128, 64, "bf16", 6),
    ([(6, 6), (6, 300), (6, 129)], 12, 3, 64, 32, "fp16", 6),
    ([(4, 2), (3, 0), (0, 50), (2, 2), (0, 0)], 4, 2, 128, 16, "bf16", 4),   # rows without keys, sequences without rows
    ([(9, 700), (2, 63), (8, 200), (3, 1000)], 8, 1, 64, 48, "bf16", 9),
    ([(40, 500), (1, 31)], 8, 2, 128, 64, "bf16", 1),                         # more rows than announced
    ([(3, 77)], 64, 1, 64, 16, "fp16", 3),                                    # 192 rows on one kv head
    ([(32, 500)], 4, 1, 128, 64, "bf16", 32),                                 # 128 rows of a kv head
    ([(33, 500)], 4, 1, 128, 64, "fp16", 33),                                 # 132
    ([(64, 127), (64, 128), (64, 129)], 4, 1, 128, 64, "bf16", 64),           # 256, key tiles of 128 with cut ends
    ([(65, 300), (64, 64), (70, 69)], 4, 1, 128, 16, "fp16", 70),             # 260, no context, more rows than keys
    ([(61, 900), (17, 300), (1, 700), (30, 30)], 16, 2, 64, 16, "fp16", 61),
    ([(256, 1000)], 2, 1, 64, 128, "bf16", 256),                              # the largest tree
    ([(256, 400), (3, 90)], 5, 1, 128, 32, "bf16", 256),                      # 1280 rows of a kv head
    ([(100, 2100)], 1, 1, 128, 1024, "bf16", 100),
    ([(48, 257), (5, 640)], 24, 8, 128, 64, "bf16", 48),
    ([(61, 6000), (5, 7000), (40, 2500), (13, 5001)], 16, 2, 64, 16, "fp16", 61),  # long runs of key tiles
    ([(61, 6000), (5, 7000), (40, 2500), (13, 5001)], 8, 2, 128, 16, "bf16", 61),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", [1, 40])  # one item and several a block, shared and whole
def test_wait_that_runs_out_is_reported(D, seqs):
    """Keys that never come: the waits end at their bound (a second), the status says so, the next call is right."""
    H, K, rows, n = 8, 2, 40, 700
    rng = np.random.default_rng(30)
    c = ac.Cache(rng, [n] * seqs, K, D, 64)
    q = ac.dev(ac.rows16(rng, (rows * seqs, H, D), "bf16", 1.0), "bf16")
    parents, lens = ac.i32(list(range(-1, rows - 1)) * seqs), ac.i32([n] * seqs)
    cu = ac.i32(ac.offsets([rows] * seqs))
    want, z = attention.attend_tree(q, c.cache, c.table, lens, cu, parents, max_rows=rows, return_lse=True)
    out, lse = torch.zeros_like(q), torch.zeros(rows * seqs, H, device="cuda")
    for flags, code in ((abi.MOE_FLAG_TEST_SKIP_READY, abi.MOE_ERR_TIMEOUT), (0, abi.MOE_OK)):
        io = abi.MoeAttendTreeIO(
            abi.MoeAttendPagedIO(q.data_ptr(), H * D, out.data_ptr(), H * D, lse.data_ptr(), c.table.data_ptr(),
                                 lens.data_ptr(), cu.data_ptr(), seqs, rows * seqs, c.max_pages, rows, H,
                                 abi.MOE_DTYPE_BF16, D ** -0.5, flags), parents.data_ptr())
        kv, st = c.cache.as_abi(), status()
        size = abi.moe_attend_tree_workspace(io, kv)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        assert abi.moe_attend_tree(io, kv, ws, size, st, torch.cuda.current_stream()) == abi.MOE_OK
        torch.cuda.synchronize()
        assert st.item() == code
    assert torch.equal(out, want) and torch.equal(lse, z)


# Rows of a kv head and (sequence, kv head) pairs on both sides of where the kernels change.
BORDERS = [(tokens, group, seqs) for tokens, group in ((32, 1), (33, 1), (12, 4), (49, 1)) for seqs in (1, 16, 17)]


@pytest.mark.parametrize("tokens, group, seqs", BORDERS, ids=[f"{t * g}rows_{n}seqs" for t, g, n in BORDERS])
@pytest.mark.parametrize("D", [64, 128])
def test_either_kind_of_kernel(tokens, group, seqs, D):
    K = 2
    run_tree([(tokens, 200 + 7 * b) for b in range(seqs)], K * group, K, D, 16, "bf16", tokens, seed=tokens + seqs)


@pytest.mark.parametrize("case", TREES, ids=[f"{c[0][0][0]}x{c[0][0][1]}_H{c[1]}_D{c[3]}_p{c[4]}_{c[5]}" for c in TREES])
@pytest.mark.parametrize("kind", ["tree", "chain", "forest"])
def test_tree_matches_the_oracle(case, kind):
    run_tree(*case, seed=len(case[0]) + case[1], kind=kind)


@pytest.mark.parametrize("max_rows", [1, 4, 12, 32, 64, 256])
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16")])
def test_any_announced_size_gives_the_result(max_rows, D, dtype):
    """max_rows picks the kernel variant, whatever the sequences have."""
    run_tree([(1, 200), (37, 410), (0, 3), (9, 150), (70, 333)], 8, 2, D, 32, dtype, max_rows, seed=max_rows)


@pytest.mark.parametrize("rows", [3, 40])
@pytest.mark.parametrize("sigma", [2.0 ** -9, 2.0 ** 6, 20.0])
def test_tree_scales(sigma, rows):
    run_tree([(rows, 190), (1, 40)], 4, 2, 128, 16, "bf16", rows, seed=20, sigma=sigma)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
@pytest.mark.parametrize("rows", [3, 40])
def test_tree_other_scales(scale, rows):
    run_tree([(rows, 300)], 4, 1, 64, 32, "bf16", rows, seed=30, scale=scale)


@pytest.mark.parametrize("rows", [2, 64])
def test_tree_long_sequence(rows):
    run_tree([(rows, 20011)], 4, 1, 128, 64, "bf16", rows, seed=21)


def test_tree_many_sequences():
    rng = np.random.default_rng(3)
    run_tree([(int(n), int(n + x)) for n, x in zip(rng.integers(0, 20, 300), rng.integers(0, 90, 300))], 4, 1, 64, 16, "bf16",
             19, seed=4)


def test_tree_many_large_trees():
    rng = np.random.default_rng(5)
    run_tree([(int(n), int(n + x)) for n, x in zip(rng.integers(30, 90, 40), rng.integers(0, 500, 40))], 8, 2, 128, 32, "bf16",
             89, seed=6)


@pytest.mark.parametrize("rows", [2, 60])
def test_tree_value_and_key_outliers(rows):
    """Values and keys 2^12 times the rest in a few tokens, and tiny ones: scales far apart within a tile and between tiles."""
    rng = np.random.default_rng(22)
    n, H, K, D = 700, 4, 1, 128
    c = ac.Cache(rng, [n], K, D, 16)
    table = c.table[0].long()
    for s, rows64 in ((c.cache.v_scales, c.v[0]), (c.cache.k_scales, c.k[0])):
        for j, shift in ((7, 10), (100, 9), (101, -12), (250, -20), (400, 12 if rows64 is c.v[0] else 3)):
            s[table[j // 16], :, j % 16] += shift
            rows64[j] *= 2.0 ** shift
    q = ac.rows16(rng, (rows, H, D), "bf16", 0.02)
    parents = tc.random_tree(rng, rows)
    out, lse = attention.attend_tree(ac.dev(q, "bf16"), c.cache, c.table, ac.i32([n]), ac.i32([0, rows]), ac.i32(parents),
                                     max_rows=rows, return_lse=True)
    tc.check_tree(out, lse, q, c.k[0], c.v[0], parents, D ** -0.5, "bf16")


def test_a_chain_gives_what_paged_attention_gives():
    rng = np.random.default_rng(8)
    H, K, D, n = 8, 2, 128, 6
    c = ac.Cache(rng, [300, 41], K, D, 64)
    q = ac.dev(ac.rows16(rng, (2 * n, H, D), "bf16", 1.5), "bf16")
    args = q, c.cache, c.table, ac.i32([300, 41]), ac.i32([0, n, 2 * n])
    want, z = attention.attend_paged(*args, max_rows=n, return_lse=True)
    got, lse = attention.attend_tree(*args, ac.i32(list(range(-1, n - 1)) * 2), max_rows=n, return_lse=True)
    # one rounding of each to bf16, and weights in fp16
    assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -8)
    assert torch.allclose(lse, z, rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("rows", [5, 50])
def test_tree_strides_and_given_outputs(rows):
    rng = np.random.default_rng(23)
    H, K, D = 8, 2, 64
    c = ac.Cache(rng, [190, 133], K, D, 32)
    q = ac.rows16(rng, (2 * rows, H + 3, D), "fp16", 1.5)
    out = torch.full((2 * rows, H + 2, D), 3.0, device="cuda").half()
    trees = [tc.random_tree(rng, rows) for _ in range(2)]
    x = ac.dev(q, "fp16")
    version = out._version
    got, lse = attention.attend_tree(x[:, 1:H + 1], c.cache, c.table, ac.i32([190, 133]), ac.i32([0, rows, 2 * rows]),
                                     ac.i32(trees[0] + trees[1]), out=out[:, :H], return_lse=True, max_rows=rows)
    assert out._version > version and (out[:, H:] == 3).all()
    for b in range(2):
        r = slice(b * rows, (b + 1) * rows)
        tc.check_tree(got[r], lse[r], q[r, 1:H + 1], c.k[b], c.v[b], trees[b], D ** -0.5, "fp16")


@pytest.mark.parametrize("case", [([(6, 777), (2, 1200), (1, 30)], 8, 2, 128, 64, "bf16", 6),
                                  ([(64, 777), (20, 1200), (33, 130)], 8, 2, 128, 64, "bf16", 64)], ids=["small", "large"])
def test_tree_repeats_bit_for_bit(case):
    c, q, parents, cu, got, lse = run_tree(*case, seed=24)
    n = int(cu[-1])
    for _ in range(3):
        again, z = attention.attend_tree(ac.dev(q, "bf16")[:n], c.cache, c.table, ac.i32([s[1] for s in case[0]]), cu,
                                         parents[:n], max_rows=case[-1], return_lse=True)
        assert torch.equal(again, got[:n]) and torch.equal(z, lse[:n])


@pytest.mark.parametrize("rows", [2, 40])
def test_tree_reports_what_is_out_of_range(rows):
    rng = np.random.default_rng(25)
    H, K, D = 4, 1, 128
    lengths = [rows + 70, rows + 40]
    c = ac.Cache(rng, lengths, K, D, 16)
    q = torch.randn(2 * rows, H, D, device="cuda").bfloat16()
    cu, chain = [0, rows, 2 * rows], ac.i32(list(range(-1, rows - 1)) * 2)
    good = attention.attend_tree(q, c.cache, c.table, ac.i32(lengths), ac.i32(cu), chain, max_rows=rows)
    bad_page, negative = c.table.clone(), c.table.clone()
    bad_page[1, 2], negative[1, 0] = 10 ** 6, -1
    own, later = chain.clone(), chain.clone()
    own[rows + 1], later[rows] = 1, 2 ** 31 - 1
    for table, lens, offsets, parents in (
            (bad_page, lengths, cu, chain), (negative, lengths, cu, chain), (c.table, [lengths[0], 10 ** 8], cu, chain),
            (c.table, [lengths[0], -5], cu, chain), (c.table, lengths, [0, rows, 9 * rows], chain),
            (c.table, lengths, [0, rows, 1], chain), (c.table, lengths, cu, own), (c.table, lengths, cu, later)):
        st = status()
        out = attention.attend_tree(q, c.cache, table, ac.i32(lens), ac.i32(offsets), parents, max_rows=rows, d_status=st)
        assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
        assert torch.equal(out[:rows], good[:rows])


def test_a_parent_that_is_not_in_front_counts_as_none():
    rng = np.random.default_rng(26)
    c = ac.Cache(rng, [60], 1, 64, 16)
    q = ac.rows16(rng, (4, 2, 64), "bf16", 1.5)
    st = status()
    out = attention.attend_tree(ac.dev(q, "bf16"), c.cache, c.table, ac.i32([60]), ac.i32([0, 4]), ac.i32([-1, 0, 3, 2]),
                                max_rows=4, d_status=st)
    assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
    tc.check_tree(out, None, q, c.k[0], c.v[0], [-1, 0, -1, 2], 64 ** -0.5, "bf16")


@pytest.mark.parametrize("max_rows", [1, 256])
def test_a_tree_that_is_too_large_is_left_alone(max_rows):
    rng = np.random.default_rng(27)
    H, K, D = 2, 1, 64
    c = ac.Cache(rng, [400, 50], K, D, 16)
    q = ac.rows16(rng, (262, H, D), "bf16", 1.5)
    parents = list(range(-1, 256)) + [-1, 0, 0, 1, 1]
    out, st = torch.full((262, H, D), 3.0, device="cuda").bfloat16(), status()
    attention.attend_tree(ac.dev(q, "bf16"), c.cache, c.table, ac.i32([400, 50]), ac.i32([0, 257, 262]), ac.i32(parents),
                          max_rows=max_rows, out=out, d_status=st)
    assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
    assert (out[:257] == 3).all()
    tc.check_tree(out[257:], None, q[257:], c.k[1], c.v[1], parents[257:], D ** -0.5, "bf16")


@pytest.mark.parametrize("rows", [3, 40])
def test_tree_nan_of_a_row_that_is_not_seen(rows):
    """An infinite scale (code 255) in a drafted key that one row sees: the other rows and the other sequence stay finite."""
    rng = np.random.default_rng(28)
    H, K, D, m = 4, 1, 128, 200
    c = ac.Cache(rng, [m, m], K, D, 16)
    parents = [-1, 0, 0] + [2] * (rows - 3)
    at = m - rows + 1  # the key of row 1, which only row 1 sees
    c.cache.k_scales[int(c.table[0, at // 16]), 0, at % 16, 2] = 255
    q = ac.rows16(rng, (2 * rows, H, D), "bf16", 1.5)
    out, lse = attention.attend_tree(ac.dev(q, "bf16"), c.cache, c.table, ac.i32([m, m]), ac.i32([0, rows, 2 * rows]),
                                     ac.i32(parents * 2), max_rows=rows, return_lse=True)
    keep = [i for i in range(rows) if i != 1]
    want = tc.osp.attend_tree(q[:rows], c.k[0], c.v[0], parents, D ** -0.5)
    o, z = out[:rows].clone(), lse[:rows].clone()
    assert torch.isfinite(o[keep]).all() and torch.isfinite(z[keep]).all()
    o[1], z[1] = torch.from_numpy(want[0][1]).to(o), torch.from_numpy(want[1][1]).to(z)
    tc.check_tree(o, z, q[:rows], c.k[0], c.v[0], parents, D ** -0.5, "bf16")
    tc.check_tree(out[rows:], lse[rows:], q[rows:], c.k[1], c.v[1], parents, D ** -0.5, "bf16")


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("rows", [3, 40])
def test_tree_of_a_poisoned_query(rows, poison):
    rng = np.random.default_rng(29)
    H, K, D, m = 4, 1, 64, 300
    c = ac.Cache(rng, [m], K, D, 16)
    q = ac.rows16(rng, (rows, H, D), "bf16", 1.5)
    x = ac.dev(q, "bf16")
    x[1, 2, 5] = poison
    parents = tc.random_tree(rng, rows)
    out, lse = attention.attend_tree(x, c.cache, c.table, ac.i32([m]), ac.i32([0, rows]), ac.i32(parents), max_rows=rows,
                                     return_lse=True)
    assert out[1, 2].isnan().all() and lse[1, 2].isnan()
    q[1, 2] = 0.0
    o, z = out.clone(), lse.clone()
    clean = tc.osp.attend_tree(q, c.k[0], c.v[0], parents, D ** -0.5)
    o[1, 2] = torch.from_numpy(clean[0][1, 2]).to(o)
    z[1, 2] = float(clean[1][1, 2])
    tc.check_tree(o, z, q, c.k[0], c.v[0], parents, D ** -0.5, "bf16")


@pytest.mark.parametrize("rows", [3, 48])
def test_tree_rising_scores(rows):
    """The maximum moves in every key tile."""
    rng = np.random.default_rng(31)
    H, K, D, m = 4, 1, 128, 900
    c = ac.Cache(rng, [m], K, D, 16)
    shift = np.arange(m) // 100
    table = c.table[0].long()
    for j in range(m):
        c.cache.k_scales[table[j // 16], :, j % 16] += int(shift[j]) - 4
        c.k[0][j] *= 2.0 ** (int(shift[j]) - 4)
    q = ac.rows16(rng, (rows, H, D), "bf16", 1.0)
    parents = tc.random_tree(rng, rows)
    out, lse = attention.attend_tree(ac.dev(q, "bf16"), c.cache, c.table, ac.i32([m]), ac.i32([0, rows]), ac.i32(parents),
                                     max_rows=rows, return_lse=True)
    tc.check_tree(out, lse, q, c.k[0], c.v[0], parents, D ** -0.5, "bf16")


@pytest.mark.parametrize("rows", [4, 64])
def test_tree_offsets_past_32_bits(rows):
    """Pages beyond 2^31 bytes of codes."""
    H, K, D, page, pages = 8, 8, 128, 64, 90_000
    c = attention.KVCacheMXFP4.empty(pages, page, K, D)
    small = attention.KVCacheMXFP4.empty(3, page, K, D)
    gen = torch.Generator("cuda").manual_seed(26)
    high = torch.tensor([pages - 1, pages - 7, pages - 3], device="cuda")
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        t = getattr(small, name)
        t.copy_(torch.randint(0, 256 if "codes" in name else 4, t.shape, generator=gen, device="cuda"))
        if "scales" in name:
            t += 124
        getattr(c, name)[high] = t
    q = torch.randn(rows, H, D, device="cuda", generator=gen).bfloat16()
    parents = ac.i32(tc.random_tree(np.random.default_rng(1), rows))
    cu, lens = ac.i32([0, rows]), ac.i32([3 * page - 5])
    want = attention.attend_tree(q, small, ac.i32([[0, 1, 2]]), lens, cu, parents, max_rows=rows)
    got = attention.attend_tree(q, c, high.int()[None].contiguous(), lens, cu, parents, max_rows=rows)
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [5, 64])
def test_tree_on_streams_and_in_graphs(rows):
    """Two captured graphs, replayed with new lengths and parents, and eager calls on two streams at once."""
    rng = np.random.default_rng(33)
    H, K, D, B = 8, 2, 128, 3
    c = ac.Cache(rng, [600] * B, K, D, 64)
    cu = ac.i32([rows * i for i in range(B + 1)])
    q = [ac.dev(ac.rows16(rng, (B * rows, H, D), "bf16", 1.5), "bf16") for _ in range(2)]
    lens = [ac.i32([600, 300, 150]) for _ in range(2)]
    parents = [ac.i32(sum((tc.random_tree(rng, rows) for _ in range(B)), [])) for _ in range(2)]
    call = lambda i: attention.attend_tree(q[i], c.cache, c.table, lens[i], cu, parents[i], max_rows=rows, return_lse=True)
    want = [call(i) for i in range(2)]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for change in range(3):
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
        lens[change % 2].copy_(ac.i32([600 - 7 * change, 200 + change, 64 + rows]))
        parents[(change + 1) % 2].copy_(ac.i32(sum((tc.random_tree(rng, rows) for _ in range(B)), [])))
        want = [call(i) for i in range(2)]
    got = []
    for s, i in zip(streams, range(2)):
        s.wait_stream(torch.cuda.current_stream())
        got.append(attention.attend_tree(q[i], c.cache, c.table, lens[i], cu, parents[i], max_rows=rows, return_lse=True,
                                         stream=s if i else s.cuda_stream))
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def test_tree_wrapper_refusals():
    c = attention.KVCacheMXFP4.empty(4, 16, 2, 64)
    q = torch.zeros(4, 8, 64, device="cuda", dtype=torch.bfloat16)
    table, lens, cu, par = ac.i32([[0, 1]]), ac.i32([20]), ac.i32([0, 4]), ac.i32([-1, 0, 0, 1])
    good = (q, c, table, lens, cu, par)
    attention.attend_tree(*good)
    for at, value, match in ((5, par[:3], "parents"), (5, par.long(), "parents"), (5, par.cpu(), "parents"), (0, q.cpu(), "CUDA"),
                             (0, q.float(), "bf16"), (2, table[0], "page_table"), (3, lens.long(), "lengths"),
                             (4, cu[:1], "cu_rows"), (1, object(), None), (0, q.clone().requires_grad_(), "no backward")):
        args = list(good)
        args[at] = value
        with pytest.raises((ValueError, AttributeError), match=match):
            attention.attend_tree(*args)
    with pytest.raises(TypeError):
        attention.attend_tree(q, c, table, lens, cu, None)
    with pytest.raises(abi.MoeError):
        attention.attend_tree(*good, max_rows=0)
    with pytest.raises(abi.MoeError):
        attention.attend_tree(*good, scale=float("nan"))
