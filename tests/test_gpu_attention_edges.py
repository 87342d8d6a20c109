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


# ------------------------------------------------------------------ offsets out of order

ORDERED = [5 * b for b in range(101)]


def offset_cases():
    yield [0, 100, 2 ** 30, 300, 400, 500], ORDERED[:5] + [500]     # far out of range: two sequences are without rows
    yield [-5, 300, 300, 400, 500], [0, 300, 300, 400, 500]
    yield [0, 300, 300, 400, 500], [0, 300, 200, 450, 500]          # the keys' alone
    for at in (3, 31, 32, 33, 64, 97):                              # in, at the end of and behind a warp's 32 sequences
        for wrong in (-1, 501, 2 ** 31 - 1):
            yield ORDERED[:at] + [wrong] + ORDERED[at + 1:], ORDERED
        yield ORDERED, ORDERED[:at] + [-1] + ORDERED[at + 1:]


@pytest.mark.parametrize("keys_behind", [0, 3000])  # with split keys too
def test_prompt_with_an_offset_out_of_order(keys_behind):
    """The sequences in order have the results that they have alone, the rows of the others are not touched."""
    H, K, D, T = 8, 2, 64, 500
    m = T + keys_behind
    q, k, v = seeded(20, T, H, D).bfloat16(), seeded(21, m, K, D).bfloat16(), seeded(22, m, K, D).bfloat16()
    top = v.float().abs().max()
    for rows, keys in offset_cases():
        keys = keys[:-1] + [keys[-1] + keys_behind]
        out = torch.full((T, H, D), 7.0, device="cuda").bfloat16()
        st = status()
        attention.attend_prompt(q, k, v, ac.i32(rows), ac.i32(keys), out=out, d_status=st)
        assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
        want = torch.full_like(out, 7.0)
        for b in range(len(rows) - 1):
            if not (0 <= rows[b] < rows[b + 1] <= T and 0 <= keys[b] <= keys[b + 1] <= m):
                continue
            x, y = slice(rows[b], rows[b + 1]), slice(keys[b], keys[b + 1])
            got = attention.attend_prompt(q[x], k[y], v[y], ac.i32([0, x.stop - x.start]), ac.i32([0, y.stop - y.start]))
            # alone, the keys may be split otherwise: both are within their bounds of one result
            assert ((out[x].float() - got.float()).abs() <= 2 * 2.0 ** -8 * (got.float().abs() + 1.1 * top)).all()
            assert not (out[x] == 7).all(-1).any()
            want[x] = out[x]
        assert torch.equal(out, want), (rows, keys)


def test_prompt_with_overlapping_sequences():
    """More tiles than the grid is made for: reported, and nothing outside of the sequences' rows is touched."""
    H, K, D, T = 4, 1, 64, 520
    q, k, v = seeded(23, T, H, D).bfloat16(), seeded(24, T, K, D).bfloat16(), seeded(25, T, K, D).bfloat16()
    cu = ac.i32([0, 300, 100, 400, 500])
    out, st = torch.full((T, H, D), 7.0, device="cuda").bfloat16(), status()
    attention.attend_prompt(q, k, v, cu, ac.i32([0, 300, 300, 400, 500]), out=out, d_status=st)
    assert st.item() == abi.MOE_ERR_DEVICE_BOUNDS
    assert (out[500:] == 7).all() and not (out[:100] == 7).all(-1).any()


# ------------------------------------------------------------------ waits


def prompt_io(q, k, v, out, lse, cr, ck, dtype=abi.MOE_DTYPE_BF16, scale=None, **kw):
    (n, H, D), (m, K) = q.shape, k.shape[:2]
    return abi.MoeAttendPromptIO(q.data_ptr(), k.data_ptr(), v.data_ptr(), H * D, K * D, K * D, out.data_ptr(), H * D,
                                 lse.data_ptr(), cr.data_ptr(), ck.data_ptr(), len(cr) - 1, n, m, H, K, D,
                                 dtype, 1, D ** -0.5 if scale is None else scale, **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", [[70], [70] * 200])  # one work, and several a block
def test_prompt_wait_that_runs_out_is_reported(D, seqs):
    """The mark that nothing sets: the waits end at their bound (a second), the status says so, the next call is right."""
    T, H, K = sum(seqs), 8, 2
    q, k, v = seeded(30, T, H, D).bfloat16(), seeded(31, T, K, D).bfloat16(), seeded(32, T, K, D).bfloat16()
    cu = ac.i32(ac.offsets(seqs))
    want, z = attention.attend_prompt(q, k, v, cu, cu, return_lse=True)
    out, lse = torch.zeros_like(q), torch.zeros(T, H, device="cuda")
    for flags, code in ((abi.MOE_FLAG_TEST_SKIP_READY, abi.MOE_ERR_TIMEOUT), (0, abi.MOE_OK)):
        io, st = prompt_io(q, k, v, out, lse, cu, cu, flags=flags), status()
        assert abi.moe_attend_prompt(io, st, torch.cuda.current_stream()) == abi.MOE_OK
        torch.cuda.synchronize()
        assert st.item() == code
    assert torch.equal(out, want) and torch.equal(lse, z)


# ------------------------------------------------------------------ PyTorch's view of the calls

def test_outputs_that_are_given_and_the_cache_count_as_written():
    """A tensor that autograd holds for a backward pass and a call then writes is noticed there."""
    H, K, D, n = 4, 2, 64, 20
    q, k, v, cu = seeded(40, n, H, D).bfloat16(), seeded(41, n, K, D).bfloat16(), seeded(42, n, K, D).bfloat16(), ac.i32([0, n])
    c = attention.KVCacheMXFP4.empty(2, 16, K, D)
    parts = (c.k_codes, c.k_scales, c.v_codes, c.v_scales)
    slots, lens = torch.arange(n, device="cuda"), ac.i32([n])
    for given, call in (
        (parts, lambda out: attention.qkv_append(q, k, v, cache=c, slots=slots)),
        (None, lambda out: attention.qkv_append(q, k, v, q_out=out)["q"]),
        (None, lambda out: attention.attend_prompt(q, k, v, cu, cu, out=out)),
        (None, lambda out: attention.attend_paged(q, c, ac.i32([[0, 1]]), lens, cu, max_rows=n, out=out)),
    ):
        out = torch.empty_like(q)
        tensors = given or (out,)
        before = [t._version for t in tensors]
        call(out)
        assert [t._version for t in tensors] == [b + 1 for b in before]
    weight = torch.ones(n, H, D, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    held = torch.ones_like(q)
    loss = (weight * held).sum()
    attention.attend_prompt(q, k, v, cu, cu, out=held)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_calls_in_inference_mode_and_without_gradients():
    H, K, D, n = 4, 2, 64, 20
    q, k, v, cu = seeded(43, n, H, D).bfloat16(), seeded(44, n, K, D).bfloat16(), seeded(45, n, K, D).bfloat16(), ac.i32([0, n])
    want = attention.attend_prompt(q, k, v, cu, cu)
    with torch.no_grad():
        got = attention.attend_prompt(q.clone().requires_grad_(), k, v, cu, cu)
        assert torch.equal(got, want) and not got.requires_grad
    with torch.inference_mode():
        out = torch.empty_like(q)
        assert torch.equal(attention.attend_prompt(q.clone(), k, v, cu, cu, out=out), want)
        c = attention.KVCacheMXFP4.empty(2, 16, K, D)
        attention.qkv_append(q, k, v, cache=c, slots=torch.arange(n, device="cuda"))
    attention.attend_prompt(q, k, v, cu, cu, out=out)  # an inference tensor outside of it
    assert torch.equal(out, want)


FIRST_CALLS = """
import threading
import torch
from moe_expert_layer_top_gb300 import attention
x = torch.randn(60, 6, 64, device="cuda").bfloat16()
cu = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
start, got = threading.Barrier(8), [None] * 8

def work(i):
    with torch.cuda.stream(torch.cuda.Stream()):
        start.wait()
        y = x if i % 2 else x.half()
        got[i] = attention.attend_prompt(y[:, :4], y[:, 4:5], y[:, 5:], cu, cu)
        torch.cuda.current_stream().synchronize()

threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
for t in threads:
    t.start()
for t in threads:
    t.join()
for i in range(8):
    y = x if i % 2 else x.half()
    assert torch.equal(got[i], attention.attend_prompt(y[:, :4], y[:, 4:5], y[:, 5:], cu, cu))
print("same")
"""


def test_first_calls_of_a_process_from_threads():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr


# ------------------------------------------------------------------ many small weights

def check_small_weights(out, lse, q, k, v, scale, dtype):
    """As attention_cases.check_attention, but a weight (in f16, times 2^7 of the reference's, which is not above the
    row's largest) loses no more than half of f16's smallest step, 2^-25, in absolute terms: 2^-32 of the row's largest.
    Divided by the sum of the weights relative to the largest that is the part of |v| that may be lost."""
    n, H, D = q.shape
    m = len(k)
    o, z, spread, reach = oa.attend(q, k, v, scale)
    delta = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -21
    top = np.stack([(k[:, h // (H // k.shape[1])] @ q[:, h].T * scale).max(0) for h in range(H)], axis=1)  # one row: sees all
    lost = 2.0 ** -32 / np.exp(z - top)
    bound = ac.HALF_STEP[dtype] * np.abs(o) + 1.05 * (2.0 ** -11 + 2 * delta + 2 * m * 2.0 ** -24)[..., None] * spread
    bound += ac.HALF_TINY[dtype] + lost[..., None] * np.repeat(np.abs(v).sum(0)[None], H // k.shape[1], axis=1)
    err = np.abs(ac.f64(out) - o)
    assert (err <= bound).all(), f"{(err / bound).max():.2f} of its bound; {np.abs(err / o).max():.3f} of the result"
    assert (np.abs(ac.f64(lse) - z) <= delta + m * 2.0 ** -24 + 4 * 2.0 ** -24 * (np.abs(z) + reach)).all()


@pytest.mark.parametrize("below", [20.0, 24.0, 25.5, 26.0])  # binary orders of a weak key's weight below the strong one's
@pytest.mark.parametrize("split", [False, True])
def test_prompt_keeps_many_small_weights(below, split):
    """One strong key with value 0 in front of 65,536 weak ones with values of about 1, in fp16."""
    rng = np.random.default_rng(int(below))
    n, H, D = 65537, 2, 64
    k, v = ac.rows16(rng, (n, 1, D), "fp16", 0.01), 1 + ac.rows16(rng, (n, 1, D), "fp16", 0.25)
    v = oa.round16(v, "fp16")
    q = ac.rows16(rng, (1, H, D), "fp16", 0.25)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[0, :, 0], v[0] = oa.round16(below * np.log(2.0), "fp16"), 0.0
    t = [ac.dev(x, "fp16") for x in (q, k, v)]
    cu = ac.i32([0, 1]), ac.i32([0, n])
    if split:
        out, lse = attention.attend_prompt(*t, *cu, scale=1.0, return_lse=True)
    else:
        out, lse, st = torch.empty_like(t[0]), torch.empty(1, H, device="cuda"), status()
        io = prompt_io(*t, out, lse, *cu, dtype=abi.MOE_DTYPE_F16, scale=1.0)
        assert abi.moe_attend_prompt(io, st, torch.cuda.current_stream()) == abi.MOE_OK and st.item() == abi.MOE_OK
    check_small_weights(out, lse, q, k, v, 1.0, "fp16")


@pytest.mark.parametrize("below", [20.0, 24.0, 25.5, 26.0])
@pytest.mark.parametrize("rows", [1, 6])
def test_paged_keeps_many_small_weights(below, rows):
    """A strong key with value 0 among every 32 (each warp's stage has one), the others weak with values of about 1."""
    rng = np.random.default_rng(int(below) + rows)
    n, H, D, page = 8192, 4, 64, 64
    k, v = ac.rows16(rng, (n, 1, D), "bf16", 0.01), oa.round16(1 + ac.rows16(rng, (n, 1, D), "bf16", 0.25), "bf16")
    q = ac.rows16(rng, (rows, H, D), "bf16", 0.25)
    q[:, :, 0], k[:, :, 0] = oa.round16(below * np.log(2.0) / 6.0, "bf16"), 0.0
    k[5::32], v[5::32] = 0.0, 0.0
    k[5::32, :, 0] = 6.0
    c = attention.KVCacheMXFP4.empty(n // page, page, 1, D)
    kept = attention.qkv_append(ac.dev(q[:1].repeat(n, 0), "bf16"), ac.dev(k, "bf16"), ac.dev(v, "bf16"), cache=c,
                                slots=torch.arange(n, device="cuda"), cached_values=True)
    kk, vv = ac.f64(kept["k_cached"]), ac.f64(kept["v_cached"])
    table, lens, cu = ac.i32([list(range(n // page))]), ac.i32([n]), ac.i32([0, rows])
    out, lse = attention.attend_paged(ac.dev(q, "bf16"), c, table, lens, cu, max_rows=rows, scale=1.0, return_lse=True)
    for i in range(rows):
        end = n - rows + i + 1
        check_small_weights(out[i:i + 1], lse[i:i + 1], q[i:i + 1], kk[:end], vv[:end], 1.0, "bf16")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sigma,scale", [(30.0, 0.1), (1.0, 0.0), (1.0, -0.2), (2.0 ** -6, 0.1), (1.0, 3.0), (1.0, 1e-30), (0.01, 1e4)])
def test_prompt_scales_in_fp16(D, sigma, scale):
    """The reference stands 2^7 below the maximum: also where the scores in between are far apart, or all one."""
    rng = np.random.default_rng(D)
    H, K, seqs = 2, 1, [(150, 150), (10, 400)]
    cr, ck = ac.offsets([s[0] for s in seqs]), ac.offsets([s[1] for s in seqs])
    q, k = ac.rows16(rng, (cr[-1], H, D), "fp16", sigma), ac.rows16(rng, (ck[-1], K, D), "fp16", sigma)
    v = ac.rows16(rng, (ck[-1], K, D), "fp16")
    st = status()
    out, lse = attention.attend_prompt(ac.dev(q, "fp16"), ac.dev(k, "fp16"), ac.dev(v, "fp16"), ac.i32(cr), ac.i32(ck),
                                       scale=scale, return_lse=True, d_status=st)
    assert st.item() == abi.MOE_OK
    for b in range(2):
        r, s = slice(cr[b], cr[b + 1]), slice(ck[b], ck[b + 1])
        ac.check_attention(out[r], lse[r], q[r], k[s], v[s], scale, "fp16", "fp16")


@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16")])
@pytest.mark.parametrize("rows,keys,gone", [(40, 400, (0, 200)), (3, 5000, (0, 700)), (3, 5000, (1024, 1800)), (300, 300, (0, 140))])
@pytest.mark.parametrize("scale", [0.1, 2.0 ** -40, 1e9])
def test_prompt_key_tiles_without_a_weight(D, dtype, rows, keys, gone, scale):
    """A row's first key tiles (of all keys, or of a part) have scores of -inf, the others far below 0: the result is that
    of the others alone."""
    rng = np.random.default_rng(keys)
    H = 2
    q, k = ac.rows16(rng, (rows, H, D), dtype, 0.1), ac.rows16(rng, (keys, 1, D), dtype, 0.1)
    v = ac.rows16(rng, (keys, 1, D), dtype)
    q[:, :, 0], k[:, :, 0] = 64.0, -64.0
    if scale == 1e9:
        q[:, :, 1:] = 0.0  # one score for all: differences would be past any weight
    x = k.copy()
    x[gone[0]:gone[1], :, 0] = -np.inf
    out, lse = attention.attend_prompt(ac.dev(q, dtype), ac.dev(x, dtype), ac.dev(v, dtype), ac.i32([0, rows]),
                                       ac.i32([0, keys]), scale=scale, return_lse=True)
    left = np.r_[0:gone[0], gone[1]:keys]
    for i in range(0, rows, 7):
        see = left[left <= keys - rows + i]
        if len(see):
            ac.check_attention(out[i:i + 1], lse[i:i + 1], q[i:i + 1], k[see], v[see], scale, dtype, dtype)
        else:
            assert torch.isneginf(lse[i]).all() and not out[i].any()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("rows,keys", [(3, 40), (3, 3000)])
def test_scores_near_the_ends_of_binary32(rows, keys, sign):
    """All scores +-2^110 or so, a factor of 2^17 inside binary32: one weight for all keys that a row sees. In parts, some
    see none of them."""
    rng = np.random.default_rng(keys)
    H, D, page = 2, 64, 16
    q, k, v = np.zeros((rows, H, D)), np.zeros((keys, 1, D)), ac.rows16(rng, (keys, 1, D), "bf16")
    q[:, :, 0], k[:, :, 0] = 2.0 ** 60, sign * 2.0 ** 50
    cu, ck = ac.i32([0, rows]), ac.i32([0, keys])
    pages = -(-keys // page)
    c = attention.KVCacheMXFP4.empty(pages, page, 1, D)
    kept = attention.qkv_append(ac.dev(k.repeat(H, 1), "bf16"), ac.dev(k, "bf16"), ac.dev(v, "bf16"), cache=c,
                                slots=torch.arange(keys, device="cuda"), cached_values=True)
    assert np.array_equal(ac.f64(kept["k_cached"]), k)
    for what in ("prompt", "paged"):
        if what == "prompt":
            vv = v
            out, lse = attention.attend_prompt(ac.dev(q, "bf16"), ac.dev(k, "bf16"), ac.dev(v, "bf16"), cu, ck, scale=1.0,
                                               return_lse=True)
        else:
            vv = ac.f64(kept["v_cached"])
            out, lse = attention.attend_paged(ac.dev(q, "bf16"), c, ac.i32([list(range(pages))]), ac.i32([keys]), cu,
                                              max_rows=rows, scale=1.0, return_lse=True)
        for i in range(rows):
            see = vv[:keys - rows + i + 1, 0]
            want = see.mean(0)
            # weights are all 1: the output's rounding, and binary32 sums
            bound = ac.HALF_STEP["bf16"] * np.abs(want) + 2 * len(see) * 2.0 ** -24 * np.abs(see).mean(0)
            assert (np.abs(ac.f64(out[i]) - want) <= bound).all(), what
            assert (np.abs(ac.f64(lse[i]) / (sign * 2.0 ** 110) - 1) <= 2.0 ** -21).all(), what


@pytest.mark.parametrize("parts", [(1, 2, 3, 4), [1, 2, 3, 4], (1, 2), None])
def test_what_only_looks_like_a_cache_is_refused(parts):
    import types
    q, cu = seeded(60, 4, 8, 64).bfloat16(), ac.i32([0, 4])
    with pytest.raises(ValueError, match="KVCacheMXFP4"):
        attention.attend_paged(q, types.SimpleNamespace(_parts=parts), ac.i32([[0]]), ac.i32([4]), cu)


# ------------------------------------------------------------------ nothing to attend to

def test_calls_without_keys_rows_or_sequences():
    """Tensors of no rows: no keys at all, a cache of no pages, tables of no columns, no sequences, no rows."""
    H, K, D = 4, 2, 64
    q, none, cu = seeded(70, 3, H, D).bfloat16(), torch.empty(0, K, D, device="cuda").bfloat16(), ac.i32([0, 3])
    st = status()
    out, lse = attention.attend_prompt(q, none, none, cu, ac.i32([0, 0]), return_lse=True, d_status=st)
    assert not out.any() and torch.isneginf(lse).all()
    k = seeded(71, 5, K, D).bfloat16()
    assert attention.attend_prompt(q[:0], k, k, ac.i32([0, 0]), ac.i32([0, 5]), d_status=st).shape == (0, H, D)
    given = torch.full_like(q, 3.0)
    for rows in ([0], [0, 0, 0]):  # no sequences; sequences without rows
        keys = ac.i32([0] * len(rows))
        attention.attend_prompt(q, k, k, ac.i32(rows), keys, out=given, d_status=st)
    empty, c = attention.KVCacheMXFP4.empty(0, 16, K, D), attention.KVCacheMXFP4.empty(1, 16, K, D)
    for cache in (empty, c):
        for columns in (0, 1):
            table = torch.zeros(1, columns, dtype=torch.int32, device="cuda")
            out, lse = attention.attend_paged(q, cache, table, ac.i32([0]), cu, max_rows=3, return_lse=True, d_status=st)
            assert not out.any() and torch.isneginf(lse).all()
    attention.attend_paged(q, c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"), ac.i32([]), ac.i32([0]), out=given,
                           d_status=st)
    attention.attend_paged(q, c, ac.i32([[0]]), ac.i32([0]), ac.i32([0, 0]), out=given, d_status=st)
    assert attention.attend_paged(q[:0], c, ac.i32([[0]]), ac.i32([0]), ac.i32([0, 0]), d_status=st).shape == (0, H, D)
    o = attention.qkv_append(q, q[:, :K], q[:, :K], cache=empty, slots=torch.full((3,), -1, device="cuda"), d_status=st,
                             cached_values=True)
    assert torch.equal(o["q"], q) and o["k_cached"].shape == (3, K, D)
    assert st.item() == abi.MOE_OK and (given == 3).all()
