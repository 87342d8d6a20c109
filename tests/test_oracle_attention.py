"""Pins of the attention oracle: torch in 64 bits, and closed forms."""
import numpy as np
import pytest
import torch

from oracle import attention as oa
import oracle


@pytest.mark.parametrize("dtype,t", [("bf16", torch.bfloat16), ("fp16", torch.float16)])
def test_round16_matches_torch_casts(dtype, t):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(20000) * 2.0 ** rng.integers(-30, 14, 20000)).astype(np.float32)
    want = torch.from_numpy(x).to(t).double().numpy()
    np.testing.assert_array_equal(oa.round16(x, dtype), want)


def test_round16_is_one_rounding():
    """Just above a tie by less than a binary32 step: a detour through binary32 would fall on the even side."""
    x = 1.0 + 2.0 ** -8 + 2.0 ** -40
    assert oa.round16(x, "bf16") == 1.0 + 2.0 ** -7
    assert torch.tensor(np.float32(x)).to(torch.bfloat16).item() == 1.0


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication_and_keeps_norms(interleaved):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 32))
    angle = rng.uniform(0, 7, (5, 8))
    y = oa.norm_rotate(x, None, 0.0, np.cos(angle), np.sin(angle), interleaved)
    np.testing.assert_array_equal(y[..., 16:], x[..., 16:])
    a, b = (x[..., 0:16:2], x[..., 1:16:2]) if interleaved else (x[..., :8], x[..., 8:16])
    c, d = (y[..., 0:16:2], y[..., 1:16:2]) if interleaved else (y[..., :8], y[..., 8:16])
    np.testing.assert_allclose(c + 1j * d, (a + 1j * b) * np.exp(1j * angle)[:, None], rtol=1e-12)


def test_norm_matches_torch():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((4, 2, 64)), rng.standard_normal(64)
    y = oa.norm_rotate(x, w, 1e-3, np.zeros((4, 0)), np.zeros((4, 0)), False)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x), (64,), torch.from_numpy(w), 1e-3).numpy()
    np.testing.assert_allclose(y, want, rtol=1e-12)


@pytest.mark.parametrize("n,m,causal", [(5, 5, True), (3, 9, True), (4, 6, False)])
def test_attend_matches_torch(n, m, causal):
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((n, 6, 16)), rng.standard_normal((m, 2, 16)), rng.standard_normal((m, 2, 16))
    out, lse, _, _ = oa.attend(q, k, v, 0.3, causal)
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, k.repeat(3, 1), v.repeat(3, 1)))
    mask = torch.ones(n, m, dtype=torch.bool).tril(m - n) if causal else None
    want = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=mask, scale=0.3).transpose(0, 1)
    np.testing.assert_allclose(out, want.numpy(), rtol=1e-11, atol=1e-13)
    s = 0.3 * torch.matmul(tq, tk.transpose(1, 2))
    if causal:
        s = s.masked_fill(~mask, -torch.inf)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).T.numpy(), rtol=1e-12)


def test_attend_rows_without_keys():
    q, k, v = np.ones((4, 2, 8)), np.ones((2, 1, 8)), np.full((2, 1, 8), 3.0)
    out, lse, _, _ = oa.attend(q, k, v, 1.0)
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()
    assert (out[2:] == 3).all() and np.allclose(lse[2:], [[8, 8], [8 + np.log(2)] * 2])


def test_a_transposed_mask_or_a_wrong_group_is_seen():
    """Planted mistakes move the result: the pins above are not blind to them."""
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((4, 4, 8)), rng.standard_normal((6, 2, 8)), rng.standard_normal((6, 2, 8))
    right = oa.attend(q, k, v, 0.5)[0]
    assert np.abs(oa.attend(q[::-1], k, v, 0.5)[0][::-1] - right).max() > 1e-2      # mask upside down
    assert np.abs(oa.attend(q, k[:, ::-1], v[:, ::-1], 0.5)[0] - right).max() > 1e-2  # heads of the wrong group
    assert oracle.mxfp4_quantize(np.zeros((1, 32)))[1][0, 0] == 0
