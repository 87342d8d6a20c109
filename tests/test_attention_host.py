"""Refusals of the attention calls. Everything here is decided on the host: no kernel runs, no GPU is needed."""
import ctypes

import pytest
import torch

import moe_expert_layer_top_gb300 as pkg
from moe_expert_layer_top_gb300 import abi, attention

INVALID, UNSUPPORTED = abi.MOE_ERR_INVALID_ARG, abi.MOE_ERR_UNSUPPORTED
P = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    pkg.build.build()
    return abi.load()


def cache(**kw):
    base = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, num_pages=4, page_size=64, num_kv_heads=8, head_dim=128)
    base.update(kw)
    return abi.MoeKvCache(**base)


def append_io(**kw):
    base = dict(q=P, k=P, v=P, q_stride=6144, k_stride=6144, v_stride=6144, num_tokens=6, num_heads=32,
                num_kv_heads=8, head_dim=128, dtype=abi.MOE_DTYPE_BF16, rotary_dim=128, interleaved=0,
                rope_positions=100, rope=P, positions=P, q_norm=P, k_norm=P, norm_eps=1e-6, slots=P, q_out=P,
                k_out=None, k_cached=None, v_cached=None)
    base.update(kw)
    return abi.MoeQkvAppendIO(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(num_tokens=-1), INVALID),
    (dict(num_heads=0), INVALID),
    (dict(num_heads=30), INVALID),                  # not a multiple of the kv heads
    (dict(head_dim=96), UNSUPPORTED),
    (dict(num_heads=2048), UNSUPPORTED),
    (dict(dtype=2), INVALID),
    (dict(rotary_dim=136), INVALID),
    (dict(rotary_dim=-16), INVALID),
    (dict(rotary_dim=63), INVALID),
    (dict(rotary_dim=24), UNSUPPORTED),             # not a multiple of 16
    (dict(norm_eps=float("nan")), INVALID),
    (dict(norm_eps=-1e-6), INVALID),
    (dict(norm_eps=float("inf")), INVALID),
    (dict(q=None), INVALID),
    (dict(k=P + 8), INVALID),
    (dict(q_out=None), INVALID),
    (dict(q_stride=4095), INVALID),
    (dict(q_stride=4100), INVALID),                 # not a multiple of 8
    (dict(v_stride=1016), INVALID),                 # shorter than a row
    (dict(k_cached=P + 2), INVALID),
    (dict(k_norm=P + 2), INVALID),
    (dict(rope=None), INVALID),
    (dict(positions=None), INVALID),
    (dict(rope_positions=0), INVALID),
    (dict(slots=None), INVALID),
    (dict(slots=P + 4), INVALID),
])
def test_append_refuses(lib, kw, expect):
    assert abi.moe_qkv_append(append_io(**kw), cache()) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(page_size=0), INVALID),
    (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=2048), UNSUPPORTED),
    (dict(num_pages=-1), INVALID),
    (dict(num_kv_heads=4), INVALID),                # not the call's
    (dict(head_dim=64), INVALID),
    (dict(head_dim=80), UNSUPPORTED),
    (dict(k_scales=None), INVALID),
    (dict(v_codes=P + 8), INVALID),
])
def test_append_refuses_caches(lib, kw, expect):
    assert abi.moe_qkv_append(append_io(), cache(**kw)) == expect


def test_append_null_and_empty(lib):
    assert lib.moe_qkv_append(None, None, None, None) == INVALID
    assert abi.moe_qkv_append(append_io(num_tokens=0, q=None), cache()) == abi.MOE_OK
    assert abi.moe_qkv_append(append_io(), cache(), d_status=P + 1) == INVALID


def paged_io(**kw):
    base = dict(q=P, q_stride=4096, out=P, out_stride=4096, lse=None, page_table=P, lengths=P, cu_rows=P, num_seqs=2,
                num_rows=12, max_pages=8, max_rows=6, num_heads=32, dtype=abi.MOE_DTYPE_BF16, scale=0.1)
    base.update(kw)
    return abi.MoeAttendPagedIO(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(num_heads=12), INVALID),
    (dict(num_heads=0), INVALID),
    (dict(dtype=7), INVALID),
    (dict(num_seqs=-1), INVALID),
    (dict(num_seqs=5000), UNSUPPORTED),
    (dict(num_rows=-1), INVALID),
    (dict(max_pages=-1), INVALID),
    (dict(max_pages=1 << 26), UNSUPPORTED),         # lengths past 2^30
    (dict(num_rows=1 << 27), UNSUPPORTED),          # 2^32 (row, head) pairs
    (dict(max_rows=0), INVALID),
    (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(q=None), INVALID),
    (dict(out=P + 8), INVALID),
    (dict(q_stride=4088), INVALID),
    (dict(out_stride=4097), INVALID),
    (dict(lengths=None), INVALID),
    (dict(cu_rows=P + 2), INVALID),
    (dict(page_table=None), INVALID),
    (dict(lse=P + 2), INVALID),
])
def test_paged_refuses(lib, kw, expect):
    assert abi.moe_attend_paged(paged_io(**kw), cache(), P, 1 << 40) == expect


def test_paged_null_and_empty(lib):
    assert lib.moe_attend_paged(None, None, None, 0, None, None) == INVALID
    assert abi.moe_attend_paged(paged_io(num_rows=0, q=None), cache(), None, 0) == abi.MOE_OK
    assert abi.moe_attend_paged(paged_io(num_seqs=0, cu_rows=None), cache(), None, 0) == abi.MOE_OK
    assert abi.moe_attend_paged(paged_io(), cache(k_codes=None), P, 1 << 40) == INVALID
    n = ctypes.c_int64(5)
    assert lib.moe_attend_paged_workspace(None, None, ctypes.byref(n)) == INVALID and n.value == 5


def prompt_io(**kw):
    base = dict(q=P, k=P, v=P, q_stride=4096, k_stride=1024, v_stride=1024, out=P, out_stride=4096, lse=None,
                cu_rows=P, cu_keys=P, num_seqs=2, num_rows=100, num_keys=100, num_heads=32, num_kv_heads=8,
                head_dim=128, dtype=abi.MOE_DTYPE_BF16, causal=1, scale=0.1)
    base.update(kw)
    return abi.MoeAttendPromptIO(**base)


@pytest.mark.parametrize("kw,expect", [
    (dict(num_heads=12), INVALID),
    (dict(num_kv_heads=0), INVALID),
    (dict(head_dim=256), UNSUPPORTED),
    (dict(dtype=3), INVALID),
    (dict(num_seqs=-2), INVALID),
    (dict(num_seqs=4097), UNSUPPORTED),
    (dict(num_rows=-1), INVALID),
    (dict(num_keys=-1), INVALID),
    (dict(num_rows=1 << 27), UNSUPPORTED),
    (dict(causal=2), INVALID),
    (dict(scale=float("-inf")), INVALID),
    (dict(q=P + 2), INVALID),
    (dict(out=None), INVALID),
    (dict(k=None), INVALID),
    (dict(v_stride=1000), INVALID),
    (dict(k_stride=1028), INVALID),
    (dict(cu_rows=None), INVALID),
    (dict(cu_keys=P + 1), INVALID),
])
def test_prompt_refuses(lib, kw, expect):
    assert abi.moe_attend_prompt(prompt_io(**kw)) == expect


def test_prompt_null_and_empty(lib):
    assert lib.moe_attend_prompt(None, None, None) == INVALID
    assert abi.moe_attend_prompt(prompt_io(num_rows=0, q=None)) == abi.MOE_OK
    assert abi.moe_attend_prompt(prompt_io(num_seqs=0)) == abi.MOE_OK


def test_wrapper_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attention.qkv_append(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        attention.attend_prompt(x, x, x, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="dimensions"):
        attention.qkv_append(x[0], x, x)
    u8 = torch.zeros(2, 8, 16, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_codes"):
        attention.KVCacheMXFP4(u8, u8, u8, u8)


def test_rope_table_is_the_formula_in_64_bits():
    t = attention.rope_table(70000, 64, 500000.0, device="cpu")
    assert t.shape == (70000, 64) and t.dtype == torch.float32
    i, p = 5, 69999
    angle = p * 500000.0 ** (-2 * i / 64)
    want = torch.tensor([angle], dtype=torch.float64)
    assert t[p, i].item() == want.cos().float().item() and t[p, 32 + i].item() == want.sin().float().item()
